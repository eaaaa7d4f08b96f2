// gated_delta_sweep_bwd.cu -- the two sequential sweeps of the gated delta
// rule's backward: one forward, which keeps what the gradients read of the
// forward, and one in reverse (dv, the gradient of the state, the sums behind
// da and dbeta).  Both hold the transposed state's dv rows on the lanes of
// tensor memory, as the forward does (gated_delta_sweep_fwd.cu).
//
// Forward, per chunk, with T and P without their diagonals:
//   y  = G S K^T - R T^T,  R = V - y's first term      z = V - y,  V' = beta z
//   o' = S (scale G Q)^T + V' P^T                      o without the token's own part
//   S  = G_63 S + (e^{b_63 - b} V') K
// kept: S (bf16, and fp32 for the sums), y, V' (bf16), and sum_dv o'.dO per token.
//
// Reverse, with E the gradient of the state that leaves the chunk (beta here and in
// T: no nearer to zero than 2^-40; dv leaves with the factor that is missing):
//   dVs' = R (E K^T) + dO P,   dV' = dVs' + P_ii dO
//   dvs  = beta dVs' + (beta dV') T,   dv = dvs + beta P_ii dO
//   E    = G_63 E + dO (scale G Q) - (G dv) K
// and per token the sums over dv of dv.y + dvs.z and of dv.z.
//
// da is a sum in which most of o.dO and of v.dv cancel.  The token's own path
// through P, which cancels exactly, is left out of both (o', dvs); and what
// the state receives and gives back is taken in three bf16 terms (24 bits) so
// that both sides of the rest see the same numbers: V' and its scaled form
// forward, E in reverse.  With two terms everywhere da was off by 1e-5 (by
// 4e-5 under strong decays) against 5e-6 so.  Everything else has two terms
// against operands exact in bf16 (K, dO), or two against two (T, P, scale G Q).
//
// A CTA is bound by the chain of products and conversions, some 7,500 cycles a
// chunk forward and 8,700 in reverse; it takes most of tensor memory, so an SM
// holds one.
//
// Long sequences with few heads are therefore cut into segments that run at
// once, as in the forward: the states that enter them come from the same pass
// (on this direction's records); the gradients of the states that leave them
// from a reverse pass from zeros and a hand-over with A^T.  Whole backward of
// 16,384 tokens, in one piece and so: 4 heads of 96 x 192 2,248 us, 440 us; 16
// heads 2,444, 1,303; 48 heads of 128 x 128 (three segments) 3,939, 2,686; of
// 1,024 tokens and 8 heads of 64 x 64 151, 93.
#include "gated_delta_tc.cuh"

namespace gla {
namespace {

template <int DK>
struct FwdCols {
    static constexpr int S = 0;                 // state terms -> dS
    static constexpr int Y = DK;                // Y -> y -> W terms 0, 1
    static constexpr int R = DK + 64;           // -R terms -> W term 2
    static constexpr int V = DK + 128;          // V', three terms: 24 columns a step of 16 tokens
    static constexpr int O = DK + 224;          // o'
};
template <int DK>
struct RevCols {
    static constexpr int E = 0;                 // E, three terms: 24 columns a step of 16 dk columns
    static constexpr int D = DK * 3 / 2;        // what E receives
    static constexpr int Y = D + DK;            // E K^T -> beta dV' terms -> G dv terms
    static constexpr int PO = Y + 64;           // dO P -> beta dVs' -> dvs
    static constexpr int X = PO + 64;           // dO, one term, two chunks
};
constexpr uint32_t kAlloc = 512;

struct __align__(8) Bars {
    uint64_t full[2], empty[2];                 // K, scalars, V and dO
    uint64_t fq, ft, fp, eq, et, ep;            // Q, T, P
    uint64_t staged[2];                         // workers -> copies: dv is in the V slice (reverse)
    uint64_t s, r, w, o, x[2];                  // workers -> issuer
    uint64_t y, z, ds, out, drain;              // issuer -> workers
    uint64_t yin[kGdWorkers];                   // reverse: this warp's y is in its buffer
    uint32_t tmem;
};

// y of a warp's 32 rows and 32 tokens: pieces of 4 tokens, [8][32 lanes][4].
constexpr int kYBytes = 32 * 32 * 4;

template <int DK>
struct Smem {
    using Rec = GdRec<DK, true>;
    static constexpr int KSC = (Rec::KSC + 1023) / 1024 * 1024;
    static constexpr int Q = 2 * KSC, T = Q + 2 * DK * 128, P = T + 16384, V = P + 16384;
    // V and dO slices of two stages behind V, then y of each worker warp
    static constexpr int bytes(int sw) { return V + 4 * kGdC * sw * 2 + kGdWorkers * kYBytes + 1024; }
};

struct Cta {
    unsigned char *smem, *slices;
    const unsigned char* rec;
    int64_t rec_step, row0, nh, u0;
    int n, h, len, nc, w0, rows, sw, active;
    int64_t at;             // this segment's slot
    int c0;                 // its first chunk, an even one
    bool last;              // the sequence ends in it
    __device__ __forceinline__ unsigned char* slice(int which, int st) const     // 0: V, 1: dO
    {
        return slices + (st * 2 + which) * kGdC * sw * 2;
    }
};

// seg0: the first segment that has work here.
template <int DK>
__device__ __forceinline__ bool setup(Cta& x, Bars& B, const GdParams& p, int sw, int nslices, int seg0, unsigned char* raw)
{
    using Rec = GdRec<DK, true>;
    // the slices of a segment side by side, so that they share its records in L2
    const int piece = blockIdx.x / nslices, pair = piece / p.nseg, seg = piece - pair * p.nseg;
    x.n = pair / p.seqs.H;
    x.h = pair - x.n * p.seqs.H;
    p.seqs.span(x.n, x.row0, x.len);
    if (x.len < 0) {
        if (threadIdx.x == 0) record_status(p.status, GLA_ERR_INVALID_ARG);
        return false;
    }
    x.smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    x.slices = x.smem + Smem<DK>::V;
    x.sw = sw;
    x.w0 = (blockIdx.x - piece * nslices) * sw;
    x.rows = min(sw, p.dv - x.w0);
    const int64_t slot0 = p.seqs.slot0(x.n, x.row0), first = static_cast<int64_t>(seg) * p.seg_chunks;
    if (seg < seg0 || (seg > 0 && first * kGdC >= x.len)) return false;
    x.c0 = static_cast<int>(first);
    x.last = p.nseg == 1 || (first + p.seg_chunks) * kGdC >= x.len;
    if (p.nseg > 1) x.len = min(x.len - x.c0 * kGdC, p.seg_chunks * kGdC);
    x.row0 += first * kGdC;
    x.nc = (x.len + kGdC - 1) / kGdC;
    x.nh = static_cast<int64_t>(x.n) * p.seqs.H + x.h;
    x.at = x.nh * p.nseg + seg;
    x.u0 = (slot0 + first) * p.seqs.H + x.h;
    x.rec = p.rec + x.u0 * Rec::BYTES;
    x.rec_step = static_cast<int64_t>(p.seqs.H) * Rec::BYTES;
    x.active = 2 * (x.rows >> 5);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.full[i], 1);
            mbar_init(&B.empty[i], 1 + x.active);
            mbar_init(&B.staged[i], x.active);
            mbar_init(&B.x[i], x.active);
        }
        for (int i = 0; i < kGdWorkers; ++i) mbar_init(&B.yin[i], 1);
        uint64_t* single[11] = {&B.fq, &B.ft, &B.fp, &B.eq, &B.et, &B.ep, &B.y, &B.z, &B.ds, &B.out, &B.drain};
        for (uint64_t* b : single) mbar_init(b, 1);
        uint64_t* from_workers[4] = {&B.s, &B.r, &B.w, &B.o};
        for (uint64_t* b : from_workers) mbar_init(b, x.active);
        mbar_init_fence();
    }
    if (warp == kGdWorkers + 1) {
        tmem_alloc(&B.tmem, kAlloc);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return true;
}

// The copy warp's work (one lane): step i = 0 .. nc - 1 is chunk i, or nc - 1 - i
// in reverse, where the workers leave dv in the V slice for it to take away.
template <int DK, bool REV, bool PRE>
__device__ void copies(const Cta& x, Bars& B, const GdParams& p, const CUtensorMap* mv, const CUtensorMap* md,
                       const CUtensorMap* mo, const WaitCtl& ctl)
{
    using M = Smem<DK>;
    using Rec = GdRec<DK, true>;
    const uint32_t slice = kGdC * x.rows * 2;
    const int col = x.h * p.dv + x.w0;
    auto chunk = [&](int i) { return REV ? x.nc - 1 - i : i; };
    auto first = [&](int i) {
        const int st = i & 1, c = chunk(i), row = static_cast<int>(x.row0) + c * kGdC;
        mbar_arrive_expect_tx(&B.full[st], Rec::KSC + (PRE ? 1 : 2) * slice);
        bulk_load(x.smem + st * M::KSC, x.rec + c * x.rec_step, Rec::KSC, &B.full[st]);
        if (!PRE) tma_load_2d(x.slice(0, st), mv, &B.full[st], col, row);
        tma_load_2d(x.slice(1, st), md, &B.full[st], col, row);
    };
    auto tile = [&](int i, uint64_t* full, uint64_t* empty, int at, int from, uint32_t bytes) {
        if (i > 0 && !mbar_wait(empty, (i - 1) & 1, ctl)) return false;
        mbar_arrive_expect_tx(full, bytes);
        bulk_load(x.smem + at, x.rec + chunk(i) * x.rec_step + from, bytes, full);
        return true;
    };
    auto out = [&](int i) {                                  // false: the wait ran out
        const int st = i & 1, c = chunk(i), valid = x.len - c * kGdC;
        if (!mbar_wait(&B.staged[st], (i >> 1) & 1, ctl)) return false;
        const int64_t row = x.row0 + static_cast<int64_t>(c) * kGdC;
        if (valid >= kGdC) {
            tma_store_2d(mo, x.slice(0, st), col, static_cast<int>(row));
        } else {                                             // the rows behind are another sequence's
            const int64_t ld = static_cast<int64_t>(p.seqs.H) * p.dv;
            for (int r = 0; r < valid; ++r)
                bulk_store(p.dvv + (row + r) * ld + col, x.slice(0, st) + r * x.rows * 2, x.rows * 2);
        }
        tma_store_commit();
        tma_store_wait_read();
        return true;
    };
    bool ok = true;
    int a = 0, q = 0, t = 0, pp = 0;
    if (x.nc > 0) first(a++);
    for (int i = 0; i < x.nc; ++i) {
        // the tiles in the order of their use
        if (REV) {
            ok = tile(i, &B.fp, &B.ep, M::P, Rec::P, 16384);
            if (!ok) break;
            ++pp;
        }
        ok = tile(i, &B.fq, &B.eq, M::Q, Rec::Q, 2 * DK * 128);
        if (!ok) break;
        ++q;
        ok = tile(i, &B.ft, &B.et, M::T, Rec::T, 16384);
        if (!ok) break;
        ++t;
        if (!REV) {
            ok = tile(i, &B.fp, &B.ep, M::P, Rec::P, 16384);
            if (!ok) break;
            ++pp;
        }
        if (i > 0) {
            ok = (!REV || PRE || out(i - 1)) && (i + 1 >= x.nc || mbar_wait(&B.empty[(i - 1) & 1], ((i - 1) >> 1) & 1, ctl));
            if (!ok) break;
        }
        if (i + 1 < x.nc) first(a++);
    }
    if (REV && !PRE && ok && x.nc > 0) out(x.nc - 1);
    // no copy may be in flight when the block ends
    tma_store_wait_read();
    for (int i = max(0, a - 2); i < a; ++i) mbar_wait(&B.full[i & 1], (i >> 1) & 1, ctl);
    if (q > 0) mbar_wait(&B.fq, (q - 1) & 1, ctl);
    if (t > 0) mbar_wait(&B.ft, (t - 1) & 1, ctl);
    if (pp > 0) mbar_wait(&B.fp, (pp - 1) & 1, ctl);
}

// Sums of 32 values over the 32 lanes: lane t has the total of value t.
__device__ __forceinline__ float lane_sums(float (&v)[32], int lane)
{
#pragma unroll
    for (int half = 16; half >= 1; half >>= 1) {
        const bool up = (lane & half) != 0;
#pragma unroll
        for (int t = 0; t < half; ++t) {
            const float send = up ? v[t] : v[t + half];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, send, half);
            v[t] = (up ? v[t + half] : v[t]) + got;
        }
    }
    return v[0];
}
// bf16 tensors that the sweeps leave in memory lie in blocks of 32 dv rows and,
// in those, in pieces of 16 values, [dv / 32][piece][32][16]: a warp stores 1,024
// bytes in a row (32 bytes of each row, rows apart, cost the store path eight
// times the lines).  The tensor core reads them as they lie, with a 32-byte
// swizzle: the two halves of a row change places in every second four rows.
// (Pieces of 32 values and a 64-byte swizzle: 268 against 265 us here, and the
// products that read them no faster.)
__device__ __forceinline__ void store_piece(__nv_bfloat16* dst, const Cols16& x, int lane)
{
    uint32_t w[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = f2_to_bf16x2(x.p[i]);
    const bool swap = (lane & 4) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = swap ? w[i ^ 4] : w[i];
    st_global_v8(dst + lane * 16, v);
}
// A thread's half row of the state.
template <int HS>
__device__ __forceinline__ void store_half_row(__nv_bfloat16* dst, const f2 (&S)[HS / 2], int lane)
{
#pragma unroll
    for (int k = 0; k < HS / 16; ++k) store_piece(dst + k * kGdPiece, cols_of<HS>(S, k), lane);
}
__device__ __forceinline__ void split_pairs(float (&f)[32], int b, const Cols16& x)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 t = f2_get(x.p[i]);
        f[16 * b + 2 * i] = t.x;
        f[16 * b + 2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------- forward
template <int DK>
__global__ void __launch_bounds__(kGdThreads, 1)
gd_sweep_keep_kernel(GdParams p, const __grid_constant__ GdMap map_v, const __grid_constant__ GdMap map_d,
                     const __grid_constant__ GdMap, int sw, int nslices, WaitCtl ctl)
{
    using C = FwdCols<DK>;
    using M = Smem<DK>;
    using Rec = GdRec<DK, true>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Bars B;
    Cta x;
    if (!setup<DK>(x, B, p, sw, nslices, 0, smem_raw)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tm = B.tmem;
    if (warp == kGdWorkers) {
        if (lane == 0) {
            const bool whole = x.rows == sw;
            copies<DK, false, false>(x, B, p, whole ? &map_v.all : &map_v.last, whole ? &map_d.all : &map_d.last, nullptr, ctl);
        }
    } else if (warp == kGdWorkers + 1) {
        if (lane == 0) {
            const uint64_t q_k = smem_desc(smem_u32(x.smem + M::Q), 16, 512, kLayoutSW64);
            const uint64_t t_k = smem_desc(smem_u32(x.smem + M::T), 16, 1024, kLayoutSW128);
            const uint64_t p_k = smem_desc(smem_u32(x.smem + M::P), 16, 1024, kLayoutSW128);
            constexpr uint32_t id64 = idesc_bf16_f32(128, 64, 0, 0), idDk = idesc_bf16_f32(128, DK, 0, 1);
            for (int c = 0; c < x.nc; ++c) {
                const uint32_t st = smem_u32(x.smem + (c & 1) * M::KSC);
                const uint64_t k_k = smem_desc(st, 16, 512, kLayoutSW64), k_n = smem_desc(st, 4096, 512, kLayoutSW64);
                if (!mbar_wait(&B.full[c & 1], (c >> 1) & 1, ctl) || !mbar_wait(&B.s, c & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t b = desc_add(k_k, (k >> 1) * 4096 + (k & 1) * 32);
                    umma_bf16_ts(tm + C::Y, tm + C::S + 16 * k, b, id64, k > 0);
                    umma_bf16_ts(tm + C::Y, tm + C::S + 16 * k + 8, b, id64, 1);
                }
                umma_commit(&B.y);
                if (!mbar_wait(&B.ft, c & 1, ctl) || !mbar_wait(&B.r, c & 1, ctl)) break;
                tc_fence_after();
                // strictly lower triangular: step s reaches tokens 16 s on
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t id = idesc_bf16_f32(128, 64 - 16 * s, 0, 0);
                    const uint64_t hi = desc_add(t_k, 2048 * s + 32 * s), lo = desc_add(hi, 8192);
                    const uint32_t d = tm + C::Y + 16 * s, a = tm + C::R + 16 * s;
                    umma_bf16_ts(d, a, hi, id, 1);
                    umma_bf16_ts(d, a + 8, hi, id, 1);
                    umma_bf16_ts(d, a, lo, id, 1);
                }
                umma_commit(&B.z);
                umma_commit(&B.et);
                // o' of the state: while the workers turn z into V'
                if (c > 0 && !mbar_wait(&B.o, (c - 1) & 1, ctl)) break;
                if (!mbar_wait(&B.fq, c & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t hi = desc_add(q_k, (k >> 1) * 4096 + (k & 1) * 32), lo = desc_add(hi, DK * 128);
                    umma_bf16_ts(tm + C::O, tm + C::S + 16 * k, hi, id64, k > 0);
                    umma_bf16_ts(tm + C::O, tm + C::S + 16 * k + 8, hi, id64, 1);
                    umma_bf16_ts(tm + C::O, tm + C::S + 16 * k, lo, id64, 1);
                }
                umma_commit(&B.eq);
                if (!mbar_wait(&B.w, c & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint64_t b = desc_add(k_n, 1024 * s);
                    umma_bf16_ts(tm + C::S, tm + C::Y + 16 * s, b, idDk, s > 0);
                    umma_bf16_ts(tm + C::S, tm + C::Y + 16 * s + 8, b, idDk, 1);
                    umma_bf16_ts(tm + C::S, tm + C::R + 16 * s, b, idDk, 1);
                }
                umma_commit(&B.ds);
                if (!mbar_wait(&B.fp, c & 1, ctl)) break;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t id = idesc_bf16_f32(128, 64 - 16 * s, 0, 0);
                    const uint64_t hi = desc_add(p_k, 2048 * s + 32 * s), lo = desc_add(hi, 8192);
                    const uint32_t d = tm + C::O + 16 * s, a = tm + C::V + 24 * s;
                    umma_bf16_ts(d, a, hi, id, 1);
                    umma_bf16_ts(d, a + 8, hi, id, 1);
                    umma_bf16_ts(d, a + 16, hi, id, 1);
                    umma_bf16_ts(d, a, lo, id, 1);
                    umma_bf16_ts(d, a + 8, lo, id, 1);           // without it da is off by 1e-5
                }
                umma_commit(&B.out);
                umma_commit(&B.ep);
                umma_commit(&B.empty[c & 1]);
            }
            umma_commit(&B.drain);
            mbar_wait(&B.drain, 0, ctl);
        }
    } else if ((warp & 3) * 32 < x.rows) {
        const int half = warp >> 2, r = x.w0 + (warp & 3) * 32 + lane, wr = r >> 5, nwr = p.dv >> 5;
        const uint32_t t0 = tm + (static_cast<uint32_t>(warp & 3) << 21);
        constexpr int HS = DK / 2;
        f2 S[HS / 2];
        const float* from = p.nseg > 1 ? p.seg_l + x.at * DK * p.dv : p.s0 ? p.s0 + x.nh * DK * p.dv : nullptr;
        load_state<HS>(S, from ? from + half * HS * p.dv + r : nullptr, p.dv);
        auto put_state = [&]() {
#pragma unroll
            for (int k = 0; k < HS / 16; ++k) put_terms<2>(t0 + C::S + half * HS + 16 * k, cols_of<HS>(S, k));
        };
        // the state in fp32, as this thread holds it
        auto keep = [&](float* dst) {
#pragma unroll
            for (int i = 0; i < HS / 2; i += 2)
                *reinterpret_cast<ulonglong2*>(dst + 2 * i * 32) = make_ulonglong2(S[i].v, S[i + 1].v);
        };
        if (x.nc > 0) {
            put_state();
            warp_done(&B.s, lane);
        }
        bool ok = true;
        for (int c = 0; c < x.nc; ++c) {
            const int ph = c & 1, s = 2 * half;              // this thread's steps of 16 tokens: s and s + 1
            const int64_t u = x.u0 + static_cast<int64_t>(c) * p.seqs.H;
            const float* sc = reinterpret_cast<const float*>(x.smem + ph * M::KSC + Rec::SC) + 16 * s;
            const int at = 16 * s * x.rows + (warp & 3) * 32 + lane;          // this row's 32 tokens in a slice
            const __nv_bfloat16* vs = reinterpret_cast<const __nv_bfloat16*>(x.slice(0, ph)) + at;
            const __nv_bfloat16* ds = reinterpret_cast<const __nv_bfloat16*>(x.slice(1, ph)) + at;
            const int left = x.len - c * kGdC - 16 * s;
            ok = warp_wait(&B.full[ph], (c >> 1) & 1, ctl);
            if (!ok) break;
            Cols16 v[2], y[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) v[b] = load_row16(vs + 16 * b * x.rows, x.rows, left - 16 * b);
            ok = warp_wait(&B.y, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            get16x2(y[0], y[1], t0 + C::Y + 16 * s, t0 + C::Y + 16 * s + 16);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                y[b] = y[b] * load16(sc + kScG * kGdC + 16 * b);
                put16(t0 + C::Y + 16 * (s + b), y[b]);
                put_terms<2>(t0 + C::R + 16 * (s + b), y[b] - v[b]);
            }
            warp_done(&B.r, lane);
            // while the products run: the state that enters the chunk
            store_half_row<HS>(p.sb + ((u * nwr + wr) * (DK / 16) + half * (HS / 16)) * kGdPiece, S, lane);
            ok = warp_wait(&B.z, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            get16x2(y[0], y[1], t0 + C::Y + 16 * s, t0 + C::Y + 16 * s + 16);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                v[b] = load16(sc + kScBeta * kGdC + 16 * b) * (v[b] - y[b]);                 // V'
                put_terms<3>(t0 + C::V + 24 * (s + b), v[b], t0 + C::V + 24 * (s + b) + 16);
                // scaled: terms 0 and 1 over y, term 2 over R
                put_terms<3>(t0 + C::Y + 16 * (s + b), v[b] * load16(sc + kScR * kGdC + 16 * b), t0 + C::R + 16 * (s + b));
            }
            warp_done(&B.w, lane);
            const float gl = sc[kScG * kGdC + kGdC - 1 - 16 * s];
            Cols16 d[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) d[b] = load_row16(ds + 16 * b * x.rows, x.rows, left - 16 * b);
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.empty[ph]);        // scalars, V and dO are read
            float* yn = p.yn + ((u * nwr + wr) * 2 + half) * (32 * 32) + lane * 4;
            __nv_bfloat16* vp = p.vp + ((u * nwr + wr) * 8 + s) * kGdPiece;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                store_piece(vp + b * kGdPiece, v[b], lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<ulonglong2*>(yn + (16 * b + 4 * i) * 32) = make_ulonglong2(y[b].p[2 * i].v, y[b].p[2 * i + 1].v);
            }
            if (x.c0 + c > 0 && (c & 1) == 0) keep(p.sn + ((u * nwr + wr) * 2 + half) * (HS * 32) + lane * 4);
            ok = warp_wait(&B.ds, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            add_cols<HS>(S, t0 + C::S + half * HS, gl);
            if (c + 1 < x.nc) {
                put_state();
                warp_done(&B.s, lane);
            }
            ok = warp_wait(&B.out, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            get16x2(y[0], y[1], t0 + C::O + 16 * s, t0 + C::O + 16 * s + 16);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.o);
            float od[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) split_pairs(od, b, d[b] * y[b]);
            p.part[(u * 3 * nwr + wr) * kGdC + half * 32 + lane] = lane_sums(od, lane);
        }
        if (ok && x.last && p.ds_final) keep(p.sn_last + ((x.nh * nwr + wr) * 2 + half) * (HS * 32) + lane * 4);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kGdWorkers + 1) tmem_dealloc(tm, kAlloc);
}

// ---------------------------------------------------------------- reverse
// PRE: over all segments but the first, from a gradient of zeros, for what a
// segment itself gives its entering state's gradient; nothing else leaves.
template <int DK, bool PRE>
__global__ void __launch_bounds__(kGdThreads, 1)
gd_sweep_rev_kernel(GdParams p, const __grid_constant__ GdMap map_v, const __grid_constant__ GdMap map_d,
                    const __grid_constant__ GdMap map_dv, int sw, int nslices, WaitCtl ctl)
{
    using C = RevCols<DK>;
    using M = Smem<DK>;
    using Rec = GdRec<DK, true>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Bars B;
    Cta x;
    if (!setup<DK>(x, B, p, sw, nslices, PRE ? 1 : 0, smem_raw)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tm = B.tmem;
    if (warp == kGdWorkers) {
        if (lane == 0) {
            const bool whole = x.rows == sw;
            copies<DK, true, PRE>(x, B, p, whole ? &map_v.all : &map_v.last, whole ? &map_d.all : &map_d.last,
                                  whole ? &map_dv.all : &map_dv.last, ctl);
        }
    } else if (warp == kGdWorkers + 1) {
        if (lane == 0) {
            const uint64_t q_n = smem_desc(smem_u32(x.smem + M::Q), 4096, 512, kLayoutSW64);
            const uint64_t t_n = smem_desc(smem_u32(x.smem + M::T), 8192, 1024, kLayoutSW128);
            const uint64_t p_n = smem_desc(smem_u32(x.smem + M::P), 8192, 1024, kLayoutSW128);
            constexpr uint32_t id64 = idesc_bf16_f32(128, 64, 0, 0), idDk = idesc_bf16_f32(128, DK, 0, 1);
            for (int i = 0; i < x.nc; ++i) {
                const uint32_t st = smem_u32(x.smem + (i & 1) * M::KSC);
                const uint64_t k_k = smem_desc(st, 16, 512, kLayoutSW64), k_n = smem_desc(st, 4096, 512, kLayoutSW64);
                const uint32_t dO = tm + C::X + (i & 1) * 32;
                if (!mbar_wait(&B.full[i & 1], (i >> 1) & 1, ctl) || !mbar_wait(&B.s, i & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t b = desc_add(k_k, (k >> 1) * 4096 + (k & 1) * 32);
#pragma unroll
                    for (int n = 0; n < 3; ++n)
                        umma_bf16_ts(tm + C::Y, tm + C::E + 24 * k + 8 * n, b, id64, k > 0 || n > 0);
                }
                if (!mbar_wait(&B.fp, i & 1, ctl) || !mbar_wait(&B.x[i & 1], (i >> 1) & 1, ctl)) break;
                tc_fence_after();
                // tokens i of a step reach tokens up to their own block: the widest step first
#pragma unroll
                for (int s = 3; s >= 0; --s) {
                    const uint32_t id = idesc_bf16_f32(128, 16 * (s + 1), 0, 1);
                    umma_bf16_ts(tm + C::PO, dO + 8 * s, desc_add(p_n, 2048 * s), id, s < 3);
                    umma_bf16_ts(tm + C::PO, dO + 8 * s, desc_add(p_n, 8192 + 2048 * s), id, 1);
                }
                umma_commit(&B.y);
                umma_commit(&B.ep);
                if (!mbar_wait(&B.fq, i & 1, ctl)) break;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    umma_bf16_ts(tm + C::D, dO + 8 * s, desc_add(q_n, 1024 * s), idDk, s > 0);
                    umma_bf16_ts(tm + C::D, dO + 8 * s, desc_add(q_n, DK * 128 + 1024 * s), idDk, 1);
                }
                umma_commit(&B.eq);
                if (!mbar_wait(&B.ft, i & 1, ctl) || !mbar_wait(&B.r, i & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 3; s >= 0; --s) {
                    const uint32_t id = idesc_bf16_f32(128, 16 * (s + 1), 0, 1), a = tm + C::Y + 16 * s;
                    umma_bf16_ts(tm + C::PO, a, desc_add(t_n, 2048 * s), id, 1);
                    umma_bf16_ts(tm + C::PO, a + 8, desc_add(t_n, 2048 * s), id, 1);
                    umma_bf16_ts(tm + C::PO, a, desc_add(t_n, 8192 + 2048 * s), id, 1);
                }
                umma_commit(&B.z);
                umma_commit(&B.et);
                if (!mbar_wait(&B.w, i & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    umma_bf16_ts(tm + C::D, tm + C::Y + 16 * s, desc_add(k_n, 1024 * s), idDk, 1);
                    umma_bf16_ts(tm + C::D, tm + C::Y + 16 * s + 8, desc_add(k_n, 1024 * s), idDk, 1);
                }
                umma_commit(&B.ds);
                umma_commit(&B.empty[i & 1]);
            }
            umma_commit(&B.drain);
            mbar_wait(&B.drain, 0, ctl);
        }
    } else if ((warp & 3) * 32 < x.rows) {
        const int half = warp >> 2, r = x.w0 + (warp & 3) * 32 + lane, wr = r >> 5, nwr = p.dv >> 5;
        unsigned char* ybuf = x.slices + 4 * kGdC * x.sw * 2 + warp * kYBytes;
        const uint32_t t0 = tm + (static_cast<uint32_t>(warp & 3) << 21);
        constexpr int HS = DK / 2;
        const int s = 2 * half;                              // this thread's steps of 16 tokens: s and s + 1
        const int at = 16 * s * x.rows + (warp & 3) * 32 + lane;              // this row's 32 tokens in a slice
        f2 E[HS / 2];
        const float* from = PRE          ? nullptr
                            : p.nseg > 1 ? p.seg_e + x.at * DK * p.dv
                            : p.ds_final ? p.ds_final + x.nh * DK * p.dv
                                         : nullptr;
        load_state<HS>(E, from ? from + half * HS * p.dv + r : nullptr, p.dv);
        auto put_grad = [&]() {
#pragma unroll
            for (int k = 0; k < HS / 16; ++k) {
                const uint32_t t = t0 + C::E + half * (HS / 2 * 3) + 24 * k;
                put_terms<3>(t, cols_of<HS>(E, k), t + 16);
            }
        };
        // dO of step i into tensor memory, and for this thread
        uint32_t dw[2][8];
        auto put_dO = [&](int i) {
            const __nv_bfloat16* ds = reinterpret_cast<const __nv_bfloat16*>(x.slice(1, i & 1)) + at;
            const int left = x.len - (x.nc - 1 - i) * kGdC - 16 * s;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = 16 * b + 2 * j;
                    const uint32_t lo = __bfloat16_as_ushort(ds[t * x.rows]), hi = __bfloat16_as_ushort(ds[(t + 1) * x.rows]);
                    dw[b][j] = lo | (hi << 16);
                }
                if (left < 32) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int t = 16 * b + 2 * j;
                        dw[b][j] = t + 1 < left ? dw[b][j] : t < left ? dw[b][j] & 0xFFFFu : 0u;
                    }
                }
                tmem_st8(t0 + C::X + (i & 1) * 32 + half * 16 + 8 * b, dw[b]);
            }
            warp_done(&B.x[i & 1], lane);
        };
        bool ok = true;
        if (x.nc > 0) {
            put_grad();
            warp_done(&B.s, lane);
            ok = warp_wait(&B.full[0], 0, ctl);
            if (ok) put_dO(0);
        }
        for (int i = 0; ok && i < x.nc; ++i) {
            const int ph = i & 1, c = x.nc - 1 - i;
            const int64_t u = x.u0 + static_cast<int64_t>(c) * p.seqs.H;
            const float* sc = reinterpret_cast<const float*>(x.smem + ph * M::KSC + Rec::SC) + 16 * s;
            __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(x.slice(0, ph)) + at;
            const int left = x.len - c * kGdC - 16 * s;
            // while the first products run: <E, state leaving> (the sum of da's
            // terms over all later tokens; after every second chunk, the next one
            // into L2) and E rounded; y of the forward is on its way
            if (!PRE) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&B.yin[warp], kYBytes);
                    bulk_load(ybuf, p.yn + ((u * nwr + wr) * 2 + half) * (32 * 32), kYBytes, &B.yin[warp]);
                }
                if (i + 1 < x.nc && (c & 1) == 0) {
                    const float* b = p.sn + ((u * nwr + wr) * 2 + half) * (HS * 32);
                    for (int k = lane; k < HS; k += 32) prefetch_l2(b + k * 32);
                }
                float dot = 0.f;
                if (i > 0 || !x.last ? (c & 1) == 1 : p.ds_final != nullptr) {
                    const float* sn = (i > 0 || !x.last ? p.sn + (((u + p.seqs.H) * nwr + wr) * 2 + half) * (HS * 32)
                                                        : p.sn_last + ((x.nh * nwr + wr) * 2 + half) * (HS * 32)) + lane * 4;
                    f2 sum = f2_splat(0.f);
#pragma unroll
                    for (int k = 0; k < HS / 2; k += 2) {
                        const ulonglong2 w = __ldcs(reinterpret_cast<const ulonglong2*>(sn + 2 * k * 32));
                        f2 a, b;
                        a.v = w.x;
                        b.v = w.y;
                        sum = f2_fma(E[k + 1], b, f2_fma(E[k], a, sum));
                    }
                    const float2 t = f2_get(sum);
                    dot = t.x + t.y;
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
                }
                if (lane == 0) p.anch[(u * nwr + wr) * 2 + half] = dot;
                store_half_row<HS>(p.eb + ((u * nwr + wr) * (DK / 16) + half * (HS / 16)) * kGdPiece, E, lane);
            }
            Cols16 d[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const Cols16 f = load16(sc + kScBt * kGdC + 16 * b) * load16(sc + kScPd * kGdC + 16 * b);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[b].p[j] = f2_mul(f.p[j], f2_from_bf16x2(dw[b][j]));       // beta P_ii dO
            }
            ok = warp_wait(&B.y, ph, ctl);
            if (!ok) {                       // no copy may be in flight when the block ends
                if (!PRE) warp_wait(&B.yin[warp], i & 1, ctl);
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                Cols16 f, q;
                get16x2(f, q, t0 + C::Y + 16 * (s + b), t0 + C::PO + 16 * (s + b));
                f = load16(sc + kScBt * kGdC + 16 * b) * fma16(load16(sc + kScR * kGdC + 16 * b), f, q);
                put16(t0 + C::PO + 16 * (s + b), f);
                put_terms<2>(t0 + C::Y + 16 * (s + b), f + d[b]);
            }
            warp_done(&B.r, lane);
            if (i + 1 < x.nc) {
                ok = warp_wait(&B.full[ph ^ 1], ((i + 1) >> 1) & 1, ctl);
                if (!ok) {
                    if (!PRE) warp_wait(&B.yin[warp], i & 1, ctl);
                    break;
                }
                put_dO(i + 1);
            }
            ok = (PRE || warp_wait(&B.yin[warp], i & 1, ctl)) && warp_wait(&B.z, ph, ctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const Cols16 full = get16(t0 + C::PO + 16 * (s + b)) + d[b];                     // dv
                Cols16 g = load16(sc + kScG * kGdC + 16 * b) * full;
#pragma unroll
                for (int j = 0; j < 8; ++j) g.p[j] = f2_mul(g.p[j], f2_splat(-1.f));
                put_terms<2>(t0 + C::Y + 16 * (s + b), g);
            }
            warp_done(&B.w, lane);
            const float gl = sc[kScG * kGdC + kGdC - 1 - 16 * s];
            // what the chain does not wait for: while the products run
            float s1[32], s2[32];
#pragma unroll
            for (int b = 0; b < 2 && !PRE; ++b) {
                const Cols16 f = get16(t0 + C::PO + 16 * (s + b)), full = f + d[b];              // dvs, dv
                const Cols16 v = load_row16(vs + 16 * b * x.rows, x.rows, left - 16 * b);
                store_row16(vs + 16 * b * x.rows, x.rows, full);
                Cols16 y;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(ybuf + (4 * b + k) * 512 + lane * 16);
                    y.p[2 * k].v = w.x;
                    y.p[2 * k + 1].v = w.y;
                }
                // dv.y + dvs.z = dvs.v + (dv - dvs).y
                split_pairs(s1, b, fma16(f, v, d[b] * y));
                const Cols16 z = v - y;
                split_pairs(s2, b, full * z);
                // V' second term, from what this sweep has in hand: bytes cost the forward one more
                store_piece(p.vp + ((u * nwr + wr) * 8 + 4 + s + b) * kGdPiece, low16(load16(sc + kScBeta * kGdC + 16 * b) * z), lane);
            }
            // what beta has that beta~ has not, on the rounded rows: nearly always 1, and as a
            // factor of dv before its rounding it cost 2% of the backward
            if (!PRE && __any_sync(0xFFFFFFFFu, sc[kScF * kGdC + lane] != 1.f)) {
#pragma unroll 1
                for (int t = 0; t < 32; ++t)
                    vs[t * x.rows] = __float2bfloat16_rn(__bfloat162float(vs[t * x.rows]) * sc[kScF * kGdC + t]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&B.staged[ph]);
                mbar_arrive(&B.empty[ph]);
            }
            if (!PRE) {
                float* part = p.part + ((u * 3 + 1) * nwr + wr) * kGdC + half * 32 + lane;
                part[0] = lane_sums(s1, lane);
                part[static_cast<int64_t>(nwr) * kGdC] = lane_sums(s2, lane);
            }
            ok = warp_wait(&B.ds, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            add_cols<HS>(E, t0 + C::D + half * HS, gl);
            if (i + 1 < x.nc) {
                put_grad();
                warp_done(&B.s, lane);
            }
        }
        if (PRE) store_state<HS>(E, p.seg_e + (x.at * DK + half * HS) * p.dv + r, p.dv);
        else if (ok && x.c0 == 0 && p.ds0) store_state<HS>(E, p.ds0 + (x.nh * DK + half * HS) * p.dv + r, p.dv);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kGdWorkers + 1) tmem_dealloc(tm, kAlloc);
}

template <class K>
gla_status start(K kernel, const char* name, const GdParams& p, int smem, const GdMap& v, const GdMap& d, const GdMap& o,
                 const GdSlices& sl, const WaitCtl& ctl, cudaStream_t st)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    trace_begin(st);
    kernel<<<static_cast<unsigned>(p.seqs.N) * p.seqs.H * p.nseg * sl.n, kGdThreads, smem, st>>>(p, v, d, o, sl.width, sl.n, ctl);
    trace_end(st, name);
    count_launch();
    return check_launch(name);
}

template <int DK>
gla_status both(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    const GdSlices sl(p.dv);
    const int64_t width = static_cast<int64_t>(p.seqs.H) * p.dv;
    const int64_t tokens = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;
    GdMap v, d, dv;
    gla_status s;
    if ((s = gd_slice_map(&v, p.v, width, p.ld_v, tokens, sl.width, sl.last)) != GLA_OK ||
        (s = gd_slice_map(&d, p.dO, width, p.ld_do, tokens, sl.width, sl.last)) != GLA_OK ||
        (s = gd_slice_map(&dv, p.dvv, width, width, tokens, sl.width, sl.last)) != GLA_OK)
        return s;
    const int smem = Smem<DK>::bytes(sl.width);
    if ((s = start(gd_sweep_keep_kernel<DK>, "gd_sweep_keep_kernel", p, smem, v, d, dv, sl, ctl, st)) != GLA_OK) return s;
    if (p.nseg > 1) {
        if ((s = start(gd_sweep_rev_kernel<DK, true>, "gd_sweep_rev_segments_kernel", p, smem, v, d, dv, sl, ctl, st)) != GLA_OK ||
            (s = gd_launch_segment_grads(p, st)) != GLA_OK)
            return s;
    }
    return start(gd_sweep_rev_kernel<DK, false>, "gd_sweep_rev_kernel", p, smem, v, d, dv, sl, ctl, st);
}

}  // namespace

gla_status gd_launch_sweeps_bwd(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    switch (p.dk) {
    case 64: return both<64>(p, ctl, st);
    case 96: return both<96>(p, ctl, st);
    default: return both<128>(p, ctl, st);
    }
}

}  // namespace gla
