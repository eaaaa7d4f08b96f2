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
// kept: S (bf16, and fp32 for the sums), y, V', and sum_dv o'.dO per token.
//
// Reverse, with E the gradient of the state that leaves the chunk:
//   dVs' = R (E K^T) + dO P,   dV' = dVs' + P_ii dO
//   dvs  = beta dVs' + (beta dV') T,   dv = dvs + beta P_ii dO
//   E    = G_63 E + dO (scale G Q) - (G dv) K
// and per token the sums over dv of dv.y + dvs.z and of dv.z.
//
// da is a sum in which most of o.dO and of v.dv cancel.  The token's own path
// through P, which cancels exactly, is left out of both (o', dvs); and what
// the state receives and gives back is taken in three bf16 terms (24 bits) so
// that both sides of the rest see the same numbers: V' and its scaled form
// forward, E in reverse.  With two terms everywhere da was off by 9e-6 (by
// 4e-5 under strong decays) against 4e-6 so.  Everything else has two terms
// against operands exact in bf16 (K, dO), or two against two (T, P, scale G Q).
//
// A CTA is bound by the chain of products and conversions, some 5,500 cycles a
// chunk; it takes most of tensor memory, so an SM holds one.
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
    uint64_t staged[2];                         // workers -> copies: V' or dv is in the V slice
    uint64_t s, r, w, o, x[2];                  // workers -> issuer
    uint64_t y, z, ds, out, drain;              // issuer -> workers
    uint32_t tmem;
};

template <int DK>
struct Smem {
    using Rec = GdRec<DK, true>;
    static constexpr int KSC = (Rec::KSC + 1023) / 1024 * 1024;
    static constexpr int Q = 2 * KSC, T = Q + 2 * DK * 128, P = T + 16384, V = P + 16384;
    // V and dO slices of two stages behind V
    static constexpr int bytes(int sw) { return V + 4 * kGdC * sw * 2 + 1024; }
};

struct Cta {
    unsigned char *smem, *slices;
    const unsigned char* rec;
    int64_t rec_step, row0, nh, u0;
    int n, h, len, nc, w0, rows, sw, active;
    __device__ __forceinline__ unsigned char* slice(int which, int st) const     // 0: V, 1: dO
    {
        return slices + (st * 2 + which) * kGdC * sw * 2;
    }
};

template <int DK>
__device__ __forceinline__ bool setup(Cta& x, Bars& B, const GdParams& p, int sw, int nslices, unsigned char* raw)
{
    using Rec = GdRec<DK, true>;
    // the slices of a (sequence, head) side by side, so that they share its records in L2
    const int pair = blockIdx.x / nslices;
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
    x.w0 = (blockIdx.x - pair * nslices) * sw;
    x.rows = min(sw, p.dv - x.w0);
    x.nc = (x.len + kGdC - 1) / kGdC;
    x.nh = static_cast<int64_t>(x.n) * p.seqs.H + x.h;
    x.u0 = p.seqs.slot0(x.n, x.row0) * p.seqs.H + x.h;
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
// in reverse.  What the workers stage in the V slice goes to out, whose row of
// chunk c is out_row0 + c * out_step; whole: all 64 rows of every chunk leave.
template <int DK, bool REV>
__device__ void copies(const Cta& x, Bars& B, const GdParams& p, const CUtensorMap* mv, const CUtensorMap* md,
                       const CUtensorMap* mo, int64_t out_row0, int64_t out_step, int out_col, const WaitCtl& ctl)
{
    using M = Smem<DK>;
    using Rec = GdRec<DK, true>;
    const uint32_t slice = kGdC * x.rows * 2;
    const int col = x.h * p.dv + x.w0;
    auto chunk = [&](int i) { return REV ? x.nc - 1 - i : i; };
    auto first = [&](int i) {
        const int st = i & 1, c = chunk(i), row = static_cast<int>(x.row0) + c * kGdC;
        mbar_arrive_expect_tx(&B.full[st], Rec::KSC + 2 * slice);
        bulk_load(x.smem + st * M::KSC, x.rec + c * x.rec_step, Rec::KSC, &B.full[st]);
        tma_load_2d(x.slice(0, st), mv, &B.full[st], col, row);
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
        const int64_t row = out_row0 + c * out_step;
        if (!REV || valid >= kGdC) {
            tma_store_2d(mo, x.slice(0, st), out_col, static_cast<int>(row));
        } else {                                             // the rows behind are another sequence's
            const int64_t ld = static_cast<int64_t>(p.seqs.H) * p.dv;
            for (int r = 0; r < valid; ++r)
                bulk_store(p.dvv + (row + r) * ld + out_col, x.slice(0, st) + r * x.rows * 2, x.rows * 2);
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
            ok = out(i - 1) && (i + 1 >= x.nc || mbar_wait(&B.empty[(i - 1) & 1], ((i - 1) >> 1) & 1, ctl));
            if (!ok) break;
        }
        if (i + 1 < x.nc) first(a++);
    }
    if (ok && x.nc > 0) out(x.nc - 1);
    // no copy may be in flight when the block ends
    tma_store_wait_read();
    for (int i = max(0, a - 2); i < a; ++i) mbar_wait(&B.full[i & 1], (i >> 1) & 1, ctl);
    if (q > 0) mbar_wait(&B.fq, (q - 1) & 1, ctl);
    if (t > 0) mbar_wait(&B.ft, (t - 1) & 1, ctl);
    if (pp > 0) mbar_wait(&B.fp, (pp - 1) & 1, ctl);
}

// Sixteen fp32 values as NT bf16 terms of 8 columns, at taddr, + 8, + 16.
template <int NT>
__device__ __forceinline__ void put_terms(uint32_t taddr, float (&x)[16])
{
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            if (n + 1 < NT) {
                x[2 * i] -= bf16_lo(w[i]);
                x[2 * i + 1] -= bf16_hi(w[i]);
            }
        }
        tmem_st8(taddr + 8 * n, w);
    }
}
__device__ __forceinline__ void put16(uint32_t taddr, const float (&x)[16])
{
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
    tmem_st16(taddr, w);
}
// This row's 32 tokens of a slice, zeros from `left` on (what lies there is
// not the sequence's).  The loads do not wait for the comparison.
__device__ __forceinline__ void load_rows(float (&f)[32], const __nv_bfloat16* s, int stride, int left)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = __bfloat162float(s[i * stride]);
    if (left < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = i < left ? f[i] : 0.f;
    }
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// Arrive for this warp once its tensor-memory accesses are done.
__device__ __forceinline__ void warp_done(uint64_t* bar, int lane)
{
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
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
// A thread's state columns, rounded to bf16, to its half row of [dv][dk].
template <int HS>
__device__ __forceinline__ void store_half_row(__nv_bfloat16* dst, const float (&S)[HS])
{
#pragma unroll
    for (int k = 0; k < HS / 16; ++k) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack_bf16(S[16 * k + 2 * i], S[16 * k + 2 * i + 1]);
        st_global_v8(dst + 16 * k, w);
    }
}

// ---------------------------------------------------------------- forward
template <int DK>
__global__ void __launch_bounds__(kGdThreads, 1)
gd_sweep_keep_kernel(GdParams p, const __grid_constant__ GdMap map_v, const __grid_constant__ GdMap map_d,
                     const __grid_constant__ GdMap map_vp, int sw, int nslices, WaitCtl ctl)
{
    using C = FwdCols<DK>;
    using M = Smem<DK>;
    using Rec = GdRec<DK, true>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Bars B;
    Cta x;
    if (!setup<DK>(x, B, p, sw, nslices, smem_raw)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tm = B.tmem;

    if (warp == kGdWorkers) {
        if (lane == 0) {
            const bool whole = x.rows == sw;
            copies<DK, false>(x, B, p, whole ? &map_v.all : &map_v.last, whole ? &map_d.all : &map_d.last,
                              whole ? &map_vp.all : &map_vp.last, x.u0 * kGdC,
                              static_cast<int64_t>(p.seqs.H) * kGdC, x.w0, ctl);
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
        float S[HS];
        const float* s0 = p.s0 ? p.s0 + (x.nh * DK + half * HS) * p.dv + r : nullptr;
#pragma unroll
        for (int i = 0; i < HS; ++i) S[i] = s0 ? s0[static_cast<int64_t>(i) * p.dv] : 0.f;
        auto put_state = [&]() {
#pragma unroll
            for (int k = 0; k < HS / 16; ++k) {
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = S[16 * k + i];
                put_terms<2>(t0 + C::S + half * HS + 16 * k, f);
            }
        };
        // the state in fp32, as this thread holds it
        auto keep = [&](float* dst) {
#pragma unroll
            for (int i = 0; i < HS; i += 4)
                *reinterpret_cast<float4*>(dst + i * 32) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        };
        if (x.nc > 0) {
            put_state();
            warp_done(&B.s, lane);
        }
        bool ok = true;
        for (int c = 0; c < x.nc; ++c) {
            const int ph = c & 1;
            const int64_t u = x.u0 + static_cast<int64_t>(c) * p.seqs.H;
            const float* sc = reinterpret_cast<const float*>(x.smem + ph * M::KSC + Rec::SC);
            __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(x.slice(0, ph)) + half * 32 * x.rows + (warp & 3) * 32 + lane;
            const __nv_bfloat16* ds = reinterpret_cast<const __nv_bfloat16*>(x.slice(1, ph)) + (vs - reinterpret_cast<__nv_bfloat16*>(x.slice(0, ph)));
            const int left = x.len - c * kGdC - half * 32;
            ok = warp_wait(&B.full[ph], (c >> 1) & 1, ctl);
            if (!ok) break;
            float v[32];
            load_rows(v, vs, x.rows, left);
            ok = warp_wait(&B.y, ph, ctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int s = half * 2 + b;
                float f[16], G[16];
                load16(G, sc + kScG * kGdC + 16 * s);
                get16(f, t0 + C::Y + 16 * s);
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] *= G[i];
                put16(t0 + C::Y + 16 * s, f);
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] -= v[16 * b + i];
                put_terms<2>(t0 + C::R + 16 * s, f);
            }
            warp_done(&B.r, lane);
            // while the products run: the state that enters the chunk
            store_half_row<HS>(p.sb + (u * p.dv + r) * DK + half * HS, S);
            ok = warp_wait(&B.z, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            float* yn = p.yn + ((u * nwr + wr) * 2 + half) * (32 * 32) + lane * 4;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int s = half * 2 + b;
                float f[16], g[16];
                get16(f, t0 + C::Y + 16 * s);
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4*>(yn + (16 * b + i) * 32) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
                load16(g, sc + kScBeta * kGdC + 16 * s);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    f[i] = g[i] * (v[16 * b + i] - f[i]);
                    v[16 * b + i] = f[i];                    // V' from here on
                }
                load16(g, sc + kScR * kGdC + 16 * s);
#pragma unroll
                for (int i = 0; i < 16; ++i) g[i] *= f[i];
                put_terms<3>(t0 + C::V + 24 * s, f);
                // the scaled V': terms 0 and 1 over y, term 2 over R
                {
                    uint32_t w[8];
#pragma unroll
                    for (int n = 0; n < 3; ++n) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            w[i] = pack_bf16(g[2 * i], g[2 * i + 1]);
                            g[2 * i] -= bf16_lo(w[i]);
                            g[2 * i + 1] -= bf16_hi(w[i]);
                        }
                        tmem_st8(t0 + (n < 2 ? C::Y + 16 * s + 8 * n : C::R + 16 * s), w);
                    }
                }
            }
            warp_done(&B.w, lane);
            const float gl = sc[kScG * kGdC + kGdC - 1];
            float d[32];
            load_rows(d, ds, x.rows, left);
#pragma unroll
            for (int i = 0; i < 32; ++i) vs[i * x.rows] = __float2bfloat16_rn(v[i]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&B.staged[ph]);
                mbar_arrive(&B.empty[ph]);                   // scalars, V and dO are read
            }
            if (c > 0 && (c & 1) == 0) keep(p.sn + ((u * nwr + wr) * 2 + half) * (HS * 32) + lane * 4);
            ok = warp_wait(&B.ds, ph, ctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < HS / 16; ++k) {
                float f[16];
                get16(f, t0 + C::S + half * HS + 16 * k);
#pragma unroll
                for (int i = 0; i < 16; ++i) S[16 * k + i] = fmaf(gl, S[16 * k + i], f[i]);
            }
            if (c + 1 < x.nc) {
                put_state();
                warp_done(&B.s, lane);
            }
            ok = warp_wait(&B.out, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t o[32];
                tmem_ld32(t0 + C::O + half * 32, o);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.o);
#pragma unroll
                for (int i = 0; i < 32; ++i) d[i] *= __uint_as_float(o[i]);
            }
            p.part[(u * 3 * nwr + wr) * kGdC + half * 32 + lane] = lane_sums(d, lane);
        }
        if (ok && p.ds_final) keep(p.sn_last + ((x.nh * nwr + wr) * 2 + half) * (HS * 32) + lane * 4);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kGdWorkers + 1) tmem_dealloc(tm, kAlloc);
}

// ---------------------------------------------------------------- reverse
template <int DK>
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
    if (!setup<DK>(x, B, p, sw, nslices, smem_raw)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tm = B.tmem;

    if (warp == kGdWorkers) {
        if (lane == 0) {
            const bool whole = x.rows == sw;
            copies<DK, true>(x, B, p, whole ? &map_v.all : &map_v.last, whole ? &map_d.all : &map_d.last,
                             whole ? &map_dv.all : &map_dv.last, x.row0, kGdC, x.h * p.dv + x.w0, ctl);
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
        const uint32_t t0 = tm + (static_cast<uint32_t>(warp & 3) << 21);
        constexpr int HS = DK / 2;
        const int at = half * 32 * x.rows + (warp & 3) * 32 + lane;              // this row's tokens in a slice
        float E[HS];
        const float* e0 = p.ds_final ? p.ds_final + (x.nh * DK + half * HS) * p.dv + r : nullptr;
#pragma unroll
        for (int i = 0; i < HS; ++i) E[i] = e0 ? e0[static_cast<int64_t>(i) * p.dv] : 0.f;
        auto put_grad = [&]() {
#pragma unroll
            for (int k = 0; k < HS / 16; ++k) {
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = E[16 * k + i];
                put_terms<3>(t0 + C::E + half * (HS / 2 * 3) + 24 * k, f);
            }
        };
        // dO of step i into tensor memory
        auto put_dO = [&](int i) {
            const __nv_bfloat16* ds = reinterpret_cast<const __nv_bfloat16*>(x.slice(1, i & 1)) + at;
            const int left = x.len - (x.nc - 1 - i) * kGdC - half * 32;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = 16 * b + 2 * j;
                    const uint32_t lo = __bfloat16_as_ushort(ds[t * x.rows]), hi = __bfloat16_as_ushort(ds[(t + 1) * x.rows]);
                    w[j] = (t < left ? lo : 0u) | (t + 1 < left ? hi << 16 : 0u);
                }
                tmem_st8(t0 + C::X + (i & 1) * 32 + half * 16 + 8 * b, w);
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
            const float* sc = reinterpret_cast<const float*>(x.smem + ph * M::KSC + Rec::SC);
            __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(x.slice(0, ph)) + at;
            const __nv_bfloat16* ds = reinterpret_cast<const __nv_bfloat16*>(x.slice(1, ph)) + at;
            const int left = x.len - c * kGdC - half * 32;
            // while the first products run: <E, state leaving> (the sum of da's
            // terms over all later tokens; after every second chunk), E rounded,
            // and y from the forward; the next step's into L2
            if (i + 1 < x.nc) {
                const int64_t un = u - p.seqs.H;
                const char* a = reinterpret_cast<const char*>(p.yn + ((un * nwr + wr) * 2 + half) * (32 * 32));
                prefetch_l2(a + lane * 128);
                if ((c & 1) == 0) {
                    const char* b = reinterpret_cast<const char*>(p.sn + ((u * nwr + wr) * 2 + half) * (HS * 32));
                    for (int k = lane; k < HS; k += 32) prefetch_l2(b + k * 128);
                }
            }
            float dot = 0.f;
            if (i > 0 ? (c & 1) == 1 : p.ds_final != nullptr) {
                const float* sn = (i > 0 ? p.sn + (((u + p.seqs.H) * nwr + wr) * 2 + half) * (HS * 32)
                                         : p.sn_last + ((x.nh * nwr + wr) * 2 + half) * (HS * 32)) + lane * 4;
#pragma unroll
                for (int k = 0; k < HS; k += 4) {
                    const float4 s = __ldcs(reinterpret_cast<const float4*>(sn + k * 32));
                    dot += E[k] * s.x + E[k + 1] * s.y + E[k + 2] * s.z + E[k + 3] * s.w;
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
            }
            if (lane == 0) p.anch[(u * nwr + wr) * 2 + half] = dot;
            store_half_row<HS>(p.eb + (u * p.dv + r) * DK + half * HS, E);
            float4 yn[8];
            const float* yp = p.yn + ((u * nwr + wr) * 2 + half) * (32 * 32) + lane * 4;
#pragma unroll
            for (int k = 0; k < 8; ++k) yn[k] = __ldcs(reinterpret_cast<const float4*>(yp + k * 128));

            ok = warp_wait(&B.y, ph, ctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int s = half * 2 + b;
                float f[16], g[16], q[16];
                get16(f, t0 + C::Y + 16 * s);
                get16(q, t0 + C::PO + 16 * s);
                load16(g, sc + kScR * kGdC + 16 * s);
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = fmaf(g[j], f[j], q[j]);
                load16(g, sc + kScBeta * kGdC + 16 * s);
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] *= g[j];
                put16(t0 + C::PO + 16 * s, f);
                load16(q, sc + kScPd * kGdC + 16 * s);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float dO = __bfloat162float(ds[(16 * b + j) * x.rows]);
                    f[j] = 16 * b + j < left ? fmaf(g[j] * q[j], dO, f[j]) : 0.f;
                }
                put_terms<2>(t0 + C::Y + 16 * s, f);
            }
            warp_done(&B.r, lane);
            if (i + 1 < x.nc) {
                ok = warp_wait(&B.full[ph ^ 1], ((i + 1) >> 1) & 1, ctl);
                if (!ok) break;
                put_dO(i + 1);
            }
            ok = warp_wait(&B.z, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            float s1[32], s2[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int s = half * 2 + b;
                float f[16], g[16], q[16];
                get16(f, t0 + C::PO + 16 * s);               // dvs
                load16(g, sc + kScBeta * kGdC + 16 * s);
                load16(q, sc + kScPd * kGdC + 16 * s);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int t = 16 * b + j;
                    const bool in = t < left;
                    const float4 y4 = yn[t >> 2];
                    const float y = (t & 3) == 0 ? y4.x : (t & 3) == 1 ? y4.y : (t & 3) == 2 ? y4.z : y4.w;
                    const float v = __bfloat162float(vs[t * x.rows]), d = __bfloat162float(ds[t * x.rows]);
                    const float z = in ? v - y : 0.f, dO = in ? d : 0.f;
                    const float full = fmaf(g[j] * q[j], dO, f[j]);
                    s1[t] = fmaf(full, y, f[j] * z);
                    s2[t] = full * z;
                    f[j] = full;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) vs[(16 * b + j) * x.rows] = __float2bfloat16_rn(f[j]);
                load16(g, sc + kScG * kGdC + 16 * s);
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] *= -g[j];
                put_terms<2>(t0 + C::Y + 16 * s, f);
            }
            warp_done(&B.w, lane);
            const float gl = sc[kScG * kGdC + kGdC - 1];
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&B.staged[ph]);
                mbar_arrive(&B.empty[ph]);
            }
            float* part = p.part + ((u * 3 + 1) * nwr + wr) * kGdC + half * 32 + lane;
            part[0] = lane_sums(s1, lane);
            part[static_cast<int64_t>(nwr) * kGdC] = lane_sums(s2, lane);
            ok = warp_wait(&B.ds, ph, ctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < HS / 16; ++k) {
                float f[16];
                get16(f, t0 + C::D + half * HS + 16 * k);
#pragma unroll
                for (int j = 0; j < 16; ++j) E[16 * k + j] = fmaf(gl, E[16 * k + j], f[j]);
            }
            if (i + 1 < x.nc) {
                put_grad();
                warp_done(&B.s, lane);
            }
        }
        if (ok && p.ds0) {
            float* s = p.ds0 + (x.nh * DK + half * HS) * p.dv + r;
#pragma unroll
            for (int i = 0; i < HS; ++i) s[static_cast<int64_t>(i) * p.dv] = E[i];
        }
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
    kernel<<<static_cast<unsigned>(p.seqs.N) * p.seqs.H * sl.n, kGdThreads, smem, st>>>(p, v, d, o, sl.width, sl.n, ctl);
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
    GdMap v, d, vp, dv;
    gla_status s;
    if ((s = gd_slice_map(&v, p.v, width, p.ld_v, tokens, sl.width, sl.last)) != GLA_OK ||
        (s = gd_slice_map(&d, p.dO, width, p.ld_do, tokens, sl.width, sl.last)) != GLA_OK ||
        (s = gd_slice_map(&vp, p.vp, p.dv, p.dv, p.slots * p.seqs.H * kGdC, sl.width, sl.last)) != GLA_OK ||
        (s = gd_slice_map(&dv, p.dvv, width, width, tokens, sl.width, sl.last)) != GLA_OK)
        return s;
    const int smem = Smem<DK>::bytes(sl.width);
    if ((s = start(gd_sweep_keep_kernel<DK>, "gd_sweep_keep_kernel", p, smem, v, d, vp, sl, ctl, st)) != GLA_OK) return s;
    return start(gd_sweep_rev_kernel<DK>, "gd_sweep_rev_kernel", p, smem, v, d, dv, sl, ctl, st);
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
