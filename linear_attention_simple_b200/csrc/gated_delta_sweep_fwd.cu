// gated_delta_sweep_fwd.cu -- the forward sweep of the gated delta rule over a
// sequence's chunks: outputs and final state.
//
// The state is held transposed, [dv][dk], dv rows on the lanes of tensor
// memory, so that every left operand of the recurrence (the state, R, V', the
// update) comes from tensor memory and only the chunk's own operands (K, Q, T,
// P) pass through shared memory, brought whole by one bulk copy a chunk.  Per
// chunk, M = 128 lanes of dv rows, N tokens or dk columns:
//
//   Y  = S K^T            workers:  R  = V - G Y
//   O  = S Q^T                               scale G O
//   Z  = R T^T                      V' = beta Z,  W = (e^{b_63 - b} V')
//   dS = W K                        S  = G_63 S + dS   (fp32, in registers)
//   O += V' P^T                     o
//
// with T = (I + tril(K K^T . D beta_j, -1))^-1.  Worker threads hold one lane
// (dv row) and half of the columns.  S, R, W and V' enter as two bf16 terms
// against operands exact in bf16 (K, Q) or of two terms (T, P): 16 bits of each
// value, for the fp32 state; o's error is its own rounding.  (One term each of S,
// scale G Q, V' and P, as o leaves in bf16, put o 3.0e-3 from 64 bits where its
// rounding alone is 1.7e-3, and took 217 us for 8 x 2,048 tokens of 16 heads of
// 96 x 192 with the chunks' kernel, 228 so.)
//
// V is read from a shared [token][row] slice and o leaves through the same
// one, two stages, each a single tensor copy (a bulk copy per token row was
// measured at twice the whole kernel's time: the copy unit takes some 80
// cycles for each, however short).  Each step waits for the one before, so a
// CTA is bound by the chain of small products and conversions; two CTAs share
// an SM (256 columns of tensor memory and about 100 KB each at dk <= 96) and
// fill each other's gaps.
//
// With few (sequence, head) pairs a long sequence is cut into segments that
// run at once.  A segment is linear in the state that enters it, S_out = A
// S_in + L, so a pass over all segments but the last finds L (from a state of
// zeros) and A (the same sweep with V = 0 from the identity: dk more rows), a
// small fp32 kernel hands the states on from segment to segment, and the sweep
// proper starts every segment from its own.  The pass needs neither Q, P nor o:
// two of its CTAs share an SM at dk = 128 too (169 us with one each, 143 so).
// One prompt of 16,384 tokens at 16 heads of 128 x 128: 858 us in one piece, 287
// us so (143 + 31 + 113).
#include "gated_delta_tc.cuh"

namespace gla {
namespace {

// Tensor memory columns.
template <int DK>
struct Cols {
    static constexpr int S = 0;                      // state terms -> Z -> dS
    static constexpr int Y = DK;                     // Y -> R terms -> W terms
    static constexpr int V = DK + 64;                // V'
    // V' second term: where two CTAs share an SM at dk = 96 all columns are taken,
    // but the last 32 of the state's are free between Z and dS
    static constexpr bool TIGHT = DK == 96;
    static constexpr int VL = TIGHT ? 64 : DK + 96;
    static constexpr int O = TIGHT ? DK + 96 : DK + 128;
    static constexpr int alloc(bool pre) { return pre || O + 64 <= 256 ? 256 : 512; }
};

struct __align__(8) Bars {
    uint64_t full[2], empty[2];                      // K, scalars and V
    uint64_t fq, ft, fp, eq, et, ep;                 // Q, T, P
    uint64_t s, r, w, o;                             // workers -> issuer
    uint64_t staged[2];                              // workers -> copies: o is in the V slice
    uint64_t y, q, z, ds, out, drain;                // issuer -> workers
    uint32_t tmem;
};

// Shared memory of a CTA.
template <int DK, bool PRE>
struct Smem {
    using Rec = GdRec<DK, false>;
    static constexpr int KSC = (Rec::KSC + 1023) / 1024 * 1024;    // a stage of K and scalars
    static constexpr int T = 2 * KSC, Q = T + 16384, P = Q + DK * 128, V = PRE ? Q : P + 16384;
    static constexpr int bytes(int sw) { return V + 2 * kGdC * sw * 2 + 1024; }
};

// What a launch does: the sweep; or the pass that finds L of every segment but
// a sequence's last, and A (its last slice is the identity's), on the forward's
// records or on the backward's, where A of the last segment is wanted too.
enum { kSweep = 0, kSegments = 1, kSegmentsBwd = 2 };
template <int DK, int MODE>
__global__ void __launch_bounds__(kGdThreads, DK <= 96 || MODE != kSweep ? 2 : 1)
gd_sweep_fwd_kernel(GdParams p, const __grid_constant__ GdMap map_v, const __grid_constant__ GdMap map_o,
                    const __grid_constant__ CUtensorMap map_q, int sw, int nslices, WaitCtl ctl)
{
    using C = Cols<DK>;
    constexpr bool PRE = MODE != kSweep;
    using M = Smem<DK, PRE>;
    using Rec = GdRec<DK, MODE == kSegmentsBwd>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Bars B;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the slices of a segment side by side, so that they share its records in L2
    const int piece = blockIdx.x / nslices, slice = blockIdx.x - piece * nslices;
    const int pair = piece / p.nseg, seg = piece - pair * p.nseg, n = pair / p.seqs.H, h = pair - n * p.seqs.H;
    int64_t row0;
    int len;
    p.seqs.span(n, row0, len);
    if (len < 0) {
        if (tid == 0) record_status(p.status, GLA_ERR_INVALID_ARG);
        return;
    }
    int64_t slot0 = p.seqs.slot0(n, row0);
    const bool last = static_cast<int64_t>(seg + 1) * p.seg_chunks * kGdC >= len;      // the sequence ends here, or before
    if (p.nseg > 1) {
        const int64_t first = static_cast<int64_t>(seg) * p.seg_chunks;
        if ((seg > 0 && first * kGdC >= len) || (PRE && last && !(MODE == kSegmentsBwd && slice == nslices - 1))) return;
        len = min(len - static_cast<int>(first) * kGdC, p.seg_chunks * kGdC);
        row0 += first * kGdC;
        slot0 += first;
    }
    const bool unit = PRE && slice == nslices - 1;
    const int w0 = unit ? 0 : slice * sw, rows = unit ? DK : min(sw, p.dv - w0);       // this CTA's dv rows
    const int nc = (len + kGdC - 1) / kGdC;
    const unsigned char* rec = p.rec + (slot0 * p.seqs.H + h) * Rec::BYTES;
    const int64_t rec_step = static_cast<int64_t>(p.seqs.H) * Rec::BYTES;
    const int64_t nh = static_cast<int64_t>(n) * p.seqs.H + h;
    const int active = 2 * (rows >> 5);                             // worker warps with rows

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.full[i], 1);
            mbar_init(&B.empty[i], 1 + active);
            mbar_init(&B.staged[i], active);
        }
        uint64_t* tiles[6] = {&B.fq, &B.ft, &B.fp, &B.eq, &B.et, &B.ep};
        for (uint64_t* b : tiles) mbar_init(b, 1);
        uint64_t* from_workers[4] = {&B.s, &B.r, &B.w, &B.o};
        for (uint64_t* b : from_workers) mbar_init(b, active);
        uint64_t* from_issuer[6] = {&B.y, &B.q, &B.z, &B.ds, &B.out, &B.drain};
        for (uint64_t* b : from_issuer) mbar_init(b, 1);
        mbar_init_fence();
    }
    if (warp == kGdWorkers + 1) {
        tmem_alloc(&B.tmem, C::alloc(PRE));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = B.tmem;

    if (warp == kGdWorkers) {
        // ---- copies
        if (lane == 0) {
            const bool whole = rows == sw;               // the last slice may be narrower
            const CUtensorMap* mv = whole ? &map_v.all : &map_v.last;
            const CUtensorMap* mo = whole ? &map_o.all : &map_o.last;
            const uint32_t vbytes = kGdC * rows * 2;
            const int col = h * p.dv + w0, hk = h / (p.seqs.H / p.seqs.Hk);
            bool ok = true;
            // K, scalars and V of chunk c (rows behind the sequence's end are not used)
            auto first = [&](int c) {
                const int st = c & 1;
                mbar_arrive_expect_tx(&B.full[st], Rec::KSC + (unit ? 0u : vbytes));
                bulk_load(smem + st * M::KSC, rec + c * rec_step, Rec::KSC, &B.full[st]);
                if (unit) return;
                tma_load_2d(smem + M::V + st * kGdC * sw * 2, mv, &B.full[st], col,
                            static_cast<int>(row0) + c * kGdC);
            };
            auto tile = [&](int c, uint64_t* full, uint64_t* empty, int at, int from, uint32_t bytes) {
                if (c > 0 && !mbar_wait(empty, (c - 1) & 1, ctl)) return false;
                mbar_arrive_expect_tx(full, bytes);
                bulk_load(smem + at, rec + c * rec_step + from, bytes, full);
                return true;
            };
            int a = 0, q = 0, t = 0, pp = 0;             // copies issued of each kind
            if (nc > 0) first(a++);
            for (int c = 0; c < nc; ++c) {
                if (!PRE) {
                    ok = c == 0 || mbar_wait(&B.eq, (c - 1) & 1, ctl);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&B.fq, DK * 128);          // (what lies behind the sequence's end gives columns of o that do not leave)
#pragma unroll
                    for (int i = 0; i < DK / 32; ++i)
                        tma_load_2d(smem + M::Q + i * 4096, &map_q, &B.fq, hk * DK + 32 * i, static_cast<int>(row0) + c * kGdC);
                    ++q;
                }
                ok = tile(c, &B.ft, &B.et, M::T, Rec::T, 16384);
                if (!ok) break;
                ++t;
                if (!PRE) {
                    ok = tile(c, &B.fp, &B.ep, M::P, Rec::P, 16384);
                    if (!ok) break;
                    ++pp;
                }
                if (PRE) {
                    if (c > 0 && c + 1 < nc) ok = mbar_wait(&B.empty[(c - 1) & 1], ((c - 1) >> 1) & 1, ctl);
                    if (!ok) break;
                } else if (c > 0) {
                    // o of the chunk before: out of its slice, which then takes the next chunk's V
                    const int st = (c - 1) & 1;
                    ok = mbar_wait(&B.staged[st], ((c - 1) >> 1) & 1, ctl);
                    if (!ok) break;
                    tma_store_2d(mo, smem + M::V + st * kGdC * sw * 2, col, static_cast<int>(row0) + (c - 1) * kGdC);
                    tma_store_commit();
                    tma_store_wait_read();
                    if (c + 1 < nc) ok = mbar_wait(&B.empty[st], ((c - 1) >> 1) & 1, ctl);
                    if (!ok) break;
                }
                if (c + 1 < nc) first(a++);
            }
            if (!PRE && ok && nc > 0) {
                const int c = nc - 1, st = c & 1, valid = len - c * kGdC;
                const unsigned char* slice = smem + M::V + st * kGdC * sw * 2;
                if (mbar_wait(&B.staged[st], (c >> 1) & 1, ctl)) {
                    if (valid == kGdC) {
                        tma_store_2d(mo, slice, col, static_cast<int>(row0) + c * kGdC);
                    } else {                             // the rows behind are another sequence's
                        const int64_t ld_o = static_cast<int64_t>(p.seqs.H) * p.dv;
                        for (int i = 0; i < valid; ++i)
                            bulk_store(p.o + (row0 + static_cast<int64_t>(c) * kGdC + i) * ld_o + col, slice + i * rows * 2,
                                       rows * 2);
                    }
                }
                tma_store_commit();
            }
            // no copy may be in flight when the block ends
            tma_store_wait_read();
            for (int c = max(0, a - 2); c < a; ++c) mbar_wait(&B.full[c & 1], (c >> 1) & 1, ctl);
            if (q > 0) mbar_wait(&B.fq, (q - 1) & 1, ctl);
            if (t > 0) mbar_wait(&B.ft, (t - 1) & 1, ctl);
            if (pp > 0) mbar_wait(&B.fp, (pp - 1) & 1, ctl);
        }
    } else if (warp == kGdWorkers + 1) {
        // ---- products
        if (lane == 0) {
            const uint64_t q_k = smem_desc(smem_u32(smem + M::Q), 16, 512, kLayoutSW64);
            const uint64_t t_k = smem_desc(smem_u32(smem + M::T), 16, 1024, kLayoutSW128);
            const uint64_t p_k = smem_desc(smem_u32(smem + M::P), 16, 1024, kLayoutSW128);
            constexpr uint32_t idDk = idesc_bf16_f32(128, DK, 0, 1);
            for (int c = 0; c < nc; ++c) {
                const uint32_t st = smem_u32(smem + (c & 1) * M::KSC);
                const uint64_t k_k = smem_desc(st, 16, 512, kLayoutSW64);
                const uint64_t k_n = smem_desc(st, 4096, 512, kLayoutSW64);
                constexpr uint32_t id64 = idesc_bf16_f32(128, 64, 0, 0);
                if (!mbar_wait(&B.full[c & 1], (c >> 1) & 1, ctl)) break;
                if (!mbar_wait(&B.s, c & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t b = desc_add(k_k, (k >> 1) * 4096 + (k & 1) * 32);
                    umma_bf16_ts(tm + C::Y, tm + C::S + 16 * k, b, id64, k > 0);
                    umma_bf16_ts(tm + C::Y, tm + C::S + 16 * k + 8, b, id64, 1);
                }
                umma_commit(&B.y);
                if (!PRE) {
                    if (c > 0 && !mbar_wait(&B.o, (c - 1) & 1, ctl)) break;
                    if (!mbar_wait(&B.fq, c & 1, ctl)) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        const uint64_t b = desc_add(q_k, (k >> 1) * 4096 + (k & 1) * 32);
                        umma_bf16_ts(tm + C::O, tm + C::S + 16 * k, b, id64, k > 0);
                        umma_bf16_ts(tm + C::O, tm + C::S + 16 * k + 8, b, id64, 1);
                    }
                    umma_commit(&B.q);
                    umma_commit(&B.eq);
                }
                if (!mbar_wait(&B.ft, c & 1, ctl)) break;
                if (!mbar_wait(&B.r, c & 1, ctl)) break;
                tc_fence_after();
                // T and P are lower triangular: step s reaches tokens 16 s on
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t id = idesc_bf16_f32(128, 64 - 16 * s, 0, 0);
                    const uint64_t hi = desc_add(t_k, 2048 * s + 32 * s), lo = desc_add(hi, 8192);
                    const uint32_t d = tm + C::S + 16 * s, a = tm + C::Y + 16 * s;
                    umma_bf16_ts(d, a, hi, id, MODE == kSegmentsBwd || s > 0);
                    umma_bf16_ts(d, a + 8, hi, id, 1);
                    umma_bf16_ts(d, a, lo, id, 1);
                }
                umma_commit(&B.z);
                umma_commit(&B.et);
                if (!mbar_wait(&B.w, c & 1, ctl)) break;
                if (!PRE && C::TIGHT && !mbar_wait(&B.fp, c & 1, ctl)) break;
                tc_fence_after();
                auto add_low = [&]() {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_bf16_ts(tm + C::O + 16 * s, tm + C::VL + 8 * s, desc_add(p_k, 2048 * s + 32 * s),
                                     idesc_bf16_f32(128, 64 - 16 * s, 0, 0), 1);
                };
                if (!PRE && C::TIGHT) add_low();             // dS takes its place
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    umma_bf16_ts(tm + C::S, tm + C::Y + 16 * s, desc_add(k_n, 1024 * s), idDk, s > 0);
                    umma_bf16_ts(tm + C::S, tm + C::Y + 16 * s + 8, desc_add(k_n, 1024 * s), idDk, 1);
                }
                umma_commit(&B.ds);
                if (!PRE) {
                    if (!C::TIGHT) {
                        if (!mbar_wait(&B.fp, c & 1, ctl)) break;
                        add_low();
                    }
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint32_t id = idesc_bf16_f32(128, 64 - 16 * s, 0, 0);
                        const uint64_t hi = desc_add(p_k, 2048 * s + 32 * s);
                        umma_bf16_ts(tm + C::O + 16 * s, tm + C::V + 8 * s, hi, id, 1);
                        umma_bf16_ts(tm + C::O + 16 * s, tm + C::V + 8 * s, desc_add(hi, 8192), id, 1);
                    }
                    umma_commit(&B.out);
                    umma_commit(&B.ep);
                }
                umma_commit(&B.empty[c & 1]);
            }
            umma_commit(&B.drain);
            mbar_wait(&B.drain, 0, ctl);
        }
    } else if ((warp & 3) * 32 < rows) {
        // ---- workers: lane = dv row, half of the columns
        const int half = warp >> 2, r = w0 + (warp & 3) * 32 + lane;
        const uint32_t t0 = tm + (static_cast<uint32_t>(warp & 3) << 21);       // lane quarter
        constexpr int HS = DK / 2;                                              // state columns of a thread
        f2 S[HS / 2];
        const int64_t at = nh * p.nseg + seg;                                   // this segment's slot
        if (PRE) {
#pragma unroll
            for (int i = 0; i < HS / 2; ++i) {
                const int k = half * HS + 2 * i;
                S[i] = unit ? f2_make(k == r ? 1.f : 0.f, k + 1 == r ? 1.f : 0.f) : f2_splat(0.f);
            }
        } else {
            // (in segments the first one's too is a copy: s_final may be s0)
            const float* from = p.nseg > 1 ? p.seg_l + at * DK * p.dv : p.s0 ? p.s0 + nh * DK * p.dv : nullptr;
            load_state<HS>(S, from ? from + half * HS * p.dv + r : nullptr, p.dv);
        }
        auto put_state = [&]() {
#pragma unroll
            for (int k = 0; k < HS / 16; ++k) put_terms<2>(t0 + C::S + half * HS + 16 * k, cols_of<HS>(S, k));
        };
        if (nc > 0) {
            put_state();
            warp_done(&B.s, lane);
        }
        bool ok = true;
        for (int c = 0; c < nc; ++c) {
            const int ph = c & 1, s = 2 * half;              // this thread's steps of 16 tokens: s and s + 1
            const float* sc = reinterpret_cast<const float*>(smem + ph * M::KSC + Rec::SC) + 16 * s;
            __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(smem + M::V) + ph * kGdC * sw + 16 * s * rows +
                                (warp & 3) * 32 + lane;                       // this row's 32 tokens
            const int left = len - c * kGdC - 16 * s;                         // tokens of those in the sequence
            ok = warp_wait(&B.full[ph], (c >> 1) & 1, ctl) && warp_wait(&B.y, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            Cols16 x[2];
            get16x2(x[0], x[1], t0 + C::Y + 16 * s, t0 + C::Y + 16 * s + 16);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const Cols16 r = (unit ? zero16() : load_row16(vs + 16 * b * rows, rows, left - 16 * b)) -
                                 load16(sc + kScG * kGdC + 16 * b) * x[b];
                put_terms<2>(t0 + C::Y + 16 * (s + b), r);
                if (MODE == kSegmentsBwd) put16(t0 + C::S + 16 * (s + b), r);         // this record's T lacks its diagonal
            }
            warp_done(&B.r, lane);
            if (!PRE) {
                // Q is exact in bf16, so its factor scale G comes here, while Z is on its way
                ok = warp_wait(&B.q, ph, ctl);
                if (!ok) break;
                tc_fence_after();
                get16x2(x[0], x[1], t0 + C::O + 16 * s, t0 + C::O + 16 * s + 16);
#pragma unroll
                for (int b = 0; b < 2; ++b) put16(t0 + C::O + 16 * (s + b), load16(sc + kScPd * kGdC + 16 * b) * x[b]);
            }
            ok = warp_wait(&B.z, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            get16x2(x[0], x[1], t0 + C::S + 16 * s, t0 + C::S + 16 * s + 16);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                x[b] = x[b] * load16(sc + (MODE == kSegmentsBwd ? kScBeta : kScBt) * kGdC + 16 * b);
                if (!PRE) put_two(t0 + C::V + 8 * (s + b), t0 + C::VL + 8 * (s + b), x[b]);
                put_terms<2>(t0 + C::Y + 16 * (s + b), x[b] * load16(sc + kScR * kGdC + 16 * b));
            }
            warp_done(&B.w, lane);
            const float gl = sc[kScG * kGdC + kGdC - 1 - 16 * s];
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.empty[ph]);          // the scalars are read
            ok = warp_wait(&B.ds, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            add_cols<HS>(S, t0 + C::S + half * HS, gl);
            if (c + 1 < nc) {
                put_state();
                warp_done(&B.s, lane);
            }
            if (PRE) continue;
            ok = warp_wait(&B.out, ph, ctl);
            if (!ok) break;
            tc_fence_after();
            get16x2(x[0], x[1], t0 + C::O + 16 * s, t0 + C::O + 16 * s + 16);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.o);
#pragma unroll
            for (int b = 0; b < 2; ++b) store_row16(vs + 16 * b * rows, rows, x[b]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.staged[ph]);
        }
        if (PRE) {
            if (unit) store_state<HS>(S, p.seg_a + (at * DK + half * HS) * DK + r, DK);
            else store_state<HS>(S, p.seg_l + (at * DK + half * HS) * p.dv + r, p.dv);
        } else if (ok && last && p.s_final) {
            store_state<HS>(S, p.s_final + (nh * DK + half * HS) * p.dv + r, p.dv);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kGdWorkers + 1) tmem_dealloc(tm, C::alloc(PRE));
}

// Hands the states on: x' = A x + L through seg_l, whose slot of a segment
// turns from L into the state that enters it; ADJ: from the last segment to the
// first, x' = A^T x + D through seg_e, whose slot turns from D (what the segment
// itself gives its entering state's gradient) into the gradient of the state
// that leaves it.  A CTA has 16 columns of the state, all its rows in shared
// memory; a thread 4 columns of DK / 32 rows and a quarter of the sum.  A of
// the next segment is on its way meanwhile.  9 segments of 16 heads at dk = 128:
// 30 us (38 with A read from L2 as it is used, 83 with whole sums a thread).
template <int DK>
struct HandOn {
    static constexpr int R = DK / 32;                         // rows of a thread
    static constexpr int AS = DK + 4, XS = 20;                // row strides of A and x: 16-byte reads of 8 rows meet all banks
    static constexpr int A = DK * AS, X = DK * XS;            // floats
    static constexpr int bytes = (2 * A + X + 3 * R * 128 * 4) * 4;
};
template <int DK, bool ADJ>
__global__ void __launch_bounds__(512) gd_segments_kernel(GdParams p)
{
    using M = HandOn<DK>;
    constexpr int R = M::R, XS = M::XS, AS = M::AS, KQ = DK / 4;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    float* sa = reinterpret_cast<float*>(smem_raw);           // A of two segments
    float* x = sa + 2 * M::A;
    float4* part = reinterpret_cast<float4*>(x + M::X);       // [3][R][128]
    const int64_t nh = blockIdx.x;
    const int n = static_cast<int>(nh / p.seqs.H);
    int64_t row0;
    int len;
    p.seqs.span(n, row0, len);
    if (len < 0) return;
    const int t = threadIdx.x & 127, q = threadIdx.x >> 7;
    const int cx = (t & 3) * 4, c = blockIdx.y * 16 + cx, r0 = t >> 2;
    auto row = [&](int i) { return ADJ ? R * r0 + i : r0 + 32 * i; };        // neighbours along A's fast axis
    const int last = len > 0 ? (len - 1) / (p.seg_chunks * kGdC) : 0;
    const float* start = ADJ ? p.ds_final : p.s0;
    float* slots = ADJ ? p.seg_e : p.seg_l;
    auto segment = [&](int j) { return nh * p.nseg + (ADJ ? last - j : j); };
    auto fetch = [&](int j) {
        const float* a = p.seg_a + segment(j) * DK * DK;
        float* dst = sa + (j & 1) * M::A;
        for (int i = threadIdx.x; i < DK * DK / 4; i += 512) cp_async16(dst + i / (DK / 4) * AS + i % (DK / 4) * 4, a + 4 * i, true);
    };
    if (last > 0) fetch(0);
    cp_async_commit();
    if (q == 0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            *reinterpret_cast<float4*>(x + row(i) * XS + cx) =
                start ? *reinterpret_cast<const float4*>(start + (nh * DK + row(i)) * p.dv + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int j = 0; j < last; ++j) {
        if (j + 1 < last) fetch(j + 1);
        cp_async_commit();
        float* l = slots + segment(j) * DK * p.dv + c;
        float4 add[R], v[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            add[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q == 0) add[i] = *reinterpret_cast<const float4*>(l + static_cast<int64_t>(row(i)) * p.dv);
        }
        cp_async_wait<1>();
        __syncthreads();                                     // A is there, x is the state at this segment
        const float* a = sa + (j & 1) * M::A;
#pragma unroll
        for (int k = q * KQ; k < (q + 1) * KQ; k += 4) {
            float w[R][4];
#pragma unroll
            for (int e = 0; e < (ADJ ? 4 : R); ++e) {
                if (!ADJ) {
                    *reinterpret_cast<float4*>(w[e]) = *reinterpret_cast<const float4*>(a + row(e) * AS + k);
                } else if (R == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(a + (k + e) * AS + 4 * r0);
                    w[0][e] = y.x;
                    w[1][e] = y.y;
                    w[R - 2][e] = y.z;
                    w[R - 1][e] = y.w;
                } else {
#pragma unroll
                    for (int i = 0; i < R; ++i) w[i][e] = a[(k + e) * AS + row(i)];
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 y = *reinterpret_cast<const float4*>(x + (k + e) * XS + cx);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    v[i].x = fmaf(w[i][e], y.x, v[i].x);
                    v[i].y = fmaf(w[i][e], y.y, v[i].y);
                    v[i].z = fmaf(w[i][e], y.z, v[i].z);
                    v[i].w = fmaf(w[i][e], y.w, v[i].w);
                }
            }
        }
        if (q > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) part[((q - 1) * R + i) * 128 + t] = v[i];
        }
        __syncthreads();
        if (q == 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float4* at = reinterpret_cast<float4*>(x + row(i) * XS + cx);
                *reinterpret_cast<float4*>(l + static_cast<int64_t>(row(i)) * p.dv) = *at;
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const float4 u = part[(e * R + i) * 128 + t];
                    v[i].x += u.x;
                    v[i].y += u.y;
                    v[i].z += u.z;
                    v[i].w += u.w;
                }
                *at = make_float4(v[i].x + add[i].x, v[i].y + add[i].y, v[i].z + add[i].z, v[i].w + add[i].w);
            }
        }
    }
    if (q == 0) {
        const int g = ADJ ? 0 : last;
#pragma unroll
        for (int i = 0; i < R; ++i)
            *reinterpret_cast<float4*>(slots + ((nh * p.nseg + g) * DK + row(i)) * p.dv + c) =
                *reinterpret_cast<const float4*>(x + row(i) * XS + cx);
    }
}

template <int DK, bool ADJ>
gla_status hand_on(const GdParams& p, cudaStream_t st)
{
    constexpr int smem = HandOn<DK>::bytes;
    const cudaError_t e = cudaFuncSetAttribute(gd_segments_kernel<DK, ADJ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    trace_begin(st);
    gd_segments_kernel<DK, ADJ><<<dim3(static_cast<unsigned>(p.seqs.N) * p.seqs.H, p.dv / 16), 512, smem, st>>>(p);
    trace_end(st, "gd_segments_kernel");
    count_launch();
    return check_launch("gd_segments_kernel");
}

// The pass over segments and the hand-over of their states.
template <int DK, int MODE>
gla_status segments(const GdParams& p, const GdMap& v, const GdMap& o, const GdSlices& sl, const WaitCtl& ctl, cudaStream_t st)
{
    const int smem = Smem<DK, true>::bytes(sl.width);
    cudaError_t e = cudaFuncSetAttribute(gd_sweep_fwd_kernel<DK, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    trace_begin(st);
    gd_sweep_fwd_kernel<DK, MODE><<<static_cast<unsigned>(p.seqs.N) * p.seqs.H * p.nseg * (sl.n + 1), kGdThreads, smem, st>>>(
        p, v, o, CUtensorMap{}, sl.width, sl.n + 1, ctl);
    trace_end(st, "gd_sweep_segments_kernel");
    count_launch();
    const gla_status s = check_launch("gd_sweep_segments_kernel");
    return s != GLA_OK ? s : hand_on<DK, false>(p, st);
}

template <int DK>
gla_status launch(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    const GdSlices sl(p.dv);
    const int64_t width = static_cast<int64_t>(p.seqs.H) * p.dv;
    const int64_t tokens = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;
    GdMap v{}, o{};
    CUtensorMap q{};
    gla_status s = GLA_OK;
    if (tokens > 0 && ((s = gd_slice_map(&v, p.v, width, p.ld_v, tokens, sl.width, sl.last)) != GLA_OK ||
                       (s = gd_slice_map(&o, p.o, width, width, tokens, sl.width, sl.last)) != GLA_OK ||
                       (s = gd_block_map(&q, p.q, static_cast<int64_t>(p.seqs.Hk) * DK, p.ld_qk, tokens, 32, 64)) != GLA_OK))
        return s;
    const int smem = Smem<DK, false>::bytes(sl.width);
    const unsigned pairs = static_cast<unsigned>(p.seqs.N) * p.seqs.H;
    cudaError_t e = cudaFuncSetAttribute(gd_sweep_fwd_kernel<DK, kSweep>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    if (p.nseg > 1 && (s = segments<DK, kSegments>(p, v, o, sl, ctl, st)) != GLA_OK) return s;
    trace_begin(st);
    gd_sweep_fwd_kernel<DK, kSweep><<<pairs * p.nseg * sl.n, kGdThreads, smem, st>>>(p, v, o, q, sl.width, sl.n, ctl);
    trace_end(st, "gd_sweep_fwd_kernel");
    count_launch();
    return check_launch("gd_sweep_fwd_kernel");
}

// The same for the backward's sweeps, which have records of their own.
template <int DK>
gla_status states(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    const GdSlices sl(p.dv);
    const int64_t tokens = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;
    GdMap v{};
    const gla_status s = gd_slice_map(&v, p.v, static_cast<int64_t>(p.seqs.H) * p.dv, p.ld_v, tokens, sl.width, sl.last);
    return s != GLA_OK ? s : segments<DK, kSegmentsBwd>(p, v, v, sl, ctl, st);
}

}  // namespace

gla_status gd_launch_segment_states(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    switch (p.dk) {
    case 64: return states<64>(p, ctl, st);
    case 96: return states<96>(p, ctl, st);
    default: return states<128>(p, ctl, st);
    }
}

gla_status gd_launch_segment_grads(const GdParams& p, cudaStream_t st)
{
    switch (p.dk) {
    case 64: return hand_on<64, true>(p, st);
    case 96: return hand_on<96, true>(p, st);
    default: return hand_on<128, true>(p, st);
    }
}

gla_status gd_launch_sweep_fwd(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    switch (p.dk) {
    case 64: return launch<64>(p, ctl, st);
    case 96: return launch<96>(p, ctl, st);
    default: return launch<128>(p, ctl, st);
    }
}

}  // namespace gla
