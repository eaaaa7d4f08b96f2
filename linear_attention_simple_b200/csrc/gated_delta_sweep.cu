// gated_delta_sweep.cu -- the two sequential sweeps of the gated delta rule:
// forward over a sequence's chunks (outputs and final state; for the backward
// also what it reads of the forward), and in reverse (dv, the gradient of the
// state, the sums behind da and dbeta).
//
// A warp owns 16 rows of the transposed state [dv][dk] (fp32, in registers)
// and nothing it computes needs another warp, so a CTA is any number of such
// warps that share the chunk's operands: K, Q, T and P in shared memory,
// brought by cp.async into one of two stages while the warps work on the
// other (one block barrier a chunk).  With few (sequence, head) pairs the dv
// rows are spread over more CTAs.
//
// Precision: the states, V' and everything the fp32 outputs hang on enter
// their products as two bf16 terms (three where the rounding would be summed
// over a chunk's tokens into da), against operands that are exact in bf16 (K,
// Q, V, dO) or two terms themselves (T, P).  The bf16 output o takes one
// term of each.
#include "gated_delta.cuh"

namespace gla {
namespace {

// Largest number of warps in a CTA: all of an SM's registers at 168 (dk = 96,
// 64) or 255 (dk = 128) a thread.
template <int DK>
constexpr int max_warps() { return DK == 128 ? 8 : 12; }

// Shared-memory stage: element offsets of its parts.
struct Stage {
    int vs;             // row stride of the V (and dO) slice
    int k, q, v, d, t, pm, sc, size;
};
__host__ __device__ inline Stage stage_of(int DK, int sw, bool with_do, int pn)
{
    Stage s;
    const int KS = DK + kGdPad;
    s.vs = sw + kGdPad;
    s.k = 0;
    s.q = s.k + kGdC * KS;
    s.v = s.q + kGdC * KS;
    s.d = s.v + kGdC * s.vs;
    s.t = s.d + (with_do ? kGdC * s.vs : 0);
    s.pm = s.t + 2 * kGdC * kGdTP;
    s.sc = s.pm + pn * kGdC * kGdTP;
    s.size = s.sc + kGdSc * kGdC * 2;
    return s;
}

// A packed 64 x 64 bf16 tile into rows of kGdTP.
__device__ __forceinline__ void load_tile(__nv_bfloat16* dst, const __nv_bfloat16* src, int tid, int n)
{
    for (int i = tid; i < kGdC * 8; i += n) {
        const int r = i >> 3, c = (i & 7) * 8;
        cp_async16(dst + r * kGdTP + c, src + r * kGdC + c, true);
    }
}

struct Where {
    int64_t row0, slot0;
    int len, nc, h, hk, n, w0, sw;   // w0: first dv column of this CTA's slice, sw its width
};

template <int DK>
__device__ __forceinline__ void load_stage(__nv_bfloat16* st, const Stage& s, const GdParams& p, const Where& x, int c,
                                           bool with_do, int pn, int tid, int nth)
{
    constexpr int KS = DK + kGdPad;
    const int64_t row = x.row0 + static_cast<int64_t>(c) * kGdC;
    const int valid = min(kGdC, x.len - c * kGdC);
    const int64_t u = (x.slot0 + c) * p.seqs.H + x.h;
    gd_load_rows(st + s.k, KS, p.k + row * p.ld_qk + x.hk * DK, p.ld_qk, DK, valid, tid, nth);
    gd_load_rows(st + s.v, s.vs, p.v + row * p.ld_v + x.h * p.dv + x.w0, p.ld_v, x.sw, valid, tid, nth);
    for (int i = 0; i < 2; ++i) load_tile(st + s.t + i * kGdC * kGdTP, p.tm + (u * 2 + i) * kGdC * kGdC, tid, nth);
    gd_load_rows(st + s.q, KS, p.q + row * p.ld_qk + x.hk * DK, p.ld_qk, DK, valid, tid, nth);
    for (int i = 0; i < pn; ++i) load_tile(st + s.pm + i * kGdC * kGdTP, p.pm + (u * pn + i) * kGdC * kGdC, tid, nth);
    if (with_do)
        gd_load_rows(st + s.d, s.vs, p.dO + row * p.ld_do + x.h * p.dv + x.w0, p.ld_do, x.sw, valid, tid, nth);
    for (int i = tid; i < kGdSc * kGdC / 4; i += nth)
        cp_async16(reinterpret_cast<float*>(st + s.sc) + 4 * i, p.sc + u * kGdSc * kGdC + 4 * i, true);
}

__device__ __forceinline__ bool locate(Where& x, const GdParams& p, int sw)
{
    x.n = blockIdx.x / p.seqs.H;
    x.h = blockIdx.x - x.n * p.seqs.H;
    x.hk = x.h / (p.seqs.H / p.seqs.Hk);
    x.sw = sw;
    x.w0 = blockIdx.y * sw;
    p.seqs.span(x.n, x.row0, x.len);
    if (x.len < 0) {
        if (threadIdx.x == 0) record_status(p.status, GLA_ERR_INVALID_ARG);
        return false;
    }
    x.slot0 = p.seqs.slot0(x.n, x.row0);
    x.nc = (x.len + kGdC - 1) / kGdC;
    return true;
}

// State rows of a warp <-> global [dk][dv] fp32.  Thread (g, c): rows g and
// g + 8, columns 8 t + 2 c and the next.
template <int DK>
__device__ __forceinline__ void state_load(float (&S)[DK / 8][4], const float* s, int dv, int col0, int lane)
{
    const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < DK / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[t][e] = s ? s[static_cast<int64_t>(8 * t + c + (e & 1)) * dv + col0 + g + 8 * (e >> 1)] : 0.f;
}
template <int DK>
__device__ __forceinline__ void state_store(const float (&S)[DK / 8][4], float* s, int dv, int col0, int lane)
{
    const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < DK / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[static_cast<int64_t>(8 * t + c + (e & 1)) * dv + col0 + g + 8 * (e >> 1)] = S[t][e];
}
// The same rows rounded to bf16, [dv][dk].
template <int DK>
__device__ __forceinline__ void state_store_bf16(const float (&S)[DK / 8][4], __nv_bfloat16* s, int lane)
{
    const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < DK / 8; ++t) {
        *reinterpret_cast<uint32_t*>(s + g * DK + 8 * t + c) = pack_bf16(S[t][0], S[t][1]);
        *reinterpret_cast<uint32_t*>(s + (g + 8) * DK + 8 * t + c) = pack_bf16(S[t][2], S[t][3]);
    }
}

// Products are issued term by term over all tiles, so that a tile's next
// product comes after those of its neighbours and finds the last one done.

// acc[token tile] += state . X^T for X = K or Q in shared memory ([token][dk]).
template <int DK, int NT>
__device__ __forceinline__ void state_times(float (&acc)[8][4], const float (&S)[DK / 8][4], uint32_t xs)
{
    constexpr int KS = DK + kGdPad;
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        const Split<NT> a = split_tiles<NT>(S[2 * s], S[2 * s + 1]);
        uint32_t b[4][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) ldsm4(b[np], xs + np * 16 * KS * 2 + s * 32);
#pragma unroll
        for (int n = NT - 1; n >= 0; --n)
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                mma_bf16(acc[2 * np], a.t[n], b[np][0], b[np][1]);
                mma_bf16(acc[2 * np + 1], a.t[n], b[np][2], b[np][3]);
            }
    }
}

// S += A . X for the 16 tokens of step s, X [token][dk] in shared memory.
template <int DK, int NT>
__device__ __forceinline__ void state_add(float (&S)[DK / 8][4], const Split<NT>& a, uint32_t xk, int s)
{
    constexpr int KS = DK + kGdPad, NP = DK / 16, GR = NP % 3 == 0 ? 3 : 4;
#pragma unroll
    for (int g = 0; g < NP; g += GR) {
        uint32_t b[GR][4];
#pragma unroll
        for (int i = 0; i < GR; ++i) ldsm4_t(b[i], xk + s * 16 * KS * 2 + (g + i) * 32);
#pragma unroll
        for (int n = NT - 1; n >= 0; --n)
#pragma unroll
            for (int i = 0; i < GR; ++i) {
                mma_bf16(S[2 * (g + i)], a.t[n], b[i][0], b[i][1]);
                mma_bf16(S[2 * (g + i) + 1], a.t[n], b[i][2], b[i][3]);
            }
    }
}

// acc[tiles 2 np, 2 np + 1] += A . B for the pairs np = N0 .. N1 - 1, B a tile
// of two terms (hi, lo) in shared memory: A hi x B lo, then each term of A x B hi.
template <int N0, int N1, int NT, bool TRANS>
__device__ __forceinline__ void pairs_add(float (&acc)[8][4], const Split<NT>& a, uint32_t hi, uint32_t lo, int step,
                                          bool with_lo)
{
    uint32_t b[4][4];
    if (with_lo) {
#pragma unroll
        for (int np = N0; np < N1; ++np) {
            if (TRANS) ldsm4_t(b[np], lo + np * step);
            else ldsm4(b[np], lo + np * step);
        }
#pragma unroll
        for (int np = N0; np < N1; ++np) {
            mma_bf16(acc[2 * np], a.t[0], b[np][0], b[np][1]);
            mma_bf16(acc[2 * np + 1], a.t[0], b[np][2], b[np][3]);
        }
    }
#pragma unroll
    for (int np = N0; np < N1; ++np) {
        if (TRANS) ldsm4_t(b[np], hi + np * step);
        else ldsm4(b[np], hi + np * step);
    }
#pragma unroll
    for (int n = NT - 1; n >= 0; --n)
#pragma unroll
        for (int np = N0; np < N1; ++np) {
            mma_bf16(acc[2 * np], a.t[n], b[np][0], b[np][1]);
            mma_bf16(acc[2 * np + 1], a.t[n], b[np][2], b[np][3]);
        }
}
// The same for step s of a triangular tile: UP: pairs s .. 3, else 0 .. s.
template <bool UP, int NT, bool TRANS>
__device__ __forceinline__ void tri_add(float (&acc)[8][4], const Split<NT>& a, uint32_t hi, uint32_t lo, int step, int s,
                                        bool with_lo)
{
    switch (s) {          // s is a constant wherever this is called
    case 0: pairs_add<0, UP ? 4 : 1, NT, TRANS>(acc, a, hi, lo, step, with_lo); break;
    case 1: pairs_add<UP ? 1 : 0, UP ? 4 : 2, NT, TRANS>(acc, a, hi, lo, step, with_lo); break;
    case 2: pairs_add<UP ? 2 : 0, UP ? 4 : 3, NT, TRANS>(acc, a, hi, lo, step, with_lo); break;
    default: pairs_add<UP ? 3 : 0, 4, NT, TRANS>(acc, a, hi, lo, step, with_lo); break;
    }
}

// Sums over a warp's 16 rows of acc-shaped values v[8][2] (a thread's own two
// rows already added): returns, in lane (g, c), the totals of tokens
// 8 g + 2 c and the next.
__device__ __forceinline__ float2 sum_rows(float (&v)[8][2], int lane)
{
    const int g = lane >> 2;
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
        const bool up = (g & half) != 0;
#pragma unroll
        for (int t = 0; t < half; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float send = up ? v[t][e] : v[t + half][e];
                const float got = __shfl_xor_sync(0xFFFFFFFFu, send, 4 * half);
                v[t][e] = (up ? v[t + half][e] : v[t][e]) + got;
            }
    }
    return make_float2(v[0][0], v[0][1]);
}

// A warp's 16 columns of a shared [64][vs] slice to global rows, 32 bytes a row.
__device__ __forceinline__ void store_cols(__nv_bfloat16* dst, int64_t ld, const __nv_bfloat16* src, int vs, int valid,
                                           int lane)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 16 + (lane >> 1), c = (lane & 1) * 8;
        if (r < valid) *reinterpret_cast<uint4*>(dst + r * ld + c) = *reinterpret_cast<const uint4*>(src + r * vs + c);
    }
}

// Forward.  BWD: the backward's own pass over the forward; it keeps the
// states (fp32 and bf16), y and V', and sums o.dO instead of writing o.
template <int DK, bool BWD>
__global__ void __launch_bounds__(max_warps<DK>() * 32, 1) gd_sweep_old_kernel(GdParams p)
{
    constexpr int KS = DK + kGdPad;
    constexpr int PN = BWD ? 2 : 1;
    constexpr int NS = BWD ? 2 : 1;      // terms of S, and of P and V', in o
    constexpr int NW = BWD ? 3 : 2;      // terms of R V'
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __nv_bfloat16* smem = reinterpret_cast<__nv_bfloat16*>(smem_raw);
    const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31, w = tid >> 5;
    Where x;
    if (!locate(x, p, (nth >> 5) * 16)) return;
    const Stage L = stage_of(DK, x.sw, BWD, PN);
    const int col = x.w0 + 16 * w;       // this warp's dv columns
    const int wt = col >> 4, wtot = p.dv >> 4;
    const int64_t nh = static_cast<int64_t>(x.n) * p.seqs.H + x.h;
    const int c2 = (lane & 3) * 2;

    float S[DK / 8][4];
    state_load<DK>(S, p.s0 ? p.s0 + nh * DK * p.dv : nullptr, p.dv, col, lane);
    if (x.nc > 0) load_stage<DK>(smem, L, p, x, 0, BWD, PN, tid, nth);
    cp_async_commit();

    for (int c = 0; c < x.nc; ++c) {
        cp_async_wait<0>();
        __syncthreads();
        if (c + 1 < x.nc) load_stage<DK>(smem + ((c + 1) & 1) * L.size, L, p, x, c + 1, BWD, PN, tid, nth);
        cp_async_commit();

        __nv_bfloat16* st = smem + (c & 1) * L.size;
        const float* sc = reinterpret_cast<const float*>(st + L.sc);
        const uint32_t kn = smem_u32(st + L.k + rows_n(lane, KS)), qn = smem_u32(st + L.q + rows_n(lane, KS));
        const uint32_t kt = smem_u32(st + L.k + rows_k(lane, KS));
        const uint32_t tn = smem_u32(st + L.t + rows_n(lane, kGdTP)), pn = smem_u32(st + L.pm + rows_n(lane, kGdTP));
        const uint32_t va = smem_u32(st + L.v + 16 * w + rows_at(lane, L.vs));
        const int vstep = 16 * L.vs * 2;
        constexpr int tstep = 16 * kGdTP * 2, tile = kGdC * kGdTP * 2;
        const int64_t u = (x.slot0 + c) * p.seqs.H + x.h;
        const int valid = min(kGdC, x.len - c * kGdC);

        if (BWD) {
            state_store_bf16<DK>(S, p.sb + (u * p.dv + col) * DK, lane);
            if (c > 0) {
                float* sn = p.sn + (u * wtot + wt) * (DK * 16) + lane * 4;
#pragma unroll
                for (int t = 0; t < DK / 8; ++t)
                    *reinterpret_cast<float4*>(sn + t * 128) = make_float4(S[t][0], S[t][1], S[t][2], S[t][3]);
            }
        }

        // y = G K S - (T - I)(V - G K S)
        float y[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[t][e] = 0.f;
        state_times<DK, 2>(y, S, kn);
        Split<2> r[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t v[4];
            ldsm4_t(v, va + s * vstep);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int t = 2 * s + hf;
                const float2 G = *reinterpret_cast<const float2*>(sc + kScG * kGdC + 8 * t + c2);
                y[t][0] *= G.x;
                y[t][1] *= G.y;
                y[t][2] *= G.x;
                y[t][3] *= G.y;
                split_pair<2>(r[s], 2 * hf, bf16_lo(v[2 * hf]) - y[t][0], bf16_hi(v[2 * hf]) - y[t][1]);
                split_pair<2>(r[s], 2 * hf + 1, bf16_lo(v[2 * hf + 1]) - y[t][2], bf16_hi(v[2 * hf + 1]) - y[t][3]);
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) tri_add<true, 2, false>(y, r[s], tn + s * 32, tn + tile + s * 32, tstep, s, true);
        if (BWD) {
            float* yn = p.yn + (u * wtot + wt) * (kGdC * 16) + lane * 4;
#pragma unroll
            for (int t = 0; t < 8; ++t)
                *reinterpret_cast<float4*>(yn + t * 128) = make_float4(y[t][0], y[t][1], y[t][2], y[t][3]);
        }
        // V' = beta (V - y), over y
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t v[4];
            ldsm4_t(v, va + s * vstep);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int t = 2 * s + hf;
                const float2 be = *reinterpret_cast<const float2*>(sc + kScBeta * kGdC + 8 * t + c2);
                y[t][0] = be.x * (bf16_lo(v[2 * hf]) - y[t][0]);
                y[t][1] = be.y * (bf16_hi(v[2 * hf]) - y[t][1]);
                y[t][2] = be.x * (bf16_lo(v[2 * hf + 1]) - y[t][2]);
                y[t][3] = be.y * (bf16_hi(v[2 * hf + 1]) - y[t][3]);
            }
        }
        // o = scale G Q S + P V', P's diagonal apart
        float o[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
        state_times<DK, NS>(o, S, qn);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float2 G = *reinterpret_cast<const float2*>(sc + kScG * kGdC + 8 * t + c2);
            G.x *= p.scale;
            G.y *= p.scale;
            o[t][0] *= G.x;
            o[t][1] *= G.y;
            o[t][2] *= G.x;
            o[t][3] *= G.y;
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const Split<BWD ? 3 : 1> a = split_tiles<BWD ? 3 : 1>(y[2 * s], y[2 * s + 1]);
            tri_add<true, BWD ? 3 : 1, false>(o, a, pn + s * 32, pn + tile + s * 32, tstep, s, BWD);
        }
        if (BWD) {
            // sum over dv of (o without its own token's part) . dO
            const uint32_t da = smem_u32(st + L.d + 16 * w + rows_at(lane, L.vs));
            float od[8][2];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t d[4];
                ldsm4_t(d, da + s * vstep);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int t = 2 * s + hf;
                    od[t][0] = o[t][0] * bf16_lo(d[2 * hf]) + o[t][2] * bf16_lo(d[2 * hf + 1]);
                    od[t][1] = o[t][1] * bf16_hi(d[2 * hf]) + o[t][3] * bf16_hi(d[2 * hf + 1]);
                }
            }
            const float2 sum = sum_rows(od, lane);
            *reinterpret_cast<float2*>(p.part + (u * 3 * wtot + wt) * kGdC + 8 * (lane >> 2) + c2) = sum;
        } else {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 pd = *reinterpret_cast<const float2*>(sc + kScPd * kGdC + 8 * t + c2);
                o[t][0] = fmaf(pd.x, y[t][0], o[t][0]);
                o[t][1] = fmaf(pd.y, y[t][1], o[t][1]);
                o[t][2] = fmaf(pd.x, y[t][2], o[t][2]);
                o[t][3] = fmaf(pd.y, y[t][3], o[t][3]);
            }
        }
        // o (BWD: V') leaves by way of this warp's columns of the V slice
        __syncwarp();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const float(&a)[4] = BWD ? y[2 * s] : o[2 * s];
            const float(&b)[4] = BWD ? y[2 * s + 1] : o[2 * s + 1];
            stsm4_t(va + s * vstep, pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]),
                    pack_bf16(b[2], b[3]));
        }
        __syncwarp();
        if (BWD)
            store_cols(p.vp + u * kGdC * p.dv + col, p.dv, st + L.v + 16 * w, L.vs, kGdC, lane);
        else
            store_cols(p.o + (x.row0 + static_cast<int64_t>(c) * kGdC) * p.seqs.H * p.dv + x.h * p.dv + col,
                       static_cast<int64_t>(p.seqs.H) * p.dv, st + L.v + 16 * w, L.vs, valid, lane);

        // S = G_63 S + K^T (R V')
        const float gl = sc[kScG * kGdC + kGdC - 1];
#pragma unroll
        for (int t = 0; t < DK / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[t][e] *= gl;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int t = 2 * s; t < 2 * s + 2; ++t) {
                const float2 R = *reinterpret_cast<const float2*>(sc + kScR * kGdC + 8 * t + c2);
                y[t][0] *= R.x;
                y[t][1] *= R.y;
                y[t][2] *= R.x;
                y[t][3] *= R.y;
            }
            const Split<NW> a = split_tiles<NW>(y[2 * s], y[2 * s + 1]);
            state_add<DK, NW>(S, a, kt, s);
        }
    }
    if (!BWD && p.s_final) state_store<DK>(S, p.s_final + nh * DK * p.dv, p.dv, col, lane);
    if (BWD && p.ds_final) {
        float* sn = p.sn_last + (nh * wtot + wt) * (DK * 16) + lane * 4;
#pragma unroll
        for (int t = 0; t < DK / 8; ++t)
            *reinterpret_cast<float4*>(sn + t * 128) = make_float4(S[t][0], S[t][1], S[t][2], S[t][3]);
    }
}

// Reverse.  With E the gradient of the state that leaves the chunk:
//   dV' = R K E + P^T dO            (P's diagonal apart: dVs')
//   dv  = T^T (beta dV')
//   E   = G_63 E + Q^T (scale G dO) - K^T (G dv)
// and per token, for da and dbeta, the sums over dv of dv.y + dvs.z and of
// dv.z, where z = V - y and dvs is dv without the token's own path through P
// (that path's two halves cancel in da and are left out of both sums).
template <int DK>
__global__ void __launch_bounds__(max_warps<DK>() * 32, 1) gd_sweep_rev_kernel(GdParams p)
{
    constexpr int KS = DK + kGdPad;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __nv_bfloat16* smem = reinterpret_cast<__nv_bfloat16*>(smem_raw);
    const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31, w = tid >> 5;
    Where x;
    if (!locate(x, p, (nth >> 5) * 16)) return;
    const Stage L = stage_of(DK, x.sw, true, 2);
    const int col = x.w0 + 16 * w;
    const int wt = col >> 4, wtot = p.dv >> 4;
    const int64_t nh = static_cast<int64_t>(x.n) * p.seqs.H + x.h;
    const int c2 = (lane & 3) * 2;

    float E[DK / 8][4];
    state_load<DK>(E, p.ds_final ? p.ds_final + nh * DK * p.dv : nullptr, p.dv, col, lane);
    if (x.nc > 0) load_stage<DK>(smem + ((x.nc - 1) & 1) * L.size, L, p, x, x.nc - 1, true, 2, tid, nth);
    cp_async_commit();

    for (int c = x.nc - 1; c >= 0; --c) {
        const int64_t u = (x.slot0 + c) * p.seqs.H + x.h;
        // <E, state leaving>: the sum of da's terms over all later tokens
        float dot = 0.f;
        if (c + 1 < x.nc || p.ds_final) {
            const float* sn = (c + 1 < x.nc ? p.sn + ((u + p.seqs.H) * wtot + wt) * (DK * 16)
                                            : p.sn_last + (nh * wtot + wt) * (DK * 16)) + lane * 4;
#pragma unroll
            for (int t = 0; t < DK / 8; ++t) {
                const float4 s = __ldcs(reinterpret_cast<const float4*>(sn + t * 128));
                dot += E[t][0] * s.x + E[t][1] * s.y + E[t][2] * s.z + E[t][3] * s.w;
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        }
        if (lane == 0) p.anch[u * wtot + wt] = dot;
        state_store_bf16<DK>(E, p.eb + (u * p.dv + col) * DK, lane);

        cp_async_wait<0>();
        __syncthreads();
        if (c > 0) load_stage<DK>(smem + ((c - 1) & 1) * L.size, L, p, x, c - 1, true, 2, tid, nth);
        cp_async_commit();

        __nv_bfloat16* st = smem + (c & 1) * L.size;
        const float* sc = reinterpret_cast<const float*>(st + L.sc);
        const uint32_t kn = smem_u32(st + L.k + rows_n(lane, KS));
        const uint32_t kt = smem_u32(st + L.k + rows_k(lane, KS)), qt = smem_u32(st + L.q + rows_k(lane, KS));
        const uint32_t tt = smem_u32(st + L.t + rows_k(lane, kGdTP)), pt = smem_u32(st + L.pm + rows_k(lane, kGdTP));
        const uint32_t va = smem_u32(st + L.v + 16 * w + rows_at(lane, L.vs));
        const uint32_t da = smem_u32(st + L.d + 16 * w + rows_at(lane, L.vs));
        const int vstep = 16 * L.vs * 2;
        constexpr int tstep = 16 * kGdTP * 2, tile = kGdC * kGdTP * 2;
        const int valid = min(kGdC, x.len - c * kGdC);

        // dVs' = R K E + P^T dO
        float y[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[t][e] = 0.f;
        state_times<DK, 3>(y, E, kn);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float2 R = *reinterpret_cast<const float2*>(sc + kScR * kGdC + 8 * t + c2);
            y[t][0] *= R.x;
            y[t][1] *= R.y;
            y[t][2] *= R.x;
            y[t][3] *= R.y;
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            Split<1> d;
            ldsm4_t(d.t[0], da + s * vstep);
            tri_add<false, 1, true>(y, d, pt + s * tstep, pt + tile + s * tstep, 32, s, true);
        }
        // y: beta dVs'; r: -beta dV' (T is kept as -(T - I)); then dvs = y + (T - I)^T (beta dV')
        Split<2> r[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t d[4];
            ldsm4_t(d, da + s * vstep);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int t = 2 * s + hf;
                const float2 be = *reinterpret_cast<const float2*>(sc + kScBeta * kGdC + 8 * t + c2);
                float2 pd = *reinterpret_cast<const float2*>(sc + kScPd * kGdC + 8 * t + c2);
                pd.x *= be.x;
                pd.y *= be.y;
                y[t][0] *= be.x;
                y[t][1] *= be.y;
                y[t][2] *= be.x;
                y[t][3] *= be.y;
                split_pair<2>(r[s], 2 * hf, -fmaf(pd.x, bf16_lo(d[2 * hf]), y[t][0]),
                              -fmaf(pd.y, bf16_hi(d[2 * hf]), y[t][1]));
                split_pair<2>(r[s], 2 * hf + 1, -fmaf(pd.x, bf16_lo(d[2 * hf + 1]), y[t][2]),
                              -fmaf(pd.y, bf16_hi(d[2 * hf + 1]), y[t][3]));
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
            tri_add<false, 2, true>(y, r[s], tt + s * tstep, tt + tile + s * tstep, 32, s, true);
        // the sums; y becomes dv
        {
            const float* yn = p.yn + (u * wtot + wt) * (kGdC * 16) + lane * 4;
            float s1[8][2], s2[8][2];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t d[4], v[4];
                ldsm4_t(d, da + s * vstep);
                ldsm4_t(v, va + s * vstep);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int t = 2 * s + hf;
                    const float2 be = *reinterpret_cast<const float2*>(sc + kScBeta * kGdC + 8 * t + c2);
                    float2 pd = *reinterpret_cast<const float2*>(sc + kScPd * kGdC + 8 * t + c2);
                    pd.x *= be.x;
                    pd.y *= be.y;
                    const float4 yy = __ldcs(reinterpret_cast<const float4*>(yn + t * 128));
                    const float ys[4] = {yy.x, yy.y, yy.z, yy.w};
                    const float vs[4] = {bf16_lo(v[2 * hf]), bf16_hi(v[2 * hf]), bf16_lo(v[2 * hf + 1]),
                                         bf16_hi(v[2 * hf + 1])};
                    const float ds[4] = {bf16_lo(d[2 * hf]), bf16_hi(d[2 * hf]), bf16_lo(d[2 * hf + 1]),
                                         bf16_hi(d[2 * hf + 1])};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = vs[e] - ys[e];
                        const float full = fmaf(e & 1 ? pd.y : pd.x, ds[e], y[t][e]);
                        const float a = fmaf(full, ys[e], y[t][e] * z), b = full * z;
                        if (e < 2) {
                            s1[t][e] = a;
                            s2[t][e] = b;
                        } else {
                            s1[t][e - 2] += a;
                            s2[t][e - 2] += b;
                        }
                        y[t][e] = full;
                    }
                }
            }
            float* part = p.part + ((u * 3 + 1) * wtot + wt) * kGdC + 8 * (lane >> 2) + c2;
            *reinterpret_cast<float2*>(part) = sum_rows(s1, lane);
            *reinterpret_cast<float2*>(part + static_cast<int64_t>(wtot) * kGdC) = sum_rows(s2, lane);
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s < 4; ++s)
            stsm4_t(va + s * vstep, pack_bf16(y[2 * s][0], y[2 * s][1]), pack_bf16(y[2 * s][2], y[2 * s][3]),
                    pack_bf16(y[2 * s + 1][0], y[2 * s + 1][1]), pack_bf16(y[2 * s + 1][2], y[2 * s + 1][3]));
        __syncwarp();
        store_cols(p.dvv + (x.row0 + static_cast<int64_t>(c) * kGdC) * p.seqs.H * p.dv + x.h * p.dv + col,
                   static_cast<int64_t>(p.seqs.H) * p.dv, st + L.v + 16 * w, L.vs, valid, lane);

        // E = G_63 E + Q^T (scale G dO) - K^T (G dv)
        const float gl = sc[kScG * kGdC + kGdC - 1];
#pragma unroll
        for (int t = 0; t < DK / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) E[t][e] *= gl;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t d[4];
            ldsm4_t(d, da + s * vstep);
            Split<2> a, b;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int t = 2 * s + hf;
                const float2 G = *reinterpret_cast<const float2*>(sc + kScG * kGdC + 8 * t + c2);
                split_pair<2>(a, 2 * hf, p.scale * G.x * bf16_lo(d[2 * hf]), p.scale * G.y * bf16_hi(d[2 * hf]));
                split_pair<2>(a, 2 * hf + 1, p.scale * G.x * bf16_lo(d[2 * hf + 1]),
                              p.scale * G.y * bf16_hi(d[2 * hf + 1]));
                split_pair<2>(b, 2 * hf, -G.x * y[t][0], -G.y * y[t][1]);
                split_pair<2>(b, 2 * hf + 1, -G.x * y[t][2], -G.y * y[t][3]);
            }
            state_add<DK, 2>(E, a, qt, s);
            state_add<DK, 2>(E, b, kt, s);
        }
    }
    if (p.ds0) state_store<DK>(E, p.ds0 + nh * DK * p.dv, p.dv, col, lane);
}

// Warps of a CTA: as many as share the chunk's operands well, but with few
// (sequence, head) pairs fewer, so that about all SMs get a CTA.
int warps_for(int dk, int dv, int64_t pairs)
{
    const int wtot = dv / 16, most = dk == 128 ? 8 : 12;
    int best = 1;
    for (int nw = 1; nw <= most; ++nw) {
        if (wtot % nw) continue;
        if (nw > 1 && pairs * (wtot / nw) < 96) break;
        best = nw;
    }
    return best;
}

template <class K>
gla_status launch(K kernel, const char* name, const GdParams& p, bool with_do, int pn, cudaStream_t st)
{
    const int64_t pairs = static_cast<int64_t>(p.seqs.N) * p.seqs.H;
    const int nw = warps_for(p.dk, p.dv, pairs);
    const int smem = 2 * stage_of(p.dk, nw * 16, with_do, pn).size * 2;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    trace_begin(st);
    kernel<<<dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(p.dv / 16 / nw)), nw * 32, smem, st>>>(p);
    trace_end(st, name);
    count_launch();
    return check_launch(name);
}

}  // namespace

gla_status gd_launch_sweep_old(const GdParams& p, bool bwd, cudaStream_t st)
{
    if (bwd) {
        switch (p.dk) {
        case 64: return launch(gd_sweep_old_kernel<64, true>, "gd_sweep_fwd_bwd_kernel", p, true, 2, st);
        case 96: return launch(gd_sweep_old_kernel<96, true>, "gd_sweep_fwd_bwd_kernel", p, true, 2, st);
        default: return launch(gd_sweep_old_kernel<128, true>, "gd_sweep_fwd_bwd_kernel", p, true, 2, st);
        }
    }
    switch (p.dk) {
    case 64: return launch(gd_sweep_old_kernel<64, false>, "gd_sweep_old_kernel", p, false, 1, st);
    case 96: return launch(gd_sweep_old_kernel<96, false>, "gd_sweep_old_kernel", p, false, 1, st);
    default: return launch(gd_sweep_old_kernel<128, false>, "gd_sweep_old_kernel", p, false, 1, st);
    }
}

gla_status gd_launch_sweep_rev(const GdParams& p, cudaStream_t st)
{
    switch (p.dk) {
    case 64: return launch(gd_sweep_rev_kernel<64>, "gd_sweep_rev_kernel", p, true, 2, st);
    case 96: return launch(gd_sweep_rev_kernel<96>, "gd_sweep_rev_kernel", p, true, 2, st);
    default: return launch(gd_sweep_rev_kernel<128>, "gd_sweep_rev_kernel", p, true, 2, st);
    }
}

}  // namespace gla
