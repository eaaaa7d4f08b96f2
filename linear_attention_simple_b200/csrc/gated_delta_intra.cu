// gated_delta_intra.cu -- what a chunk of the gated delta rule needs from its
// own tokens alone: the decay factors, T = (I + tril(K K^T . D beta, -1))^-1
// and P = tril(scale Q K^T . D).  One CTA of 4 warps per (chunk, value head);
// every chunk at once.
//
// K K^T and Q K^T are exact products of bf16 values summed in fp32 (one
// 16-row block of the 64 x 64 tiles per warp, tiles above the diagonal left
// out).  T is found by forward substitution in fp32, a column per thread with
// the column in registers: t_i = -sum_{m<i} L_im t_m.  The running sum of the
// log-decays is taken in 64 bits, so that the differences b_i - b_j behind a
// strong decay (a reset between documents) keep their precision; a is taken
// no lower than -10^4, below which e^a is 0 in any case.
#include "gated_delta.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kLs = kGdC + 4;            // row stride of the fp32 L tile

// Sequence of a chunk slot (the last n whose first slot is <= slot).
__device__ __forceinline__ int seq_of_slot(const GdSeqs& s, int64_t slot)
{
    if (!s.cu) return static_cast<int>(slot / ((s.T + kGdC - 1) / kGdC));
    int lo = 0, hi = s.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        int c = s.cu[mid];
        c = c < 0 ? 0 : c;
        if (c / kGdC + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A 64 x 64 shared tile (row stride kGdTP) to packed global rows.
__device__ __forceinline__ void store_tile(__nv_bfloat16* dst, const __nv_bfloat16* src, int tid, int n)
{
    for (int i = tid; i < kGdC * 8; i += n) {
        const int r = i >> 3, c = (i & 7) * 8;
        *reinterpret_cast<uint4*>(dst + r * kGdC + c) = *reinterpret_cast<const uint4*>(src + r * kGdTP + c);
    }
}

template <int DK, bool BWD>
__global__ void __launch_bounds__(kThreads) gd_intra_kernel(GdParams p)
{
    constexpr int KS = DK + kGdPad;
    constexpr int PN = BWD ? 2 : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    __nv_bfloat16* sk = reinterpret_cast<__nv_bfloat16*>(smem);
    __nv_bfloat16* sq = sk + kGdC * KS;
    __nv_bfloat16* sp = sq + kGdC * KS;                            // P: PN tiles
    float* sl = reinterpret_cast<float*>(sp + PN * kGdC * kGdTP);  // L
    __nv_bfloat16* stile = sk;                                     // -(T - I): 2 tiles, over K and Q once both are read
    __shared__ double sb[kGdC];
    __shared__ float sc[kGdSc][kGdC];

    const int64_t slot = blockIdx.x;
    const int h = blockIdx.y;
    const int n = seq_of_slot(p.seqs, slot);
    int64_t row0;
    int len;
    p.seqs.span(n, row0, len);
    if (len < 0) return;                               // the sweep reports it
    const int64_t c = slot - p.seqs.slot0(n, row0);
    if (c < 0 || c * kGdC >= len) return;              // a slot between two sequences
    const int valid = min(kGdC, len - static_cast<int>(c) * kGdC);
    const int64_t row = row0 + c * kGdC;
    const int64_t u = slot * p.seqs.H + h;
    const int hk = h / (p.seqs.H / p.seqs.Hk);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;

    gd_load_rows(sk, KS, p.k + row * p.ld_qk + hk * DK, p.ld_qk, DK, valid, tid, kThreads);
    gd_load_rows(sq, KS, p.q + row * p.ld_qk + hk * DK, p.ld_qk, DK, valid, tid, kThreads);
    cp_async_commit();
    if (w == 0) {
        double x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            const int64_t at = (row + i) * p.seqs.H + h;
            float av = 0.f, be = 0.f;
            if (i < valid) {
                av = fmaxf(p.a[at], -1e4f);
                be = p.beta[at];
            }
            // beta = 0 would leave dbeta = <dv, z> / beta undefined: a value too
            // small to matter takes its place.
            if (fabsf(be) < 1e-30f) be = 1e-30f;
            sc[kScBeta][i] = be;
            x[e] = static_cast<double>(av) * 1.4426950408889634074;
        }
        double s = x[0] + x[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += y;
        }
        sb[2 * lane] = s - x[1];
        sb[2 * lane + 1] = s;
        const double last = __shfl_sync(0xFFFFFFFFu, s, 31);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            const double b = e ? s : s - x[1];
            sc[kScG][i] = gd_exp2(static_cast<float>(b));
            sc[kScR][i] = gd_exp2(static_cast<float>(last - b));
            const float bh = static_cast<float>(b);
            sc[kScBh][i] = bh;
            sc[kScBl][i] = static_cast<float>(b - static_cast<double>(bh));
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // rows 16 w .. 16 w + 15 of K K^T and Q K^T, tiles up to the diagonal
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[t][e] = qk[t][e] = 0.f;
    const uint32_t ka = smem_u32(sk + 16 * w * KS + rows_a(lane, KS));
    const uint32_t qa = smem_u32(sq + 16 * w * KS + rows_a(lane, KS));
    const uint32_t kb = smem_u32(sk + rows_n(lane, KS));
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        uint32_t fk[4], fq[4];
        ldsm4(fk, ka + s * 32);
        ldsm4(fq, qa + s * 32);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > w) continue;
            uint32_t b[4];
            ldsm4(b, kb + np * 16 * KS * 2 + s * 32);
            mma_bf16(kk[2 * np], fk, b[0], b[1]);
            mma_bf16(kk[2 * np + 1], fk, b[2], b[3]);
            mma_bf16(qk[2 * np], fq, b[0], b[1]);
            mma_bf16(qk[2 * np + 1], fq, b[2], b[3]);
        }
    }
    const int g = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = 16 * w + g + 8 * hf;
            float l[2], pv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 8 * t + c2 + e;
                l[e] = pv[e] = 0.f;
                if (j <= i) {
                    const float d = gd_exp2(static_cast<float>(sb[i] - sb[j]));
                    const float x = p.scale * d * qk[t][2 * hf + e];
                    if (j < i) {
                        l[e] = kk[t][2 * hf + e] * d * sc[kScBeta][j];
                        pv[e] = x;
                    } else {
                        sc[kScPd][i] = x;
                    }
                }
            }
            *reinterpret_cast<float2*>(sl + i * kLs + 8 * t + c2) = make_float2(l[0], l[1]);
            const uint32_t hi = pack_bf16(pv[0], pv[1]);
            *reinterpret_cast<uint32_t*>(sp + i * kGdTP + 8 * t + c2) = hi;
            if (BWD)
                *reinterpret_cast<uint32_t*>(sp + kGdC * kGdTP + i * kGdTP + 8 * t + c2) =
                    pack_bf16(pv[0] - bf16_lo(hi), pv[1] - bf16_hi(hi));
        }
    }
    __syncthreads();

    if (tid < kGdC) {
        // column tid of T
        float t[kGdC];
#pragma unroll
        for (int i = 0; i < kGdC; ++i) {
            float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 l = *reinterpret_cast<const float4*>(sl + i * kLs + m);
                s0 = fmaf(l.x, t[m], s0);
                if (m + 1 < i) s1 = fmaf(l.y, t[m + 1], s1);
                if (m + 2 < i) s2 = fmaf(l.z, t[m + 2], s2);
                if (m + 3 < i) s3 = fmaf(l.w, t[m + 3], s3);
            }
            t[i] = i < tid ? 0.f : (i == tid ? 1.f : -((s0 + s1) + (s2 + s3)));
        }
#pragma unroll
        for (int i = 0; i < kGdC; ++i) {
            const float x = i > tid ? -t[i] : 0.f;
            const __nv_bfloat16 hi = __float2bfloat16_rn(x);
            stile[i * kGdTP + tid] = hi;
            stile[(kGdC + i) * kGdTP + tid] = __float2bfloat16_rn(x - __bfloat162float(hi));
        }
    } else {
        const int r = tid - kGdC;
        store_tile(p.pm + u * PN * kGdC * kGdC, sp, r, kThreads - kGdC);
        if (BWD) store_tile(p.pm + (u * PN + 1) * kGdC * kGdC, sp + kGdC * kGdTP, r, kThreads - kGdC);
        for (int i = r; i < kGdSc * kGdC; i += kThreads - kGdC) p.sc[u * kGdSc * kGdC + i] = (&sc[0][0])[i];
    }
    __syncthreads();
    store_tile(p.tm + u * 2 * kGdC * kGdC, stile, tid, kThreads);
    store_tile(p.tm + (u * 2 + 1) * kGdC * kGdC, stile + kGdC * kGdTP, tid, kThreads);
}

template <int DK, bool BWD>
gla_status launch(const GdParams& p, cudaStream_t st)
{
    constexpr int smem = 2 * kGdC * (DK + kGdPad) * 2 + (BWD ? 2 : 1) * kGdC * kGdTP * 2 + kGdC * kLs * 4;
    static_assert(2 * kGdC * (DK + kGdPad) >= 2 * kGdC * kGdTP, "the T tiles take the place of K and Q");
    cudaError_t e = cudaFuncSetAttribute(gd_intra_kernel<DK, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    trace_begin(st);
    gd_intra_kernel<DK, BWD><<<dim3(static_cast<unsigned>(p.slots), static_cast<unsigned>(p.seqs.H)), kThreads, smem, st>>>(p);
    trace_end(st, BWD ? "gd_intra_bwd_kernel" : "gd_intra_kernel");
    count_launch();
    return check_launch("gd_intra_kernel");
}

template <int DK>
gla_status pick(const GdParams& p, bool bwd, cudaStream_t st)
{
    return bwd ? launch<DK, true>(p, st) : launch<DK, false>(p, st);
}

}  // namespace

gla_status gd_launch_intra(const GdParams& p, bool bwd, cudaStream_t st)
{
    if (p.slots == 0) return GLA_OK;
    switch (p.dk) {
    case 64: return pick<64>(p, bwd, st);
    case 96: return pick<96>(p, bwd, st);
    default: return pick<128>(p, bwd, st);
    }
}

}  // namespace gla
