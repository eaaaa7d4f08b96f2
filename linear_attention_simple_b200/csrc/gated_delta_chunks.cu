// gated_delta_chunks.cu -- what the sweeps of the gated delta rule need of a
// chunk's own tokens: decay factors, K and scale G Q, the triangular inverse
// T = (I + tril(K K^T . D beta_j, -1))^-1 and P = tril(scale Q K^T . D), as one
// record per (chunk, value head).  Every chunk at once, a CTA of 4 warps each.
//
// K K^T and Q K^T are exact products of bf16 values summed in fp32, a 16-row
// block of the 64 x 64 tiles per warp, tiles above the diagonal left out.  The
// inverse is taken in fp32 by halves: the four 16 x 16 diagonal blocks by
// forward substitution, a warp each and a column per lane; then the blocks
// below them, -T22 L21 T11, at 16 and at 32 rows, all threads together.
// (Substitution over all 64 rows, a column per thread, left two of the four
// warps waiting: 125 us against 69 at 8 x 16 heads x 2,048 tokens.)  The
// running sum of the log-decays is taken in 64 bits, so that the differences
// behind a strong decay (a reset between documents) keep their precision; a
// is taken no lower than -10^4, where e^a is 0 in any case.
#include "gated_delta.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kLs = kGdC + 4;            // row stride of the fp32 tiles

__device__ __forceinline__ void mul8(float (&f)[8], const uint4& w, float s)
{
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = s * bf16_lo(a[i]);
        f[2 * i + 1] = s * bf16_hi(a[i]);
    }
}
// Eight values as one or two bf16 terms of 16 bytes.
template <bool TWO>
__device__ __forceinline__ void put8(unsigned char* hi, unsigned char* lo, const float (&f)[8])
{
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        if (TWO) b[i] = pack_bf16(f[2 * i] - bf16_lo(a[i]), f[2 * i + 1] - bf16_hi(a[i]));
    }
    *reinterpret_cast<uint4*>(hi) = make_uint4(a[0], a[1], a[2], a[3]);
    if (TWO) *reinterpret_cast<uint4*>(lo) = make_uint4(b[0], b[1], b[2], b[3]);
}

// out[R x 4 of a thread] = A B for square blocks of NB rows in fp32 tiles:
// thread `t` of NB * NB / (4 R) has rows r0 .. r0 + R - 1, columns c0 .. c0 + 3.
template <int NB, int R>
__device__ __forceinline__ void block_mul(float (&o)[R][4], const float* a, const float* b, int r0, int c0)
{
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
#pragma unroll 8
    for (int k = 0; k < NB; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(b + k * kLs + c0);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float x = a[(r0 + i) * kLs + k];
            o[i][0] = fmaf(x, y.x, o[i][0]);
            o[i][1] = fmaf(x, y.y, o[i][1]);
            o[i][2] = fmaf(x, y.z, o[i][2]);
            o[i][3] = fmaf(x, y.w, o[i][3]);
        }
    }
}
template <int R>
__device__ __forceinline__ void block_put(float* d, const float (&o)[R][4], int r0, int c0, float s)
{
#pragma unroll
    for (int i = 0; i < R; ++i)
        *reinterpret_cast<float4*>(d + (r0 + i) * kLs + c0) = make_float4(s * o[i][0], s * o[i][1], s * o[i][2], s * o[i][3]);
}

template <int DK, bool BWD>
__global__ void __launch_bounds__(kThreads) gd_chunks_kernel(GdParams p)
{
    using Rec = GdRec<DK, BWD>;
    constexpr int KS = DK + kGdPad;
    extern __shared__ __align__(16) unsigned char smem[];
    __nv_bfloat16* sk = reinterpret_cast<__nv_bfloat16*>(smem);
    __nv_bfloat16* sq = sk + kGdC * KS;
    float* sl = reinterpret_cast<float*>(sq + kGdC * KS);          // L
    float* tt = reinterpret_cast<float*>(smem);                    // T, over K and Q once both are read
    __shared__ float sc[kGdSc][kGdC];

    const int64_t slot = blockIdx.x;
    const int h = blockIdx.y;
    const int n = gd_seq_of_slot(p.seqs, slot);
    int64_t row0;
    int len;
    p.seqs.span(n, row0, len);
    if (len < 0) return;                               // the sweep reports it
    const int64_t c = slot - p.seqs.slot0(n, row0);
    if (c < 0 || c * kGdC >= len) return;              // a slot between two sequences
    const int valid = min(kGdC, len - static_cast<int>(c) * kGdC);
    const int64_t row = row0 + c * kGdC;
    const int hk = h / (p.seqs.H / p.seqs.Hk);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    unsigned char* rec = p.rec + (slot * p.seqs.H + h) * Rec::BYTES;

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
    // K and scale G Q into the record
    for (int i = tid; i < kGdC * (DK / 8); i += kThreads) {
        const int r = i / (DK / 8), j = i - r * (DK / 8);
        const uint32_t at = (j >> 2) * 4096 + swz_off(r, j & 3, 64);
        *reinterpret_cast<uint4*>(rec + Rec::K + at) = *reinterpret_cast<const uint4*>(sk + r * KS + 8 * j);
        float f[8];
        mul8(f, *reinterpret_cast<const uint4*>(sq + r * KS + 8 * j), p.scale * sc[kScG][r]);
        put8<BWD>(rec + Rec::Q + at, rec + Rec::QL + at, f);
    }
    const int g = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = 16 * w + g + 8 * hf, j0 = 8 * t + c2;
            float l[2] = {0.f, 0.f}, pv[2] = {0.f, 0.f};
            if ((t >> 1) <= w) {
                const float bh = sc[kScBh][i], bl = sc[kScBl][i];
                const float2 jh = *reinterpret_cast<const float2*>(&sc[kScBh][j0]);
                const float2 jl = *reinterpret_cast<const float2*>(&sc[kScBl][j0]);
                const float2 be = *reinterpret_cast<const float2*>(&sc[kScBeta][j0]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + e;
                    const float d = gd_exp2((bh - (e ? jh.y : jh.x)) + (bl - (e ? jl.y : jl.x)));
                    const float x = p.scale * d * qk[t][2 * hf + e];
                    if (j < i) l[e] = kk[t][2 * hf + e] * d * (e ? be.y : be.x);
                    if (j < i || (!BWD && j == i)) pv[e] = x;
                    if (BWD && j == i) sc[kScPd][i] = x;
                }
                *reinterpret_cast<float2*>(sl + i * kLs + j0) = make_float2(l[0], l[1]);
            }
            const uint32_t hi = pack_bf16(pv[0], pv[1]);
            const uint32_t at = swz_off(i, t, 128) + (lane & 3) * 4;
            *reinterpret_cast<uint32_t*>(rec + Rec::P + at) = hi;
            if (BWD)
                *reinterpret_cast<uint32_t*>(rec + Rec::PL + at) = pack_bf16(pv[0] - bf16_lo(hi), pv[1] - bf16_hi(hi));
        }
    }
    __syncthreads();

    // the diagonal blocks: lanes 0-15 a column each (the other half repeats them)
    {
        const float* l0 = sl + 16 * w * kLs + 16 * w;
        const int j = lane & 15;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 l = *reinterpret_cast<const float4*>(l0 + i * kLs + m);
                s0 = fmaf(l.x, t[m], s0);
                if (m + 1 < i) s1 = fmaf(l.y, t[m + 1], s1);
                if (m + 2 < i) s0 = fmaf(l.z, t[m + 2], s0);
                if (m + 3 < i) s1 = fmaf(l.w, t[m + 3], s1);
            }
            t[i] = i < j ? 0.f : (i == j ? 1.f : -(s0 + s1));
        }
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) tt[(16 * w + i) * kLs + 16 * w + j] = t[i];
        }
    }
    __syncthreads();
    // 16-row blocks (1,0) and (3,2), two warps each; L T11 in the other corner
    {
        const int blk = tid >> 6, t = tid & 63, r0 = t >> 2, c0 = (t & 3) * 4, o = 32 * blk;
        float x[1][4];
        block_mul<16, 1>(x, sl + (o + 16) * kLs + o, tt + o * kLs + o, r0, c0);
        block_put<1>(tt + o * kLs + o + 16, x, r0, c0, 1.f);
        __syncthreads();
        block_mul<16, 1>(x, tt + (o + 16) * kLs + o + 16, tt + o * kLs + o + 16, r0, c0);
        block_put<1>(tt + (o + 16) * kLs + o, x, r0, c0, -1.f);
        __syncthreads();
        *reinterpret_cast<float4*>(tt + (o + r0) * kLs + o + 16 + c0) = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
    }
    // the 32-row block
    {
        const int r0 = (tid >> 3) * 2, c0 = (tid & 7) * 4;
        float x[2][4];
        block_mul<32, 2>(x, sl + 32 * kLs, tt, r0, c0);
        block_put<2>(tt + 32, x, r0, c0, 1.f);
        __syncthreads();
        block_mul<32, 2>(x, tt + 32 * kLs + 32, tt + 32, r0, c0);
        block_put<2>(tt + 32 * kLs, x, r0, c0, -1.f);
    }
    __syncthreads();
    for (int i = tid; i < kGdC * 8; i += kThreads) {
        const int r = i >> 3, j0 = (i & 7) * 8;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) *reinterpret_cast<float4*>(f + e) = *reinterpret_cast<const float4*>(tt + r * kLs + j0 + e);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (j0 + e > r || (BWD && j0 + e == r)) f[e] = 0.f;
        const uint32_t at = swz_off(r, i & 7, 128);
        put8<true>(rec + Rec::T + at, rec + Rec::TL + at, f);
    }
    for (int i = tid; i < kGdSc * kGdC / 4; i += kThreads)
        reinterpret_cast<float4*>(rec + Rec::SC)[i] = reinterpret_cast<const float4*>(&sc[0][0])[i];
}

template <int DK, bool BWD>
gla_status launch(const GdParams& p, cudaStream_t st)
{
    constexpr int smem = 2 * kGdC * (DK + kGdPad) * 2 + kGdC * kLs * 4;
    static_assert(2 * kGdC * (DK + kGdPad) * 2 >= kGdC * kLs * 4, "T takes the place of K and Q");
    cudaError_t e = cudaFuncSetAttribute(gd_chunks_kernel<DK, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    trace_begin(st);
    gd_chunks_kernel<DK, BWD><<<dim3(static_cast<unsigned>(p.slots), static_cast<unsigned>(p.seqs.H)), kThreads, smem, st>>>(p);
    trace_end(st, "gd_chunks_kernel");
    count_launch();
    return check_launch("gd_chunks_kernel");
}

template <int DK>
gla_status pick(const GdParams& p, bool bwd, cudaStream_t st)
{
    return bwd ? launch<DK, true>(p, st) : launch<DK, false>(p, st);
}

}  // namespace

gla_status gd_launch_chunks(const GdParams& p, bool bwd, cudaStream_t st)
{
    if (p.slots == 0) return GLA_OK;
    switch (p.dk) {
    case 64: return pick<64>(p, bwd, st);
    case 96: return pick<96>(p, bwd, st);
    default: return pick<128>(p, bwd, st);
    }
}

}  // namespace gla
