// gated_delta_chunks.cu -- what the sweeps of the gated delta rule need of a
// chunk's own tokens: decay factors, K (backward: and scale G Q), the triangular inverse
// T = (I + tril(K K^T . D beta_j, -1))^-1 and P = tril(scale Q K^T . D), as one
// record per (chunk, value head).  Every chunk at once, a CTA of 4 warps each.
//
// K K^T and Q K^T are exact products of bf16 values summed in fp32, a 16-row
// block of the 64 x 64 tiles per warp, tiles above the diagonal left out.  The
// inverse is taken in fp32 by halves: the four 16 x 16 diagonal blocks by
// forward substitution, a warp each and a column per lane; then the blocks
// below them, -T22 L21 T11, at 16 and at 32 rows.  (Substitution over all 64
// rows, a column per thread, left two of the four warps waiting: 125 us
// against 91 at 8 x 16 heads x 2,048 tokens, 80 with the blocks on tensor
// cores.)  The running sum of the log-decays is taken in 64 bits, so that the differences
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
// Eight values as two bf16 terms of 16 bytes.
__device__ __forceinline__ void put8(unsigned char* hi, unsigned char* lo, const float (&f)[8])
{
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        b[i] = pack_bf16(f[2 * i] - bf16_lo(a[i]), f[2 * i + 1] - bf16_hi(a[i]));
    }
    *reinterpret_cast<uint4*>(hi) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4*>(lo) = make_uint4(b[0], b[1], b[2], b[3]);
}

// Three bf16 terms of a pair.
__device__ __forceinline__ void terms3(uint32_t (&t)[3], float x, float y)
{
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        t[n] = pack_bf16(x, y);
        x -= bf16_lo(t[n]);
        y -= bf16_hi(t[n]);
    }
}
// d = f A B for a 16 x 16 block of a warp, A and B rows of fp32 tiles, NB deep:
// tensor core products of three bf16 terms each (all six of 2^-24 and above),
// so fp32 but for its last bits.  The same product by fp32 multiply-adds kept
// the shared-memory pipe busy: eight times the reads.
template <int NB>
__device__ __forceinline__ void block_mul(float* d, const float* a, const float* b, float f, int lane)
{
    const int g = lane >> 2, c = (lane & 3) * 2;
    float o[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
#pragma unroll
    for (int k = 0; k < NB; k += 16) {
        uint32_t fa[4][3], fb[2][2][3], at[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = *reinterpret_cast<const float2*>(a + (g + 8 * (i & 1)) * kLs + k + c + 8 * (i >> 1));
            terms3(fa[i], x.x, x.y);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float* y = b + (k + c + 8 * i) * kLs + 8 * t + g;
                terms3(fb[t][i], y[0], y[kLs]);
            }
#pragma unroll
        for (int n = 0; n < 3; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) at[n][i] = fa[i][n];
#pragma unroll
        for (int n = 2; n >= 0; --n)
#pragma unroll
            for (int m = 0; m <= n; ++m)
#pragma unroll
                for (int t = 0; t < 2; ++t) mma_bf16(o[t], at[m], fb[t][0][n - m], fb[t][1][n - m]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(d + (g + 8 * e) * kLs + 8 * t + c) = make_float2(f * o[t][2 * e], f * o[t][2 * e + 1]);
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
    constexpr int kSc = gd_scalars(false);             // (the backward's last two: five CTAs share an SM without them)
    __shared__ float sc[kSc][kGdC];

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
        float be[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            const int64_t at = (row + i) * p.seqs.H + h;
            float av = 0.f;
            be[e] = 0.f;
            if (i < valid) {
                av = p.a[at];
                av = av < -1e4f ? -1e4f : av;          // (a NaN stays one)
                be[e] = p.beta[at];
            }
            sc[kScBt][i] = BWD && fabsf(be[e]) < kGdBetaMin ? kGdBetaMin : be[e];
            x[e] = static_cast<double>(av) * 1.4426950408889634074;
        }
        if (BWD) {
            int64_t u = slot;                          // (the address is formed anew later: held so long it costs an SM its fifth CTA)
            asm volatile("" : "+l"(u));
            float2* more = reinterpret_cast<float2*>(p.rec + (u * p.seqs.H + h) * Rec::BYTES + Rec::SC) + lane;
            auto missing = [](float v) { return fabsf(v) < kGdBetaMin ? v * (1.f / kGdBetaMin) : 1.f; };
            more[kScBeta * kGdC / 2] = make_float2(be[0], be[1]);
            more[kScF * kGdC / 2] = make_float2(missing(be[0]), missing(be[1]));
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
            if (!BWD) sc[kScPd][i] = p.scale * sc[kScG][i];
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
    // K and, for the backward, scale G Q into the record
    for (int i = tid; i < kGdC * (DK / 8); i += kThreads) {
        const int r = i / (DK / 8), j = i - r * (DK / 8);
        const uint32_t at = (j >> 2) * 4096 + swz_off(r, j & 3, 64);
        *reinterpret_cast<uint4*>(rec + Rec::K + at) = *reinterpret_cast<const uint4*>(sk + r * KS + 8 * j);
        if (!BWD) continue;
        float f[8];
        mul8(f, *reinterpret_cast<const uint4*>(sq + r * KS + 8 * j), p.scale * sc[kScG][r]);
        put8(rec + Rec::Q + at, rec + Rec::QL + at, f);
    }
    const int g = lane >> 2, c2 = (lane & 3) * 2;
    uint32_t ph[8][2], pl[8][2];                       // P as it leaves, once L's tile is free to carry it
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
                const float2 be = *reinterpret_cast<const float2*>(&sc[kScBt][j0]);
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
            ph[t][hf] = pack_bf16(pv[0], pv[1]);
            pl[t][hf] = pack_bf16(pv[0] - bf16_lo(ph[t][hf]), pv[1] - bf16_hi(ph[t][hf]));
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
    // 16-row blocks (1,0) and (3,2), a warp each; L T11 on the way in the other corner
    if (w < 2) {
        const int o = 32 * w;
        float* corner = tt + o * kLs + o + 16;
        block_mul<16>(corner, sl + (o + 16) * kLs + o, tt + o * kLs + o, 1.f, lane);
        __syncwarp();
        block_mul<16>(tt + (o + 16) * kLs + o, tt + (o + 16) * kLs + o + 16, corner, -1.f, lane);
        __syncwarp();
        for (int i = lane; i < 64; i += 32)
            *reinterpret_cast<float4*>(corner + (i >> 2) * kLs + (i & 3) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    // the 32-row block, a 16 x 16 quarter a warp
    {
        const int r0 = (w >> 1) * 16, c0 = (w & 1) * 16;
        block_mul<32>(tt + r0 * kLs + 32 + c0, sl + (32 + r0) * kLs, tt + c0, 1.f, lane);
        __syncthreads();                               // L is read
        unsigned char* sp = reinterpret_cast<unsigned char*>(sl);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t at = swz_off(16 * w + g + 8 * hf, t, 128) + (lane & 3) * 4;
                *reinterpret_cast<uint32_t*>(sp + at) = ph[t][hf];
                *reinterpret_cast<uint32_t*>(sp + 8192 + at) = pl[t][hf];
            }
        block_mul<32>(tt + (32 + r0) * kLs + c0, tt + (32 + r0) * kLs + 32, tt + 32 + c0, -1.f, lane);
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
        put8(rec + Rec::T + at, rec + Rec::TL + at, f);
    }
    for (int i = tid; i < 1024; i += kThreads)
        reinterpret_cast<uint4*>(rec + Rec::P)[i] = reinterpret_cast<const uint4*>(sl)[i];
    for (int i = tid; i < kSc * kGdC / 4; i += kThreads)
        reinterpret_cast<float4*>(rec + Rec::SC)[i] = reinterpret_cast<const float4*>(&sc[0][0])[i];
}

template <int DK, bool BWD>
gla_status launch(const GdParams& p, cudaStream_t st)
{
    constexpr int smem = 2 * kGdC * (DK + kGdPad) * 2 + kGdC * kLs * 4;
    static_assert(2 * kGdC * (DK + kGdPad) * 2 >= kGdC * kLs * 4, "T takes the place of K and Q");
    static_assert(kGdC * kLs * 4 >= 16384, "P takes the place of L");
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
