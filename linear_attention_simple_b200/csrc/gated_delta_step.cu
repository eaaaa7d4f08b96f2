// gated_delta_step.cu -- the gated delta rule token by token, in place on a
// pool of fp32 states: decoding (one token per sequence) and short runs of
// drafted tokens.  Per token, with S' = e^a S:
//
//   z = v - k S',  u = beta z,  S = S' + k^T u,  o = scale (q S' + (q.k) u)
//
// so k S', q S' and q.k come from one pass over the state and one reduction.
// The state is read once and written once whatever the number of tokens, and
// at one token that stream is all there is (0.9 flop a byte): HBM bandwidth
// bounds it.  One CTA per (sequence, head, slice of columns); a thread holds
// a float4 of columns in every RG-th row, all loads in flight before the
// first use.  Columns of S do not meet, so they may be spread over more CTAs.
// Everything is fp32.
#include <cuda_bf16.h>

#include "gated_delta.cuh"

namespace gla {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p)
{
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

struct StepParams {
    float* state;
    const int32_t* slot_idx;
    const void *q, *k, *v;
    const float *a, *beta;
    float* o;
    int n_slots, T, H, Hk, dv, sw;
    int64_t ld_qk, ld_v;
    float scale;
    int* status;
};

// Sixteen rows a thread: 64 registers of state, and room for the rest below
// kRegs, so that two CTAs share an SM at 192 columns.
template <int DK>
constexpr int row_groups() { return DK / 16; }
constexpr int kRegs = 96;
constexpr int kMaxQuads = 64;              // float4 column groups of a CTA (dv <= 256)

template <int DK, class Tin>
__global__ void __maxnreg__(kRegs) gd_step_kernel(StepParams p)
{
    constexpr int RG = row_groups<DK>(), R = DK / RG;
    __shared__ float2 s_kq[2][DK];
    __shared__ float4 s_k[RG][kMaxQuads], s_q[RG][kMaxQuads];
    __shared__ float s_d[RG];
    const int unit = blockIdx.x, n = unit / p.H, h = unit - n * p.H, hk = h / (p.H / p.Hk);
    const int quads = p.sw >> 2, t = threadIdx.x, nth = blockDim.x;
    const int rg = t / quads, c4 = t - rg * quads;
    const int col = blockIdx.y * p.sw + 4 * c4;

    const int64_t slot = p.slot_idx ? static_cast<int64_t>(p.slot_idx[n]) : static_cast<int64_t>(n);
    if (slot < 0 || slot >= p.n_slots) {           // a slot outside the pool: touch nothing
        if (t == 0) record_status(p.status, GLA_ERR_INVALID_ARG);
        return;
    }
    float* S = p.state + ((slot * p.H + h) * DK + rg) * p.dv + col;
    const int step = RG * p.dv;                    // elements between a thread's rows
    float4 s[R];
    {
        const float* at = S;
#pragma unroll
        for (int i = 0; i < R; ++i, at += step) s[i] = __ldcs(reinterpret_cast<const float4*>(at));
    }

    const Tin* q = static_cast<const Tin*>(p.q) + static_cast<int64_t>(n) * p.T * p.ld_qk + hk * DK;
    const Tin* k = static_cast<const Tin*>(p.k) + static_cast<int64_t>(n) * p.T * p.ld_qk + hk * DK;
    const Tin* v = static_cast<const Tin*>(p.v) + static_cast<int64_t>(n) * p.T * p.ld_v + static_cast<int64_t>(h) * p.dv + col;
    const int64_t ab = static_cast<int64_t>(n) * p.T * p.H + h;
    float* o = p.o + ab * p.dv + col;
    for (int i = t; i < DK; i += nth) s_kq[0][i] = make_float2(to_f(k[i]), to_f(q[i]));

    for (int tok = 0; tok < p.T; ++tok) {
        const float4 vv = load4(v + tok * p.ld_v);
        const float g = expf(p.a[ab + static_cast<int64_t>(tok) * p.H]), be = p.beta[ab + static_cast<int64_t>(tok) * p.H];
        __syncthreads();
        const float2* kq = s_kq[tok & 1];
        float4 ak = make_float4(0.f, 0.f, 0.f, 0.f), aq = ak;
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 x = kq[rg + RG * i];
            s[i].x *= g;
            s[i].y *= g;
            s[i].z *= g;
            s[i].w *= g;
            ak.x = fmaf(x.x, s[i].x, ak.x);
            ak.y = fmaf(x.x, s[i].y, ak.y);
            ak.z = fmaf(x.x, s[i].z, ak.z);
            ak.w = fmaf(x.x, s[i].w, ak.w);
            aq.x = fmaf(x.y, s[i].x, aq.x);
            aq.y = fmaf(x.y, s[i].y, aq.y);
            aq.z = fmaf(x.y, s[i].z, aq.z);
            aq.w = fmaf(x.y, s[i].w, aq.w);
            d = fmaf(x.x, x.y, d);
        }
        s_k[rg][c4] = ak;
        s_q[rg][c4] = aq;
        if (c4 == 0) s_d[rg] = d;
        if (tok + 1 < p.T)
            for (int i = t; i < DK; i += nth)
                s_kq[(tok + 1) & 1][i] = make_float2(to_f(k[(tok + 1) * p.ld_qk + i]), to_f(q[(tok + 1) * p.ld_qk + i]));
        __syncthreads();
        float4 zk = s_k[0][c4], zq = s_q[0][c4];
        d = s_d[0];
#pragma unroll
        for (int r = 1; r < RG; ++r) {
            const float4 a = s_k[r][c4], b = s_q[r][c4];
            zk.x += a.x; zk.y += a.y; zk.z += a.z; zk.w += a.w;
            zq.x += b.x; zq.y += b.y; zq.z += b.z; zq.w += b.w;
            d += s_d[r];
        }
        const float4 u = make_float4(be * (vv.x - zk.x), be * (vv.y - zk.y), be * (vv.z - zk.z), be * (vv.w - zk.w));
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float x = kq[rg + RG * i].x;
            s[i].x = fmaf(x, u.x, s[i].x);
            s[i].y = fmaf(x, u.y, s[i].y);
            s[i].z = fmaf(x, u.z, s[i].z);
            s[i].w = fmaf(x, u.w, s[i].w);
        }
        if (rg == 0)
            *reinterpret_cast<float4*>(o + static_cast<int64_t>(tok) * p.H * p.dv) =
                make_float4(p.scale * fmaf(d, u.x, zq.x), p.scale * fmaf(d, u.y, zq.y), p.scale * fmaf(d, u.z, zq.z),
                            p.scale * fmaf(d, u.w, zq.w));
    }
    asm volatile("" : "+l"(S));                    // the rows' addresses are formed anew, not kept in registers
#pragma unroll
    for (int i = 0; i < R; ++i, S += step) __stcs(reinterpret_cast<float4*>(S), s[i]);
}

template <int DK>
gla_status launch(const StepParams& p, int N, bool f32, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(N) * p.H, p.dv / p.sw);
    const int threads = row_groups<DK>() * (p.sw >> 2);
    trace_begin(st);
    if (f32) gd_step_kernel<DK, float><<<grid, threads, 0, st>>>(p);
    else gd_step_kernel<DK, __nv_bfloat16><<<grid, threads, 0, st>>>(p);
    trace_end(st, "gd_step_kernel");
    count_launch();
    return check_launch("gd_step_kernel");
}

// Columns of a CTA.  64 keep the most threads on an SM, and the tokens' barriers
// in few warps; 16 heads, whole rows against 64 columns: 300 sequences of 128 x
// 256 252 and 212 us, of 96 x 192 with four tokens 194 and 162, one sequence 9.7
// and 8.6.  But where whole rows leave as many threads on the SM (576 or more of
// the 682 that the registers allow; 96 x 192, 64 x 192, 64 x 128, 96 x 128) and
// there is one token, their longer runs in memory pay: 1,280 sequences of 96 x 192
// 483 against 505 us, of 64 x 192 327 and 344, 300 of them 86 and 88; the narrower
// two the same within 1%.  Widths that are no multiple of 64 take whole rows (300 sequences of
// 64 x 160 68 us, 109 with 32 columns), or 32 columns while there are too few
// CTAs (3 sequences of 96 x 96 10.0 and 9.2).
int slice_width(int64_t units, int T, int dk, int dv)
{
    const int threads = dk / 16 * (dv >> 2), fit = 65536 / kRegs / threads * threads;
    const bool many = units >= 296;
    if (dv % 64 == 0) return many && T == 1 && fit >= 576 ? dv : 64;
    return many ? dv : 32;
}

}  // namespace

gla_status gd_launch_step(float* state, const int32_t* slot_idx, int n_slots, const void* q, const void* k,
                          const void* v, const float* a, const float* beta, float* o, int N, int T, int Hk, int H,
                          int dk, int dv, int64_t ld_qk, int64_t ld_v, float scale, bool f32, int* status,
                          cudaStream_t st)
{
    const StepParams p{state, slot_idx, q, k, v, a, beta, o, n_slots, T, H, Hk, dv,
                       slice_width(static_cast<int64_t>(N) * H, T, dk, dv), ld_qk, ld_v, scale, status};
    switch (dk) {
    case 64: return launch<64>(p, N, f32, st);
    case 96: return launch<96>(p, N, f32, st);
    default: return launch<128>(p, N, f32, st);
    }
}

}  // namespace gla
