// group_norm.cu -- group norm of each token's channels with an activation,
// channels last: the norm and gate behind a mixer's output, and its backward.
//
//   x^ = (x - mean) rstd          over the d channels of a group (mean 0 when
//                                 not centred: root mean square only)
//   n  = x^ weight + bias,   y = n silu(gate), or silu(n), or n
//
// Backward, with dn the gradient of n and g = dn weight:
//   dx = rstd (g - x^ <g x^> - <g>),  <.> the mean over the group (<g> only
//   when centred);  dweight = sum dn x^, dbias = sum dn over the rows.
//
// Pure streams: HBM bandwidth bounds them as long as enough loads are in
// flight.  A group is held by `lanes` lanes of a warp (a power of two) with NV
// vectors of 8 channels each, lanes x NV as close to d / 8 as it gets, so its
// sums are a few shuffles, every row is read once and no lane idles (d = 192:
// 8 lanes of 3 vectors).  The forward walks neighbouring groups of a row with
// neighbouring lanes and loads its next row while it works on this one.  In
// the backward a CTA stays with one group: weight and bias sit in shared
// memory, the sums over rows in registers until they are added up within the
// CTA, and one partial row per CTA goes to the workspace; a second kernel adds
// those in a fixed order.
#include <cuda_bf16.h>

#include "gla_device.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 148;

struct NormParams {
    const void* x;
    const __nv_bfloat16 *gate, *dy;
    const float *weight, *bias;
    __nv_bfloat16* y;
    void* dx;
    __nv_bfloat16* dgate;
    float* part;                           // [CTAs of a group][2][G d]
    int64_t ld_x, ld_gate;
    int M, G, d, shared_w, center, act, walkers;
    float eps;
};

// Eight channels as they lie in memory.
template <class T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8])
{
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// The fast exponential and quotient are good to a few 2^-22 here, far below
// the bf16 rounding of y and the fp32 sums; 1 + e^-z past 2^126 gives 0.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// x^ in place of x (zeros behind d), and rstd of the group.
template <int NV>
__device__ __forceinline__ float normalise(float (&x)[NV][8], int lane, int lanes, const NormParams& p)
{
    const float inv = 1.f / static_cast<float>(p.d);
    if (p.center) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += x[j][e];
        const float mean = lanes_sum(sum, lanes) * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float m = (j * lanes + lane) * 8 < p.d ? mean : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] -= m;
        }
    }
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(x[j][e], x[j][e], sq);
    const float rstd = rsqrtf(lanes_sum(sq, lanes) * inv + p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= rstd;
    return rstd;
}

template <int NV, class T, bool GATE>
__global__ void __launch_bounds__(kThreads) group_norm_silu_kernel(NormParams p, int lanes)
{
    const int64_t seat = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / lanes;
    const int lane = threadIdx.x & (lanes - 1), g = static_cast<int>(seat % p.G);
    const int64_t walker = seat / p.G;
    const int c0 = lane * 8, cstep = lanes * 8;
    float w[NV][8], b[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * cstep, at = (p.shared_w ? 0 : g * p.d) + c;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[j][e] = p.weight && c < p.d ? p.weight[at + e] : 1.f;
            b[j][e] = p.bias && c < p.d ? p.bias[at + e] : 0.f;
        }
    }
    const T* px = static_cast<const T*>(p.x) + g * p.d + c0;
    const __nv_bfloat16* pg = p.gate + g * p.d + c0;
    Raw<T> rx[NV];
    Raw<__nv_bfloat16> rz[NV];
    auto fetch = [&](int64_t r) {
        const bool on = walker < p.walkers && r < p.M;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            rx[j].zero();
            if (GATE) rz[j].zero();
            if (on && c0 + j * cstep < p.d) {
                rx[j].load(px + r * p.ld_x + j * cstep);
                if (GATE) rz[j].load(pg + r * p.ld_gate + j * cstep);
            }
        }
    };
    fetch(walker);
    // every lane of a warp makes the same number of steps: the sums are shuffles
    for (int64_t r0 = 0; r0 < p.M; r0 += p.walkers) {
        const int64_t r = r0 + walker;
        const bool on = walker < p.walkers && r < p.M;
        float f[NV][8], z[NV][8];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            rx[j].get(f[j]);
            if (GATE) rz[j].get(z[j]);
        }
        if (r0 + p.walkers < p.M) fetch(r + p.walkers);
        normalise<NV>(f, lane, lanes, p);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * cstep;
            if (!on || c >= p.d) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = fmaf(f[j][e], w[j][e], b[j][e]);
                const float a = GATE ? z[j][e] : n;
                const float s = p.act ? a * sigmoid_f(a) : a;
                f[j][e] = GATE ? n * s : s;
            }
            store8(p.y + (r * p.G + g) * p.d + c, f[j]);
        }
    }
}

template <int NV, class T, bool GATE>
__global__ void __launch_bounds__(kThreads, NV > 2 ? 1 : 2) group_norm_silu_bwd_kernel(NormParams p, int lanes)
{
    extern __shared__ __align__(16) float smem[];          // weight, bias [2][d]; later the warps' sums [8][2][d]
    const int lane = threadIdx.x & (lanes - 1), g = blockIdx.x % p.G;
    const int64_t walker = static_cast<int64_t>(blockIdx.x / p.G) * (kThreads / lanes) + threadIdx.x / lanes;
    const int c0 = lane * 8, cstep = lanes * 8;
    for (int i = threadIdx.x; i < p.d; i += kThreads) {
        const int at = (p.shared_w ? 0 : g * p.d) + i;
        smem[i] = p.weight ? p.weight[at] : 1.f;
        smem[p.d + i] = p.bias ? p.bias[at] : 0.f;
    }
    __syncthreads();
    float sw[NV][8], sb[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sw[j][e] = sb[j][e] = 0.f;
    const T* px = static_cast<const T*>(p.x) + g * p.d + c0;
    const __nv_bfloat16* pg = p.gate + g * p.d + c0;
    const float inv = 1.f / static_cast<float>(p.d);
    Raw<T> rx[NV];
    Raw<__nv_bfloat16> rz[NV], rd[NV];
    auto fetch = [&](int64_t r) {
        const bool on = r < p.M;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            rx[j].zero();
            rd[j].zero();
            if (GATE) rz[j].zero();
            if (on && c0 + j * cstep < p.d) {
                rx[j].load(px + r * p.ld_x + j * cstep);
                rd[j].load(p.dy + (r * p.G + g) * p.d + c0 + j * cstep);
                if (GATE) rz[j].load(pg + r * p.ld_gate + j * cstep);
            }
        }
    };
    fetch(walker);
    for (int64_t r0 = 0; r0 < p.M; r0 += p.walkers) {
        const int64_t r = r0 + walker;
        const bool on = r < p.M;
        const int64_t at = (r * p.G + g) * p.d;
        float f[NV][8], z[NV][8], dn[NV][8];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            rx[j].get(f[j]);
            rd[j].get(dn[j]);
            if (GATE) rz[j].get(z[j]);
        }
        if (r0 + p.walkers < p.M) fetch(r + p.walkers);
        const float rstd = normalise<NV>(f, lane, lanes, p);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * cstep;
            if (c >= p.d) continue;
            float w[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                *reinterpret_cast<float4*>(w + e) = *reinterpret_cast<const float4*>(smem + c + e);
                *reinterpret_cast<float4*>(b + e) = *reinterpret_cast<const float4*>(smem + p.d + c + e);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = fmaf(f[j][e], w[e], b[e]);
                const float a = GATE ? z[j][e] : n;
                float val = a, slope = 1.f;
                if (p.act) {
                    const float sg = sigmoid_f(a);
                    val = a * sg;
                    slope = sg * fmaf(a, 1.f - sg, 1.f);
                }
                const float dy = dn[j][e];
                dn[j][e] = dy * (GATE ? val : slope);
                z[j][e] = dy * n * slope;
                sw[j][e] = fmaf(dn[j][e], f[j][e], sw[j][e]);
                sb[j][e] += dn[j][e];
                dn[j][e] *= w[e];
                s1 += dn[j][e];
                s2 = fmaf(dn[j][e], f[j][e], s2);
            }
            if (GATE && on) store8(p.dgate + at + c, z[j]);
        }
        s1 = p.center ? lanes_sum(s1, lanes) * inv : 0.f;
        s2 = lanes_sum(s2, lanes) * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * cstep;
            if (!on || c >= p.d) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[j][e] = rstd * (dn[j][e] - fmaf(f[j][e], s2, s1));
            store8(static_cast<T*>(p.dx) + at + c, f[j]);
        }
    }
    if (!p.part) return;
    // the seats of a warp, then the warps, in a fixed order
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            for (int o = lanes; o < 32; o <<= 1) {
                sw[j][e] += __shfl_xor_sync(0xFFFFFFFFu, sw[j][e], o);
                sb[j][e] += __shfl_xor_sync(0xFFFFFFFFu, sb[j][e], o);
            }
    __syncthreads();
    float* mine = smem + (threadIdx.x >> 5) * 2 * p.d;
    if ((threadIdx.x & 31) < lanes) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * cstep;
            if (c >= p.d) continue;
            store8(mine + c, sw[j]);
            store8(mine + p.d + c, sb[j]);
        }
    }
    __syncthreads();
    float* part = p.part + static_cast<int64_t>(blockIdx.x / p.G) * 2 * p.G * p.d + g * p.d;
    for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
        float v = 0.f;
        for (int k = 0; k < kThreads / 32; ++k) v += smem[k * 2 * p.d + i];
        part[i < p.d ? i : p.G * p.d + i - p.d] = v;
    }
}

// dweight, dbias [C]: the partial rows, and with a shared weight the groups,
// added in a fixed order.  32 channels a CTA, 8 threads a channel.
__global__ void __launch_bounds__(256) group_norm_reduce_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                                float* __restrict__ db, int rows, int G, int d,
                                                                int shared_w)
{
    __shared__ float s[2][8][32];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int C = shared_w ? d : G * d, ch = blockIdx.x * 32 + c;
    const int groups = shared_w ? G : 1;
    float w = 0.f, b = 0.f;
    if (ch < C) {
        for (int i = k; i < rows * groups; i += 8) {
            const int r = i / groups, g = i - r * groups;
            const float* p = part + static_cast<int64_t>(r) * 2 * G * d + g * d + ch;
            w += p[0];
            b += p[static_cast<int64_t>(G) * d];
        }
    }
    s[0][k][c] = w;
    s[1][k][c] = b;
    __syncthreads();
    if (k == 0 && ch < C) {
        for (int r = 1; r < 8; ++r) {
            w += s[0][r][c];
            b += s[1][r][c];
        }
        if (dw) dw[ch] = w;
        if (db) db[ch] = b;
    }
}

// Lanes of a group and vectors of a lane: the least idle of 1 to 4 vectors,
// of equals two (loads in flight) before one (lanes).
void shape_for(int d, int* lanes, int* nv)
{
    const int v = d / 8;
    int best = 1 << 30;
    const int order[4] = {2, 1, 3, 4};
    for (int n : order) {
        int l = 1;
        while (l < 32 && l * n < v) l *= 2;
        if (l * n >= v && l * n < best) {
            best = l * n;
            *lanes = l;
            *nv = n;
        }
    }
}

// The backward's CTAs of a group: about four a SM over all groups, no more
// than the rows need.
int ctas_of_group(int M, int G, int d)
{
    int lanes, nv;
    shape_for(d, &lanes, &nv);
    const int seats = kThreads / lanes;
    const int want = (4 * kSms + G - 1) / G, need = (M + seats - 1) / seats;
    return want < need ? want : (need > 0 ? need : 1);
}

template <class T, bool BWD, bool GATE, int NV>
gla_status start(const NormParams& p, int lanes, int blocks, cudaStream_t st)
{
    trace_begin(st);
    if (BWD) {
        const int smem = (kThreads / 32) * 2 * p.d * 4;      // 64 KB at most
        cudaError_t e = cudaSuccess;
        if (smem > 48 * 1024)
            e = cudaFuncSetAttribute(group_norm_silu_bwd_kernel<NV, T, GATE>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return status_of(e);
        group_norm_silu_bwd_kernel<NV, T, GATE><<<blocks, kThreads, smem, st>>>(p, lanes);
    } else {
        group_norm_silu_kernel<NV, T, GATE><<<blocks, kThreads, 0, st>>>(p, lanes);
    }
    trace_end(st, BWD ? "group_norm_silu_bwd_kernel" : "group_norm_silu_kernel");
    count_launch();
    return check_launch("group_norm_silu_kernel");
}

template <class T, bool BWD, bool GATE>
gla_status run(const NormParams& q, cudaStream_t st)
{
    NormParams p = q;
    int lanes = 32, nv = 4;
    shape_for(p.d, &lanes, &nv);
    int64_t blocks;
    if (BWD) {
        const int per = ctas_of_group(p.M, p.G, p.d);
        p.walkers = per * (kThreads / lanes);
        blocks = static_cast<int64_t>(per) * p.G;
    } else {
        const int64_t w = static_cast<int64_t>(kSms) * 8 * kThreads / lanes / p.G;
        p.walkers = static_cast<int>(w < 1 ? 1 : (w < p.M ? w : p.M));
        blocks = (static_cast<int64_t>(p.walkers) * p.G * lanes + kThreads - 1) / kThreads;
    }
    switch (nv) {
    case 1: return start<T, BWD, GATE, 1>(p, lanes, static_cast<int>(blocks), st);
    case 2: return start<T, BWD, GATE, 2>(p, lanes, static_cast<int>(blocks), st);
    case 3: return start<T, BWD, GATE, 3>(p, lanes, static_cast<int>(blocks), st);
    default: return start<T, BWD, GATE, 4>(p, lanes, static_cast<int>(blocks), st);
    }
}

template <bool BWD>
gla_status run_any(const NormParams& p, bool f32, cudaStream_t st)
{
    if (f32) return p.gate ? run<float, BWD, true>(p, st) : run<float, BWD, false>(p, st);
    return p.gate ? run<__nv_bfloat16, BWD, true>(p, st) : run<__nv_bfloat16, BWD, false>(p, st);
}

}  // namespace

size_t group_norm_bwd_workspace_bytes(int M, int G, int d)
{
    return static_cast<size_t>(ctas_of_group(M, G, d)) * 2 * G * d * 4;
}

gla_status launch_group_norm(const void* x, bool f32, const void* gate, const float* weight, const float* bias, void* y,
                             int M, int G, int d, int64_t ld_x, int64_t ld_gate, bool shared_w, bool center, bool act,
                             float eps, cudaStream_t st)
{
    NormParams p{};
    p.x = x;
    p.gate = static_cast<const __nv_bfloat16*>(gate);
    p.weight = weight;
    p.bias = bias;
    p.y = static_cast<__nv_bfloat16*>(y);
    p.ld_x = ld_x;
    p.ld_gate = ld_gate;
    p.M = M;
    p.G = G;
    p.d = d;
    p.shared_w = shared_w;
    p.center = center;
    p.act = act;
    p.eps = eps;
    return run_any<false>(p, f32, st);
}

gla_status launch_group_norm_bwd(const void* x, bool f32, const void* gate, const float* weight, const float* bias,
                                 const void* dy, void* dx, void* dgate, float* dweight, float* dbias, float* ws, int M,
                                 int G, int d, int64_t ld_x, int64_t ld_gate, bool shared_w, bool center, bool act,
                                 float eps, cudaStream_t st)
{
    NormParams p{};
    p.x = x;
    p.gate = static_cast<const __nv_bfloat16*>(gate);
    p.dy = static_cast<const __nv_bfloat16*>(dy);
    p.weight = weight;
    p.bias = bias;
    p.dx = dx;
    p.dgate = static_cast<__nv_bfloat16*>(dgate);
    p.part = dweight || dbias ? ws : nullptr;
    p.ld_x = ld_x;
    p.ld_gate = ld_gate;
    p.M = M;
    p.G = G;
    p.d = d;
    p.shared_w = shared_w;
    p.center = center;
    p.act = act;
    p.eps = eps;
    if (M > 0) {
        const gla_status s = run_any<true>(p, f32, st);
        if (s != GLA_OK || !p.part) return s;
    }
    if (!dweight && !dbias) return GLA_OK;
    const int C = shared_w ? d : G * d;
    trace_begin(st);
    group_norm_reduce_kernel<<<(C + 31) / 32, 256, 0, st>>>(ws, dweight, dbias, M > 0 ? ctas_of_group(M, G, d) : 0, G, d, shared_w);
    trace_end(st, "group_norm_reduce_kernel");
    count_launch();
    return check_launch("group_norm_reduce_kernel");
}

}  // namespace gla
