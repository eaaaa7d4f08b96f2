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
// Pure streams: a few flops per byte, HBM bandwidth bounds them.  A group is
// held by 1 to 32 lanes of a warp, 8 channels (16 bytes of bf16) a lane and
// step, so its sums are a few shuffles and every row is read once.  A lane
// keeps its channels for all rows it walks, so weight and bias are read once
// a thread, and the backward's sums over rows stay in registers until one
// partial row per walker goes to the workspace; a second kernel adds those in
// a fixed order.
#include <cuda_bf16.h>

#include "gla_device.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxWalkers = 296;           // partial rows of the backward

struct NormParams {
    const void* x;
    const __nv_bfloat16 *gate, *dy;
    const float *weight, *bias;
    __nv_bfloat16* y;
    void* dx;
    __nv_bfloat16* dgate;
    float* part;                           // [walkers][2][G d]
    int64_t ld_x, ld_gate;
    int M, G, d, shared_w, center, act, walkers;
    float eps;
};

__device__ __forceinline__ void load8(float (&f)[8], const __nv_bfloat16* p)
{
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(a[i]);
        f[2 * i + 1] = bf16_hi(a[i]);
    }
}
__device__ __forceinline__ void load8(float (&f)[8], const float* p)
{
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
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
__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

// The lanes of one group and the rows they walk.  NV: steps of 8 channels a lane.
struct Walk {
    int lane, g, walker, lanes;
    bool on;                               // whether this thread has a group
    __device__ __forceinline__ Walk(const NormParams& p, int lanes_)
    {
        lanes = lanes_;
        const int64_t seat = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / lanes;
        lane = threadIdx.x & (lanes - 1);
        g = static_cast<int>(seat % p.G);
        walker = static_cast<int>(seat / p.G);
        on = walker < p.walkers;
    }
};

// x^ of this lane's channels (zeros behind d) and rstd of the group.
template <int NV, class T>
__device__ __forceinline__ float normalise(float (&x)[NV][8], const T* px, bool on, const Walk& k, const NormParams& p)
{
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * k.lanes + k.lane) * 8;
        if (on && c < p.d) {
            load8(x[j], px + c);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += x[j][e];
    }
    const float inv = 1.f / static_cast<float>(p.d);
    const float mean = p.center ? lanes_sum(sum, k.lanes) * inv : 0.f;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const bool in = (j * k.lanes + k.lane) * 8 < p.d;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[j][e] = in ? x[j][e] - mean : 0.f;
            sq = fmaf(x[j][e], x[j][e], sq);
        }
    }
    const float rstd = rsqrtf(lanes_sum(sq, k.lanes) * inv + p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= rstd;
    return rstd;
}

template <int NV>
__device__ __forceinline__ void load_params(float (&w)[NV][8], float (&b)[NV][8], const Walk& k, const NormParams& p)
{
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * k.lanes + k.lane) * 8;
        const int at = (p.shared_w ? 0 : k.g * p.d) + c;
        const bool in = k.on && c < p.d;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[j][e] = 1.f;
            b[j][e] = 0.f;
        }
        if (in && p.weight) load8(w[j], p.weight + at);
        if (in && p.bias) load8(b[j], p.bias + at);
    }
}

template <int NV, class T>
__global__ void __launch_bounds__(kThreads) group_norm_silu_kernel(NormParams p, int lanes)
{
    const Walk k(p, lanes);
    float w[NV][8], b[NV][8];
    load_params<NV>(w, b, k, p);
    const T* x = static_cast<const T*>(p.x);
    // every lane of a warp makes the same number of steps: the sums are shuffles
    for (int64_t r0 = 0; r0 < p.M; r0 += p.walkers) {
        const int64_t r = r0 + k.walker;
        const bool on = k.on && r < p.M;
        float f[NV][8], z[NV][8];
        if (p.gate) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * lanes + k.lane) * 8;
                if (on && c < p.d) load8(z[j], p.gate + r * p.ld_gate + k.g * p.d + c);
            }
        }
        normalise<NV>(f, x + r * p.ld_x + k.g * p.d, on, k, p);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * lanes + k.lane) * 8;
            if (!on || c >= p.d) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = fmaf(f[j][e], w[j][e], b[j][e]);
                const float a = p.gate ? z[j][e] : n;
                const float s = p.act ? a * sigmoid_f(a) : a;
                f[j][e] = p.gate ? n * s : s;
            }
            store8(p.y + (r * p.G + k.g) * p.d + c, f[j]);
        }
    }
}

template <int NV, class T>
__global__ void __launch_bounds__(kThreads) group_norm_silu_bwd_kernel(NormParams p, int lanes)
{
    const Walk k(p, lanes);
    float w[NV][8], b[NV][8], sw[NV][8], sb[NV][8];
    load_params<NV>(w, b, k, p);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sw[j][e] = sb[j][e] = 0.f;
    const T* x = static_cast<const T*>(p.x);
    const float inv = 1.f / static_cast<float>(p.d);
    for (int64_t r0 = 0; r0 < p.M; r0 += p.walkers) {
        const int64_t r = r0 + k.walker;
        const bool on = k.on && r < p.M;
        const int64_t at = (r * p.G + k.g) * p.d;
        float f[NV][8], z[NV][8], dn[NV][8];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * lanes + k.lane) * 8;
            if (on && c < p.d) {
                load8(dn[j], p.dy + at + c);
                if (p.gate) load8(z[j], p.gate + r * p.ld_gate + k.g * p.d + c);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) dn[j][e] = z[j][e] = 0.f;
            }
        }
        const float rstd = normalise<NV>(f, x + r * p.ld_x + k.g * p.d, on, k, p);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * lanes + k.lane) * 8;
            const bool in = on && c < p.d;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = fmaf(f[j][e], w[j][e], b[j][e]);
                const float a = p.gate ? z[j][e] : n;
                float val = a, slope = 1.f;
                if (p.act) {
                    const float sg = sigmoid_f(a);
                    val = a * sg;
                    slope = sg * fmaf(a, 1.f - sg, 1.f);
                }
                const float dy = dn[j][e];
                dn[j][e] = dy * (p.gate ? val : slope);
                z[j][e] = dy * n * slope;
                sw[j][e] = fmaf(dn[j][e], f[j][e], sw[j][e]);
                sb[j][e] += dn[j][e];
                dn[j][e] *= w[j][e];
                s1 += dn[j][e];
                s2 = fmaf(dn[j][e], f[j][e], s2);
            }
            if (in && p.gate) store8(p.dgate + at + c, z[j]);
        }
        s1 = p.center ? lanes_sum(s1, lanes) * inv : 0.f;
        s2 = lanes_sum(s2, lanes) * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * lanes + k.lane) * 8;
            if (!on || c >= p.d) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[j][e] = rstd * (dn[j][e] - fmaf(f[j][e], s2, s1));
            store8(static_cast<T*>(p.dx) + at + c, f[j]);
        }
    }
    if (p.part && k.on) {
        float* part = p.part + static_cast<int64_t>(k.walker) * 2 * p.G * p.d + k.g * p.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * lanes + k.lane) * 8;
            if (c >= p.d) continue;
            store8(part + c, sw[j]);
            store8(part + p.G * p.d + c, sb[j]);
        }
    }
}

// dweight, dbias [C]: the partial rows, and with a shared weight the groups,
// added in a fixed order.  32 channels a CTA, 8 threads a channel.
__global__ void __launch_bounds__(256) group_norm_reduce_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                                float* __restrict__ db, int walkers, int G, int d,
                                                                int shared_w)
{
    __shared__ float s[2][8][32];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int C = shared_w ? d : G * d, ch = blockIdx.x * 32 + c;
    const int groups = shared_w ? G : 1;
    float w = 0.f, b = 0.f;
    if (ch < C) {
        for (int r = k; r < walkers; r += 8)
            for (int g = 0; g < groups; ++g) {
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

// Lanes of a group: as few as hold d channels at 8 a lane, at most a warp.
int lanes_for(int d)
{
    int l = 1;
    while (l < 32 && l * 8 < d) l *= 2;
    return l;
}

// Rows are dealt to `walkers` seats per group; at most four CTAs' worth a SM.
int walkers_for(int M, int G, int d, bool bwd)
{
    const int64_t seats = static_cast<int64_t>(148) * (bwd ? 4 : 8) * kThreads / lanes_for(d);
    int64_t w = seats / G;
    if (w < 1) w = 1;
    if (bwd && w > kMaxWalkers) w = kMaxWalkers;
    return static_cast<int>(w < M ? w : (M > 0 ? M : 1));
}

template <class T, bool BWD>
gla_status run(const NormParams& p, cudaStream_t st)
{
    const int lanes = lanes_for(p.d);
    const int64_t blocks = (static_cast<int64_t>(p.walkers) * p.G * lanes + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(blocks));
    const int nv = (p.d + lanes * 8 - 1) / (lanes * 8);
    trace_begin(st);
#define GLA_NORM(NV) \
    if (BWD) group_norm_silu_bwd_kernel<NV, T><<<grid, kThreads, 0, st>>>(p, lanes); \
    else group_norm_silu_kernel<NV, T><<<grid, kThreads, 0, st>>>(p, lanes)
    if (nv == 1) { GLA_NORM(1); }
    else if (nv == 2) { GLA_NORM(2); }
    else { GLA_NORM(4); }
#undef GLA_NORM
    trace_end(st, BWD ? "group_norm_silu_bwd_kernel" : "group_norm_silu_kernel");
    count_launch();
    return check_launch("group_norm_silu_kernel");
}

}  // namespace

size_t group_norm_bwd_workspace_bytes(int M, int G, int d)
{
    return static_cast<size_t>(walkers_for(M, G, d, true)) * 2 * G * d * 4;
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
    p.walkers = walkers_for(M, G, d, false);
    return f32 ? run<float, false>(p, st) : run<__nv_bfloat16, false>(p, st);
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
    p.walkers = walkers_for(M, G, d, true);
    if (M > 0) {
        const gla_status s = f32 ? run<float, true>(p, st) : run<__nv_bfloat16, true>(p, st);
        if (s != GLA_OK || !p.part) return s;
    }
    if (!dweight && !dbias) return GLA_OK;
    const int C = shared_w ? d : G * d;
    trace_begin(st);
    group_norm_reduce_kernel<<<(C + 31) / 32, 256, 0, st>>>(ws, dweight, dbias, M > 0 ? p.walkers : 0, G, d, shared_w);
    trace_end(st, "group_norm_reduce_kernel");
    count_launch();
    return check_launch("group_norm_reduce_kernel");
}

}  // namespace gla
