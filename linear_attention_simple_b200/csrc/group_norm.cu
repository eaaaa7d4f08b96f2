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
// neighbouring lanes and loads its next row while it works on this one: 16,384
// rows of 16 x 192 bf16 with a gate 57 us, 5.3 TB/s (61 with four times the CTAs
// that are resident; 69 with a ring of rows in shared memory; 70 with more warps
// and spills).  In the backward a CTA stays with its groups: weight and bias sit
// in shared memory, the sums over rows in registers until they are added up
// within the CTA, and one partial row per CTA goes to the workspace; a second
// kernel adds those in a fixed order.
#include <cuda_bf16.h>

#include "gla_device.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kBwdThreads = 128;
constexpr int kSms = 148;
// CTAs of an SM, all resident; each walks over its rows.
constexpr int fwd_ctas(int nv) { return nv > 2 ? 2 : 3; }
constexpr int bwd_ctas(int nv) { return nv > 2 ? 3 : 4; }

struct NormParams {
    const void* x;
    const __nv_bfloat16 *gate, *dy;
    const float *weight, *bias;
    __nv_bfloat16* y;
    void* dx;
    __nv_bfloat16* dgate;
    float* part;                           // [CTAs of a block of groups][2][G d]
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
    __device__ __forceinline__ void get(f2 (&f)[4]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f2_from_bf16x2(w[i]);
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
    __device__ __forceinline__ void get(f2 (&f)[4]) const
    {
        f[0] = f2_make(a.x, a.y);
        f[1] = f2_make(a.z, a.w);
        f[2] = f2_make(b.x, b.y);
        f[3] = f2_make(b.z, b.w);
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f2 (&f)[4])
{
    *reinterpret_cast<uint4*>(p) =
        make_uint4(f2_to_bf16x2(f[0]), f2_to_bf16x2(f[1]), f2_to_bf16x2(f[2]), f2_to_bf16x2(f[3]));
}
__device__ __forceinline__ void store8(float* p, const f2 (&f)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = f2_get(f[2 * i]), b = f2_get(f[2 * i + 1]);
        reinterpret_cast<float4*>(p)[i] = make_float4(a.x, a.y, b.x, b.y);
    }
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Sigmoids of a pair, by the hardware's exponential and reciprocal: good to a
// few 2^-22, far below the bf16 rounding of y and the sums' own; e^-z past the
// largest fp32 gives 0.
__device__ __forceinline__ f2 sigmoid2(f2 z)
{
    const float2 t = f2_get(f2_mul(z, f2_splat(-1.4426950408889634f)));
    float a, b;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(t.y));
    const float2 u = f2_get(f2_add(f2_make(a, b), f2_splat(1.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(u.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(u.y));
    return f2_make(a, b);
}

// x^ in place of x (zeros behind d), and rstd of the group.
template <int NV>
__device__ __forceinline__ float normalise(f2 (&x)[NV][4], int lane, int lanes, const NormParams& p)
{
    const float inv = 1.f / static_cast<float>(p.d);
    if (p.center) {
        f2 sum = f2_splat(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = f2_add(sum, x[j][e]);
        const float2 t = f2_get(sum);
        const float mean = lanes_sum(t.x + t.y, lanes) * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const f2 m = f2_splat((j * lanes + lane) * 8 < p.d ? mean : 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] = f2_sub(x[j][e], m);
        }
    }
    f2 sq = f2_splat(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = f2_fma(x[j][e], x[j][e], sq);
    const float2 t = f2_get(sq);
    const float rstd = rsqrtf(lanes_sum(t.x + t.y, lanes) * inv + p.eps);
    const f2 rs = f2_splat(rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = f2_mul(x[j][e], rs);
    return rstd;
}

template <int NV, class T, bool GATE>
__global__ void __launch_bounds__(kThreads, fwd_ctas(NV)) group_norm_silu_kernel(NormParams p, int lanes)
{
    const int64_t seat = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / lanes;
    const int lane = threadIdx.x & (lanes - 1), g = static_cast<int>(seat % p.G);
    const int64_t walker = seat / p.G;
    const int c0 = lane * 8, cstep = lanes * 8;
    const int at = (p.shared_w ? 0 : g * p.d) + c0;
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
        f2 f[NV][4], z[NV][4];
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
            // weight and bias stay in L1: held in registers they cost half of the warps
            if (p.weight) {
                Raw<float> t;
                f2 w[4];
                t.load(p.weight + at + j * cstep);
                t.get(w);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[j][e] = f2_mul(f[j][e], w[e]);
            }
            if (p.bias) {
                Raw<float> t;
                f2 b[4];
                t.load(p.bias + at + j * cstep);
                t.get(b);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[j][e] = f2_add(f[j][e], b[e]);
            }
            if (GATE) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[j][e] = f2_mul(f[j][e], z[j][e]);
            }
            if (p.act) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[j][e] = f2_mul(f[j][e], sigmoid2(GATE ? z[j][e] : f[j][e]));
            }
            store8(p.y + (r * p.G + g) * p.d + c, f[j]);
        }
    }
}

template <int NV, class T, bool GATE>
__global__ void __launch_bounds__(kBwdThreads, bwd_ctas(NV)) group_norm_silu_bwd_kernel(NormParams p, int lanes)
{
    extern __shared__ __align__(16) float smem[];          // weight, bias [S][2][d]; later the warps' sums [4][S][2][d]
    // a warp has S neighbouring groups of one row, a CTA the same groups of its warps' rows
    const int S = 32 / lanes, blocks = (p.G + S - 1) / S, g0 = (blockIdx.x % blocks) * S;
    const int lane = threadIdx.x & (lanes - 1), seat = (threadIdx.x & 31) / lanes, g = g0 + seat;
    const int64_t walker = static_cast<int64_t>(blockIdx.x / blocks) * (kBwdThreads / 32) + (threadIdx.x >> 5);
    const int c0 = lane * 8, cstep = lanes * 8;
    for (int k = 0; k < S; ++k)
        for (int i = threadIdx.x; i < p.d; i += kBwdThreads) {
            const int at = (p.shared_w ? 0 : (g0 + k) * p.d) + i;
            const bool in = g0 + k < p.G;
            smem[k * 2 * p.d + i] = p.weight && in ? p.weight[at] : 1.f;
            smem[k * 2 * p.d + p.d + i] = p.bias && in ? p.bias[at] : 0.f;
        }
    __syncthreads();
    const float* params = smem + seat * 2 * p.d;
    f2 sw[NV][4], sb[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sw[j][e] = sb[j][e] = f2_splat(0.f);
    const T* px = static_cast<const T*>(p.x) + g * p.d + c0;
    const __nv_bfloat16* pg = p.gate + g * p.d + c0;
    const float inv = 1.f / static_cast<float>(p.d);
    Raw<T> rx[NV];
    Raw<__nv_bfloat16> rz[NV], rd[NV];
    auto fetch = [&](int64_t r) {
        const bool on = g < p.G && r < p.M;
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
    for (int64_t r0 = 0; r0 < p.M; r0 += p.walkers) {
        const int64_t r = r0 + walker;
        const bool on = g < p.G && r < p.M;
        const int64_t at = (r * p.G + g) * p.d;
        f2 f[NV][4], dn[NV][4];
        fetch(r);
        // the next row into L2, a line per lane (its registers are not to be had)
        if (g < p.G && r + p.walkers < p.M) {
            const int64_t rn = r + p.walkers;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if ((lane & 7) != 0 || c0 + j * cstep >= p.d) continue;
                prefetch_l2(px + rn * p.ld_x + j * cstep);
                prefetch_l2(p.dy + (rn * p.G + g) * p.d + c0 + j * cstep);
                if (GATE) prefetch_l2(pg + rn * p.ld_gate + j * cstep);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) rx[j].get(f[j]);
        const float rstd = normalise<NV>(f, lane, lanes, p);
        f2 s1 = f2_splat(0.f), s2 = s1;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * cstep;
            // a row that is not there adds nothing (its x^ is NaN at eps = 0)
            if (!on || c >= p.d) continue;
            f2 w[4], n[4], z[4], slope[4];
            Raw<float> t;
            t.a = *reinterpret_cast<const float4*>(params + c);
            t.b = *reinterpret_cast<const float4*>(params + c + 4);
            t.get(w);
            t.a = *reinterpret_cast<const float4*>(params + p.d + c);
            t.b = *reinterpret_cast<const float4*>(params + p.d + c + 4);
            t.get(n);
            rd[j].get(dn[j]);
            if (GATE) rz[j].get(z);
#pragma unroll
            for (int e = 0; e < 4; ++e) n[e] = f2_fma(f[j][e], w[e], n[e]);
            // val: act of the gate or of n; slope: its derivative
            f2 val[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                val[e] = GATE ? z[e] : n[e];
                slope[e] = f2_splat(1.f);
            }
            if (p.act) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f2 a = val[e], sg = sigmoid2(a);
                    val[e] = f2_mul(a, sg);
                    slope[e] = f2_fma(f2_sub(a, val[e]), sg, sg);    // sg (1 + a (1 - sg))
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 d = f2_mul(dn[j][e], GATE ? val[e] : slope[e]);
                if (GATE) z[e] = f2_mul(f2_mul(dn[j][e], n[e]), slope[e]);
                sw[j][e] = f2_fma(d, f[j][e], sw[j][e]);
                sb[j][e] = f2_add(sb[j][e], d);
                dn[j][e] = f2_mul(d, w[e]);
                s1 = f2_add(s1, dn[j][e]);
                s2 = f2_fma(dn[j][e], f[j][e], s2);
            }
            if (GATE) store8(p.dgate + at + c, z);
        }
        const float2 t1 = f2_get(s1), t2 = f2_get(s2);
        const float m1 = p.center ? lanes_sum(t1.x + t1.y, lanes) * inv : 0.f;
        const float m2 = lanes_sum(t2.x + t2.y, lanes) * inv;
        const f2 a1 = f2_splat(-rstd * m1), a2 = f2_splat(-rstd * m2), rs = f2_splat(rstd);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * cstep;
            if (!on || c >= p.d) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) f[j][e] = f2_fma(rs, dn[j][e], f2_fma(a2, f[j][e], a1));
            store8(static_cast<T*>(p.dx) + at + c, f[j]);
        }
    }
    if (!p.part) return;
    // the warps, in a fixed order
    __syncthreads();
    float* mine = smem + ((threadIdx.x >> 5) * S + seat) * 2 * p.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * cstep;
        if (c >= p.d) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            *reinterpret_cast<float2*>(mine + c + 2 * e) = f2_get(sw[j][e]);
            *reinterpret_cast<float2*>(mine + p.d + c + 2 * e) = f2_get(sb[j][e]);
        }
    }
    __syncthreads();
    float* part = p.part + static_cast<int64_t>(blockIdx.x / blocks) * 2 * p.G * p.d;
    for (int k = 0; k < S && g0 + k < p.G; ++k)
        for (int i = threadIdx.x; i < 2 * p.d; i += kBwdThreads) {
            float v = 0.f;
            for (int q = 0; q < kBwdThreads / 32; ++q) v += smem[(q * S + k) * 2 * p.d + i];
            part[(i < p.d ? 0 : p.G * p.d - p.d) + (g0 + k) * p.d + i] = v;
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

// The backward's CTAs of a block of neighbouring groups: all that fit the GPU
// at once over all blocks, no more than the rows need.
int ctas_of_block(int M, int G, int d, int* blocks)
{
    int lanes, nv;
    shape_for(d, &lanes, &nv);
    const int S = 32 / lanes, warps = kBwdThreads / 32;
    *blocks = (G + S - 1) / S;
    const int fit = bwd_ctas(nv) * kSms / *blocks, want = fit > 0 ? fit : 1, need = (M + warps - 1) / warps;
    return want < need ? want : (need > 0 ? need : 1);
}

template <class T, bool BWD, bool GATE, int NV>
gla_status start(const NormParams& p, int lanes, int blocks, cudaStream_t st)
{
    trace_begin(st);
    if (BWD) {
        const int smem = (kBwdThreads / 32) * (32 / lanes) * 2 * p.d * 4;      // 32 KB at most
        group_norm_silu_bwd_kernel<NV, T, GATE><<<blocks, kBwdThreads, smem, st>>>(p, lanes);
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
        int n;
        const int per = ctas_of_block(p.M, p.G, p.d, &n);
        p.walkers = per * (kBwdThreads / 32);
        blocks = static_cast<int64_t>(per) * n;
    } else {
        const int64_t w = static_cast<int64_t>(kSms) * fwd_ctas(nv) * kThreads / lanes / p.G;
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
    int blocks;
    return static_cast<size_t>(ctas_of_block(M, G, d, &blocks)) * 2 * G * d * 4;
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
    int blocks;
    const int C = shared_w ? d : G * d;
    if ((!dweight && !dbias) || C == 0) return GLA_OK;
    trace_begin(st);
    group_norm_reduce_kernel<<<(C + 31) / 32, 256, 0, st>>>(ws, dweight, dbias, M > 0 ? ctas_of_block(M, G, d, &blocks) : 0, G, d, shared_w);
    trace_end(st, "group_norm_reduce_kernel");
    count_launch();
    return check_launch("group_norm_reduce_kernel");
}

}  // namespace gla
