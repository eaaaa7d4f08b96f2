// gated_delta_tc.cuh -- shared by the gated delta rule's sweeps on tcgen05:
// copies, tensor-memory access in 16-column pieces, bf16 terms.
#pragma once

#include "gated_delta.cuh"

namespace gla {

constexpr int kGdWorkers = 8;                              // worker warps: lane quarter w % 4, half of the columns w / 4
constexpr int kGdThreads = (kGdWorkers + 2) * 32;          // + a copy warp and an issue warp

// Tensor maps of token slices; the last slice of dv may be narrower than the others.
struct GdMap {
    CUtensorMap all, last;
};

// Slices of dv rows: as few as 128 lanes allow, of equal width but for the
// last (a CTA's time does not depend on how many of its lanes hold rows).
struct GdSlices {
    int n, width, last;
    explicit GdSlices(int dv)
    {
        n = (dv + 127) / 128;
        width = (dv / 32 + n - 1) / n * 32;
        last = dv - (n - 1) * width;
    }
};

// [token][width of all heads] bf16 rows, ld apart; a box is a chunk's tokens of one slice.
inline gla_status gd_slice_map(GdMap* m, const void* base, int64_t width, int64_t ld, int64_t tokens, int box, int last)
{
    const uint64_t dims[2] = {static_cast<uint64_t>(width), static_cast<uint64_t>(tokens)};
    const uint64_t strides[2] = {2, static_cast<uint64_t>(ld) * 2};
    const uint32_t boxes[2] = {static_cast<uint32_t>(box), kGdC}, tail[2] = {static_cast<uint32_t>(last), kGdC};
    const gla_status s = make_tmap(&m->all, base, 2, dims, strides, boxes, 2, 0);
    return s != GLA_OK ? s : make_tmap(&m->last, base, 2, dims, strides, tail, 2, 0);
}

// The same rows in boxes of `box` columns, swizzled.
inline gla_status gd_block_map(CUtensorMap* m, const void* base, int64_t width, int64_t ld, int64_t tokens, int box, int swizzle)
{
    const uint64_t dims[2] = {static_cast<uint64_t>(width), static_cast<uint64_t>(tokens)};
    const uint64_t strides[2] = {2, static_cast<uint64_t>(ld) * 2};
    const uint32_t boxes[2] = {static_cast<uint32_t>(box), kGdC};
    return make_tmap(m, base, 2, dims, strides, boxes, 2, swizzle);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
                     "r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// Sixteen fp32 columns of a thread as pairs: the arithmetic between tensor
// memory accesses is what the sweeps' schedulers are busy with, and a packed
// instruction does two of them.
struct Cols16 {
    f2 p[8];
};
__device__ __forceinline__ Cols16 operator*(const Cols16& a, const Cols16& b)
{
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[i] = f2_mul(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ Cols16 operator+(const Cols16& a, const Cols16& b)
{
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[i] = f2_add(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ Cols16 operator-(const Cols16& a, const Cols16& b)
{
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[i] = f2_sub(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ Cols16 fma16(const Cols16& a, const Cols16& b, const Cols16& c)
{
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[i] = f2_fma(a.p[i], b.p[i], c.p[i]);
    return r;
}
// What one bf16 term leaves of a value.
__device__ __forceinline__ Cols16 low16(const Cols16& a)
{
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[i] = f2_sub(a.p[i], f2_from_bf16x2(f2_to_bf16x2(a.p[i])));
    return r;
}
__device__ __forceinline__ Cols16 zero16()
{
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[i] = f2_splat(0.f);
    return r;
}
// From shared memory (16-byte aligned), the same for all lanes.
__device__ __forceinline__ Cols16 load16(const float* p)
{
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 w = reinterpret_cast<const ulonglong2*>(p)[i];
        r.p[2 * i].v = w.x;
        r.p[2 * i + 1].v = w.y;
    }
    return r;
}
// This row's 16 tokens of a [token][row] bf16 slice; zeros from `left` on (what
// lies there is not the sequence's; the loads do not wait for the comparison).
__device__ __forceinline__ Cols16 load_row16(const __nv_bfloat16* s, int stride, int left)
{
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = __bfloat162float(s[i * stride]);
    if (left < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = i < left ? f[i] : 0.f;
    }
    Cols16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[i] = f2_make(f[2 * i], f[2 * i + 1]);
    return r;
}
__device__ __forceinline__ void store_row16(__nv_bfloat16* s, int stride, const Cols16& x)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = f2_to_bf16x2(x.p[i]);
        s[2 * i * stride] = __ushort_as_bfloat16(static_cast<unsigned short>(w));
        s[(2 * i + 1) * stride] = __ushort_as_bfloat16(static_cast<unsigned short>(w >> 16));
    }
}
__device__ __forceinline__ Cols16 cols16(const uint32_t (&r)[16])
{
    Cols16 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.p[i] = f2_make(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    return x;
}
// Tensor memory, one and two pieces of 16 columns behind one wait.
__device__ __forceinline__ Cols16 get16(uint32_t taddr)
{
    uint32_t r[16];
    tmem_ld16(taddr, r);
    tmem_ld_wait();
    return cols16(r);
}
__device__ __forceinline__ void get16x2(Cols16& x, Cols16& y, uint32_t tx, uint32_t ty)
{
    uint32_t a[16], b[16];
    tmem_ld16(tx, a);
    tmem_ld16(ty, b);
    tmem_ld_wait();
    x = cols16(a);
    y = cols16(b);
}
__device__ __forceinline__ void put16(uint32_t taddr, const Cols16& x)
{
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 t = f2_get(x.p[i]);
        w[2 * i] = __float_as_uint(t.x);
        w[2 * i + 1] = __float_as_uint(t.y);
    }
    tmem_st16(taddr, w);
}
// As NT bf16 terms of 8 columns each, at taddr, taddr + 8 and at taddr2.  Two
// terms hold 16 bits of a value (off by at most 2^-17 of it), three 24, where
// one rounding (2^-9) would be all of the fp32 outputs' error.
template <int NT>
__device__ __forceinline__ void put_terms(uint32_t (&at)[NT], const Cols16& v)
{
    Cols16 x = v;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = f2_to_bf16x2(x.p[i]);
            if (n + 1 < NT) x.p[i] = f2_sub(x.p[i], f2_from_bf16x2(w[i]));
        }
        tmem_st8(at[n], w);
    }
}
template <int NT>
__device__ __forceinline__ void put_terms(uint32_t taddr, const Cols16& v, uint32_t taddr2 = 0)
{
    uint32_t at[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) at[n] = n < 2 ? taddr + 8 * n : taddr2;
    put_terms<NT>(at, v);
}
__device__ __forceinline__ void put_two(uint32_t high, uint32_t low, const Cols16& v)
{
    uint32_t at[2] = {high, low};
    put_terms<2>(at, v);
}
// S = f S + HS columns of what the products added.
template <int HS>
__device__ __forceinline__ void add_cols(f2 (&S)[HS / 2], uint32_t taddr, float f)
{
    const f2 g = f2_splat(f);
    uint32_t r[HS / 16][16];
#pragma unroll
    for (int k = 0; k < HS / 16; ++k) tmem_ld16(taddr + 16 * k, r[k]);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < HS / 16; ++k) {
        const Cols16 x = cols16(r[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) S[8 * k + i] = f2_fma(g, S[8 * k + i], x.p[i]);
    }
}
template <int HS>
__device__ __forceinline__ Cols16 cols_of(const f2 (&S)[HS / 2], int k)
{
    Cols16 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.p[i] = S[8 * k + i];
    return x;
}
// A thread's HS state columns (rows of the [dk][dv] state, dv apart) from and to memory.
template <int HS>
__device__ __forceinline__ void load_state(f2 (&S)[HS / 2], const float* s, int dv)
{
#pragma unroll
    for (int i = 0; i < HS / 2; ++i)
        S[i] = s ? f2_make(s[static_cast<int64_t>(2 * i) * dv], s[static_cast<int64_t>(2 * i + 1) * dv]) : f2_splat(0.f);
}
template <int HS>
__device__ __forceinline__ void store_state(const f2 (&S)[HS / 2], float* s, int dv)
{
#pragma unroll
    for (int i = 0; i < HS / 2; ++i) {
        const float2 t = f2_get(S[i]);
        s[static_cast<int64_t>(2 * i) * dv] = t.x;
        s[static_cast<int64_t>(2 * i + 1) * dv] = t.y;
    }
}
// Arrive for this warp once its tensor-memory stores are done.
__device__ __forceinline__ void warp_done(uint64_t* bar, int lane)
{
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// A wait of a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, ctl));
}

}  // namespace gla
