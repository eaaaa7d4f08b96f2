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

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
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

// Sixteen fp32 values as two bf16 terms: 8 columns each.
__device__ __forceinline__ void split16(const float (&x)[16], uint32_t (&hi)[8], uint32_t (&lo)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        lo[i] = pack_bf16(x[2 * i] - bf16_lo(hi[i]), x[2 * i + 1] - bf16_hi(hi[i]));
    }
}
__device__ __forceinline__ void load16(float (&x)[16], const float* p)
{
#pragma unroll
    for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(p + i);
}
__device__ __forceinline__ void get16(float (&x)[16], uint32_t taddr)
{
    uint32_t r[16];
    tmem_ld16(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}

// A wait of a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, ctl));
}

}  // namespace gla
