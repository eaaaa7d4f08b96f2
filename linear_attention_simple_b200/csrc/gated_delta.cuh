// gated_delta.cuh -- shared by the gated delta rule's kernels: the sequence
// geometry, the records and the workspace, warp-level matrix products on bf16
// fragments.
//
// Chunks have 64 tokens.  With b the running sum of the log-decays inside a
// chunk, G_i = e^{b_i}, R_i = e^{b_63 - b_i}, D_ij = e^{b_i - b_j} and S the
// state that enters the chunk:
//
//   T  = (I + tril(K K^T . D_ij beta_j, -1))^-1        unit lower triangular
//   y  = G K S - (T - I)(V - G K S)                    what the state predicts
//   z  = V - y,   V' = beta z
//   o  = scale G Q S + P V',   P = tril(scale Q K^T . D)
//   S' = G_63 S + K^T (R V')
//
// The all-chunks kernel (gated_delta_chunks.cu) finds T and P; the sweeps
// (gated_delta_sweep_fwd.cu, gated_delta_sweep_bwd.cu) walk the chunks with the
// state transposed, [dv][dk], its rows on the lanes of tensor memory: rows of
// the state never meet, so a slice of them is a CTA's own.
#pragma once

#include <cuda_bf16.h>

#include "gla_device.cuh"

namespace gla {

constexpr int kGdC = 64;                 // tokens per chunk
constexpr int kGdPad = 8;                // bf16 elements behind each shared-memory row: rows an odd
                                         // multiple of 16 bytes apart, so ldmatrix has no bank conflicts
constexpr int kGdPiece = 32 * 16;        // a piece: 16 values of each of 32 dv rows (32-byte swizzle)
// Per-token scalars of a chunk: G, R, beta~, P_ii, b (high, low).  beta~ is beta in
// the forward; in the backward it is beta but no nearer to zero than 2^-40, and two
// scalars more are beta and beta / beta~.  dbeta is <dv, z> / beta, and dv = beta dV'
// would lose its bits (at beta = 0 all of them): so T and the reverse sweep have
// beta~, which changes their sums by 2^-40 of a term; V' has beta, and dv leaves with
// the factor.  (1e-30 in beta~'s place left dbeta 14 bits at a dO of 2^-30 and none
// at 2^-60.)
constexpr int gd_scalars(bool bwd) { return bwd ? 8 : 6; }
enum { kScG = 0, kScR = 1, kScBt = 2, kScPd = 3, kScBh = 4, kScBl = 5, kScBeta = 6, kScF = 7 };
constexpr float kGdBetaMin = 0x1p-40f;

// Sequences of one call: dense [N][T] (cu null) or packed rows cu[n] .. cu[n+1]-1.
struct GdSeqs {
    const int* cu;
    int N, T;          // T: tokens of each sequence (dense), of all together (packed)
    int H, Hk;         // value heads, query/key heads
    // Row of token 0 and length of sequence n; length -1 for packed offsets
    // that are not inside 0 .. T.
    __device__ __forceinline__ void span(int n, int64_t& row, int& len) const
    {
        if (!cu) {
            row = static_cast<int64_t>(n) * T;
            len = T;
            return;
        }
        const int s = cu[n], e = cu[n + 1];
        const bool ok = s >= 0 && e >= s && e <= T;
        row = ok ? s : 0;
        len = ok ? e - s : -1;
    }
    // Chunk slot of sequence n's first chunk: distinct for all chunks of all
    // sequences, without the lengths on the host.
    __device__ __forceinline__ int64_t slot0(int n, int64_t row) const
    {
        return cu ? row / kGdC + n : static_cast<int64_t>(n) * ((T + kGdC - 1) / kGdC);
    }
};

// What the all-chunks kernel leaves of a (chunk, value head) for the sweeps:
// one record, copied to shared memory as it is, its tiles in the layouts that
// the tensor core reads: K as blocks of [64 tokens][32] (64-byte swizzle), T and
// P in two bf16 terms as [64][64] (128-byte swizzle); and the scalars, in the
// forward's record scale G in the place of P_ii.  The backward's has scale G Q
// too, in two terms, T without its unit diagonal and P without its diagonal.
template <int DK, bool BWD>
struct GdRec {
    static constexpr int K = 0;
    static constexpr int SC = DK * 128;
    static constexpr int KSC = SC + gd_scalars(BWD) * kGdC * 4;    // K and the scalars: one copy
    static constexpr int Q = (KSC + 1023) / 1024 * 1024;           // tiles start on their swizzle's period
    static constexpr int QL = Q + DK * 128;                        // Q: BWD only
    static constexpr int T = BWD ? QL + DK * 128 : Q;
    static constexpr int TL = T + 8192;
    static constexpr int P = TL + 8192;
    static constexpr int PL = P + 8192;
    static constexpr int BYTES = PL + 8192;
};
inline size_t gd_rec_bytes(int dk, bool bwd)
{
    switch (dk) {
    case 64: return bwd ? GdRec<64, true>::BYTES : GdRec<64, false>::BYTES;
    case 96: return bwd ? GdRec<96, true>::BYTES : GdRec<96, false>::BYTES;
    default: return bwd ? GdRec<128, true>::BYTES : GdRec<128, false>::BYTES;
    }
}

// Sequence of a chunk slot (the last n whose first slot is <= slot).
__device__ __forceinline__ int gd_seq_of_slot(const GdSeqs& s, int64_t slot)
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

inline int64_t gd_slots(bool packed, int64_t N, int64_t T)
{
    return packed ? T / kGdC + N : N * ((T + kGdC - 1) / kGdC);
}

// ---- asynchronous copies: 16 bytes, zero-filled when !valid (src readable anyway).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// 64 rows of `width` bf16 values into rows of `stride`; rows from `valid` on are zeros.
__device__ __forceinline__ void gd_load_rows(__nv_bfloat16* dst, int stride, const __nv_bfloat16* src, int64_t ld,
                                             int width, int valid, int tid, int nthreads)
{
    const int per = width >> 3;
    for (int i = tid; i < kGdC * per; i += nthreads) {
        const int r = i / per, c = (i - r * per) * 8;
        const bool ok = r < valid;
        cp_async16(dst + r * stride + c, ok ? src + r * ld + c : src, ok);
    }
}

// ---- fragments
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Address of this lane's row for ldmatrix, as an element offset from the tile's
// origin, `ld` elements a row.
//   rows_n: a 16 x 16 tile stored [n][k]: r0, r1 = the right operand of n 0-7
//           (k 0-7, k 8-15), r2, r3 of n 8-15.
//   rows_a: a left operand of 16 rows from a tile stored [m][k].
__device__ __forceinline__ int rows_n(int lane, int ld) { return ((lane & 7) + ((lane >> 4) << 3)) * ld + (((lane >> 3) & 1) << 3); }
__device__ __forceinline__ int rows_a(int lane, int ld) { return (lane & 15) * ld + ((lane >> 4) << 3); }

// 2^x for the decay factors, x <= 0 where the result is used (0 -> 1, below
// -126 -> 0: such a factor is lost in any sum with others).
__device__ __forceinline__ float gd_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- parameters
struct GdParams {
    GdSeqs seqs;
    const __nv_bfloat16 *q, *k, *v, *dO;
    const float *a, *beta, *s0, *ds_final;
    int64_t ld_qk, ld_v, ld_do;
    int dk, dv;
    float scale;
    __nv_bfloat16 *o, *dq, *dkk, *dvv;
    float *s_final, *da, *dbeta, *ds0;
    // workspace, one entry per chunk slot and value head (u = slot * H + h)
    unsigned char* rec;     // [u]: GdRec
    // backward only; a "half row" is a thread's: one dv row, half of the columns
    __nv_bfloat16 *sb, *eb; // [u][dv / 32][dk / 16][piece]: the state entering, the gradient of the state leaving
    float* sn;              // [u][dv / 32][2][dk / 8][32 lanes][4]: the state entering in fp32, half rows
    float* sn_last;         // [N H][..]: the final state in the same form
    float* yn;              // [u][dv / 32][2][8][32 lanes][4]: y, half rows
    __nv_bfloat16* vp;      // [u][dv / 32][2][4][piece]: V', two terms, 16 tokens a piece
    float* part;            // [u][3][dv / 32][64]: sums over 32 dv rows, per token
    float* anch;            // [u][dv / 32][2]: <gradient of the state leaving, state leaving>
    // segments of seg_chunks chunks, at most nseg of a sequence; per (sequence,
    // head, segment) the state that enters [dk][dv], A [dk][dk] and (backward)
    // the gradient of the state that leaves [dk][dv]
    int nseg, seg_chunks;
    float *seg_l, *seg_a, *seg_e;
    int64_t slots;
    int* status;
};

gla_status gd_launch_chunks(const GdParams& p, bool bwd, cudaStream_t st);
gla_status gd_launch_sweep_fwd(const GdParams& p, const WaitCtl& ctl, cudaStream_t st);
gla_status gd_launch_segment_states(const GdParams& p, const WaitCtl& ctl, cudaStream_t st);
gla_status gd_launch_segment_grads(const GdParams& p, cudaStream_t st);
gla_status gd_launch_sweeps_bwd(const GdParams& p, const WaitCtl& ctl, cudaStream_t st);
gla_status gd_launch_grad(const GdParams& p, const WaitCtl& ctl, cudaStream_t st);

}  // namespace gla
