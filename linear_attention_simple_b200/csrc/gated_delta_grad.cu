// gated_delta_grad.cu -- dq, dk, da and dbeta of the gated delta rule, every
// chunk at once.  With X = scale dO, Y = -dv, the state S that enters the
// chunk and the gradient E of the state that leaves it:
//
//   A_ij = X_i . v'_j D_ij (i >= j)      B_ij = Y_i . v'_j D_ij (i > j)
//   dq = A K + G X S^T
//   dk = A^T Q + B^T K + B K + G Y S^T + R V' E^T
//   da_t = sum over i >= t of (o.dO - dv.y - dvs.z)_i up to the next <E, S'>
//          (every 128 tokens), and that
//
// One CTA of 4 warps per (chunk, q/k head), 16 token rows to a warp; the
// value heads that share the q/k head are summed in its accumulators.  A
// first pass over dv (32 columns a stage, two stages) gives A and B, each warp
// its own rows, the tiles above the diagonal left out; they are rounded to
// bf16, multiply K from the registers and, from shared memory, transposed, Q
// and K; a second pass adds the three products with the states.  dq and dk
// leave in bf16, so every operand is one bf16 rounding of its value; the sums
// behind da and dbeta come in fp32 from the sweeps.
//
// Latency bounds it (three CTAs an SM, 12 warps): where a value head has a
// q/k head of its own (ONE), the accumulators of dq and dk start only after
// the first pass, which leaves 168 registers a thread enough.
#include "gated_delta.cuh"

namespace gla {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kMaxWarps = 8;               // of 32 dv rows (dv <= 256)
constexpr int kSl = 32;                    // dv columns per stage
constexpr int kVs = kSl + kGdPad;          // row stride of a staged token slice

template <int DK>
struct GradSmem {
    static constexpr int KS = DK + kGdPad;
    static constexpr int tok = kGdC * kVs;             // one staged token slice of dO or dv
    // V' and the states as they lie in memory, in pieces of 8 values of 32 dv
    // rows: 16 bytes a row, so that ldmatrix meets every bank once
    static constexpr int vt = kSl * kGdC;
    static constexpr int st = kSl * DK;
    static constexpr int stage1 = 2 * tok + vt, stage2 = stage1 + 2 * st;
    // elements: the first pass's stages, later A and B; then K and Q; the
    // second pass's stages over all of them
    static constexpr int ab = kGdC * (kGdC + kGdPad);
    static constexpr int kq = 2 * stage1;
    static constexpr int all = kq + 2 * kGdC * KS > 2 * stage2 ? kq + 2 * kGdC * KS : 2 * stage2;
    static constexpr int bytes = all * 2 + kGdSc * kGdC * 4;
};

struct Src {
    const __nv_bfloat16 *d, *y, *vp, *s, *e;
    int64_t ld_do, ld_dv;
    int dv, valid;
};

// Stage i of pass 1 (dO, dv, V') or of pass 2 (those and both states).
template <int DK>
__device__ __forceinline__ void load_slice(__nv_bfloat16* st, const Src& x, int col, bool states, int tid)
{
    constexpr int KS = GradSmem<DK>::KS, tok = GradSmem<DK>::tok;
    gd_load_rows(st, kVs, x.d + col, x.ld_do, kSl, x.valid, tid, kThreads);
    gd_load_rows(st + tok, kVs, x.y + col, x.ld_dv, kSl, x.valid, tid, kThreads);
    __nv_bfloat16* sv = st + 2 * tok;
    for (int i = tid; i < GradSmem<DK>::vt / 8; i += kThreads)
        cp_async16(sv + 8 * i, x.vp + static_cast<int64_t>(col) * kGdC + 8 * i, true);
    if (states) {
        constexpr int n = GradSmem<DK>::st / 8;
        __nv_bfloat16* ss = st + GradSmem<DK>::stage1;
        for (int i = tid; i < n; i += kThreads) {
            cp_async16(ss + 8 * i, x.s + static_cast<int64_t>(col) * DK + 8 * i, true);
            cp_async16(ss + 8 * (n + i), x.e + static_cast<int64_t>(col) * DK + 8 * i, true);
        }
    }
}

// The rows_k and rows_at patterns on pieces.
__device__ __forceinline__ int piece_k(int lane) { return (lane >> 4) * kGdPiece + ((lane & 7) + (((lane >> 3) & 1) << 3)) * 8; }
__device__ __forceinline__ int piece_at(int lane) { return ((lane >> 3) & 1) * kGdPiece + ((lane & 7) + ((lane >> 4) << 3)) * 8; }

// A left operand's rows g and g + 8 times f0 and f1.
__device__ __forceinline__ void scale_a(uint32_t (&r)[4], float f0, float f1)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = i & 1 ? f1 : f0;
        r[i] = pack_bf16(f * bf16_lo(r[i]), f * bf16_hi(r[i]));
    }
}

template <int DK, bool ONE>
__global__ void __launch_bounds__(kThreads, ONE ? 3 : 2) gd_grad_kernel(GdParams p)
{
    using M = GradSmem<DK>;
    constexpr int KS = M::KS, NT = DK / 8;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    constexpr int AS = kGdC + kGdPad;                      // row stride of A and B
    __nv_bfloat16* sst = reinterpret_cast<__nv_bfloat16*>(smem_raw);
    __nv_bfloat16* sk = sst + M::kq;
    __nv_bfloat16* sq = sk + kGdC * KS;
    float* sc = reinterpret_cast<float*>(sst + M::all);

    const int64_t slot = blockIdx.x;
    const int hk = blockIdx.y;
    const int n = gd_seq_of_slot(p.seqs, slot);
    int64_t row0;
    int len;
    p.seqs.span(n, row0, len);
    if (len < 0) return;
    const int64_t c = slot - p.seqs.slot0(n, row0);
    if (c < 0 || c * kGdC >= len) return;
    const int valid = min(kGdC, len - static_cast<int>(c) * kGdC);
    const int64_t row = row0 + c * kGdC;
    [[maybe_unused]] const int64_t rows = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;   // of the checking build
    const int H = p.seqs.H, group = H / p.seqs.Hk;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, c2 = (lane & 3) * 2;
    const int nst = p.dv / kSl, wtot = p.dv >> 5;

    float dq[NT][4], dk[NT][4];
    if (!ONE) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) dq[t][e] = dk[t][e] = 0.f;
    }

    for (int j = 0; j < (ONE ? 1 : group); ++j) {
        const int h = hk * group + j;
        const int64_t u = slot * H + h;
        Src x{p.dO + row * p.ld_do + static_cast<int64_t>(h) * p.dv, p.dvv + row * H * p.dv + static_cast<int64_t>(h) * p.dv,
              p.vp + u * kGdC * p.dv, p.sb + u * p.dv * DK, p.eb + u * p.dv * DK,
              p.ld_do, static_cast<int64_t>(H) * p.dv, p.dv, valid};
        __syncthreads();                   // the last head's scalars and stages are read
        const float* src_sc = reinterpret_cast<const float*>(p.rec + u * GdRec<DK, true>::BYTES + GdRec<DK, true>::SC);
        for (int i = tid; i < kGdSc * kGdC; i += kThreads) sc[i] = src_sc[i];
        load_slice<DK>(sst, x, 0, false, tid);
        gd_load_rows(sk, KS, p.k + row * p.ld_qk + hk * DK, p.ld_qk, DK, valid, tid, kThreads);
        gd_load_rows(sq, KS, p.q + row * p.ld_qk + hk * DK, p.ld_qk, DK, valid, tid, kThreads);
        cp_async_commit();

        // pass 1: products over dv of 16 rows with the tokens up to them, before the masks
        float fa[8][4], fb[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) fa[t][e] = fb[t][e] = 0.f;
        for (int i = 0; i < nst; ++i) {
            cp_async_wait<0>();
            __syncthreads();
            if (i + 1 < nst) load_slice<DK>(sst + ((i + 1) & 1) * M::stage1, x, (i + 1) * kSl, false, tid);
            cp_async_commit();
            const __nv_bfloat16* st = sst + (i & 1) * M::stage1;
            const uint32_t ar = smem_u32(st + 16 * w * kVs + rows_a(lane, kVs));
            const uint32_t br = smem_u32(st + 2 * M::tok + piece_k(lane));
            constexpr int tk = M::tok * 2;
#pragma unroll
            for (int s = 0; s < kSl / 16; ++s) {
                uint32_t d[4], y[4];
                ldsm4(d, ar + s * 32);
                ldsm4(y, ar + tk + s * 32);
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    if (np > w) continue;
                    uint32_t b[4];
                    ldsm4_t(b, br + s * 256 + np * 4 * kGdPiece);
                    mma_bf16(fa[2 * np], d, b[0], b[1]);
                    mma_bf16(fa[2 * np + 1], d, b[2], b[3]);
                    mma_bf16(fb[2 * np], y, b[0], b[1]);
                    mma_bf16(fb[2 * np + 1], y, b[2], b[3]);
                }
            }
        }
        __syncthreads();                   // both stages are read

        // da and dbeta of this head: one warp, two tokens a lane
        if (w == (j & 3)) {
            // <E, S'> is there after every second chunk and the last; before the
            // others come the sums of the chunk in between
            const float* part = p.part + u * 3 * wtot * kGdC + 2 * lane;
            const bool between = (c & 1) == 0 && (c + 1) * kGdC < len;
            float2 od = make_float2(0.f, 0.f), s1 = od, s2 = od;
            float tail = 0.f, next = 0.f;
#pragma unroll
            for (int t = 0; t < kMaxWarps; ++t) {          // all loads at once
                if (t >= wtot) continue;
                const float2 a = *reinterpret_cast<const float2*>(part + t * kGdC);
                const float2 b = *reinterpret_cast<const float2*>(part + (wtot + t) * kGdC);
                const float2 e = *reinterpret_cast<const float2*>(part + (2 * wtot + t) * kGdC);
                od.x += a.x; od.y += a.y;
                s1.x += b.x; s1.y += b.y;
                s2.x += e.x; s2.y += e.y;
                const int64_t un = between ? u + H : u;
                const float2 an = *reinterpret_cast<const float2*>(p.anch + (un * wtot + t) * 2);
                tail += an.x + an.y;
                if (between) {
                    const float* pn = part + static_cast<int64_t>(H) * 3 * wtot * kGdC;
                    const float2 f = *reinterpret_cast<const float2*>(pn + t * kGdC);
                    const float2 k = *reinterpret_cast<const float2*>(pn + (wtot + t) * kGdC);
                    next += (f.x - k.x) + (f.y - k.y);
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) next += __shfl_xor_sync(0xFFFFFFFFu, next, o);
            tail += next;
            const float d1 = od.y - s1.y;
            float s = (od.x - s1.x) + d1;          // sums over this lane's tokens and all later ones
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float z = __shfl_down_sync(0xFFFFFFFFu, s, o);
                if (lane + o < 32) s += z;
            }
            const float after = __shfl_down_sync(0xFFFFFFFFu, s, 1);
            const float later = lane < 31 ? after : 0.f;
            const int64_t at = (row + 2 * lane) * H + h;
            if (2 * lane < valid && GLA_DCHECK(at >= 0 && at < rows * H, p.status)) {
                p.da[at] = s + tail;
                p.dbeta[at] = s2.x / sc[kScBeta * kGdC + 2 * lane];
            }
            if (2 * lane + 1 < valid && GLA_DCHECK(at + H < rows * H, p.status)) {
                p.da[at + H] = later + d1 + tail;
                p.dbeta[at + H] = s2.y / sc[kScBeta * kGdC + 2 * lane + 1];
            }
        }

        // masks and decays; A and B as left operands, and to shared memory
        uint32_t pa[4][4], pb[4][4];
        {
            const float bh0 = sc[kScBh * kGdC + 16 * w + g], bl0 = sc[kScBl * kGdC + 16 * w + g];
            const float bh1 = sc[kScBh * kGdC + 16 * w + g + 8], bl1 = sc[kScBl * kGdC + 16 * w + g + 8];
            uint32_t* sa = reinterpret_cast<uint32_t*>(sst + (16 * w + g) * AS + c2);
            uint32_t* sb = reinterpret_cast<uint32_t*>(sst + M::ab + (16 * w + g) * AS + c2);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if ((t >> 1) > w) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) pa[t >> 1][2 * (t & 1) + e] = pb[t >> 1][2 * (t & 1) + e] = 0u;
                    continue;
                }
                const float2 qh = *reinterpret_cast<const float2*>(sc + kScBh * kGdC + 8 * t + c2);
                const float2 ql = *reinterpret_cast<const float2*>(sc + kScBl * kGdC + 8 * t + c2);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 16 * w + g + 8 * (e >> 1), q = 8 * t + c2 + (e & 1);
                    const float diff = ((e >> 1 ? bh1 : bh0) - (e & 1 ? qh.y : qh.x)) + ((e >> 1 ? bl1 : bl0) - (e & 1 ? ql.y : ql.x));
                    const float d = q <= r ? gd_exp2(diff) : 0.f;
                    fa[t][e] *= d * p.scale;
                    fb[t][e] = q < r ? -fb[t][e] * d : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t a = pack_bf16(fa[t][2 * e], fa[t][2 * e + 1]), b = pack_bf16(fb[t][2 * e], fb[t][2 * e + 1]);
                    pa[t >> 1][2 * (t & 1) + e] = a;
                    pb[t >> 1][2 * (t & 1) + e] = b;
                    sa[(8 * e * AS + 8 * t) / 2] = a;
                    sb[(8 * e * AS + 8 * t) / 2] = b;
                }
            }
        }
        __syncthreads();
        // dq += A K; dk += A^T Q + B K + B^T K
        {
            if (ONE) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dq[t][e] = dk[t][e] = 0.f;
            }
            const uint32_t kt = smem_u32(sk + rows_k(lane, KS)), qt = smem_u32(sq + rows_k(lane, KS));
            const uint32_t ta = smem_u32(sst + 16 * w + rows_at(lane, AS)), tb = ta + M::ab * 2;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t at[4], bt[4];
                if (s >= w) {
                    ldsm4_t(at, ta + s * 16 * AS * 2);
                    ldsm4_t(bt, tb + s * 16 * AS * 2);
                }
#pragma unroll
                for (int np = 0; np < DK / 16; ++np) {
                    uint32_t kf[4], qf[4];
                    ldsm4_t(kf, kt + s * 16 * KS * 2 + np * 32);
                    if (s <= w) {
                        mma_bf16(dq[2 * np], pa[s], kf[0], kf[1]);
                        mma_bf16(dq[2 * np + 1], pa[s], kf[2], kf[3]);
                        mma_bf16(dk[2 * np], pb[s], kf[0], kf[1]);
                        mma_bf16(dk[2 * np + 1], pb[s], kf[2], kf[3]);
                    }
                    if (s >= w) {
                        ldsm4_t(qf, qt + s * 16 * KS * 2 + np * 32);
                        mma_bf16(dk[2 * np], bt, kf[0], kf[1]);
                        mma_bf16(dk[2 * np + 1], bt, kf[2], kf[3]);
                        mma_bf16(dk[2 * np], at, qf[0], qf[1]);
                        mma_bf16(dk[2 * np + 1], at, qf[2], qf[3]);
                    }
                }
            }
        }
        __syncthreads();                   // K, Q, A and B are read
        load_slice<DK>(sst, x, 0, true, tid);
        cp_async_commit();

        // pass 2: dq += G X S^T, dk += G Y S^T + R V' E^T
        const float G0 = sc[kScG * kGdC + 16 * w + g], G1 = sc[kScG * kGdC + 16 * w + g + 8];
        const float R0 = sc[kScR * kGdC + 16 * w + g], R1 = sc[kScR * kGdC + 16 * w + g + 8];
        for (int i = 0; i < nst; ++i) {
            cp_async_wait<0>();
            __syncthreads();
            if (i + 1 < nst) load_slice<DK>(sst + ((i + 1) & 1) * M::stage2, x, (i + 1) * kSl, true, tid);
            cp_async_commit();
            const __nv_bfloat16* st = sst + (i & 1) * M::stage2;
            const uint32_t ar = smem_u32(st + 16 * w * kVs + rows_a(lane, kVs));
            const uint32_t vr = smem_u32(st + 2 * M::tok + 2 * w * kGdPiece + piece_at(lane));
            const uint32_t sr = smem_u32(st + M::stage1 + piece_k(lane));
            constexpr int tk = M::tok * 2;
#pragma unroll
            for (int s = 0; s < kSl / 16; ++s) {
                uint32_t d[4], y[4], v[4];
                ldsm4(d, ar + s * 32);
                ldsm4(y, ar + tk + s * 32);
                ldsm4_t(v, vr + s * 256);
                scale_a(d, p.scale * G0, p.scale * G1);
                scale_a(y, -G0, -G1);
                scale_a(v, R0, R1);
#pragma unroll
                for (int np = 0; np < DK / 16; ++np) {
                    uint32_t sf[4], ef[4];
                    ldsm4_t(sf, sr + s * 256 + np * 4 * kGdPiece);
                    ldsm4_t(ef, sr + M::st * 2 + s * 256 + np * 4 * kGdPiece);
                    mma_bf16(dq[2 * np], d, sf[0], sf[1]);
                    mma_bf16(dq[2 * np + 1], d, sf[2], sf[3]);
                    mma_bf16(dk[2 * np], y, sf[0], sf[1]);
                    mma_bf16(dk[2 * np + 1], y, sf[2], sf[3]);
                    mma_bf16(dk[2 * np], v, ef[0], ef[1]);
                    mma_bf16(dk[2 * np + 1], v, ef[2], ef[3]);
                }
            }
        }
    }
    // out through this warp's own rows of the K and Q tiles
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int at = (16 * w + g + 8 * hf) * KS + 8 * t + c2;
            *reinterpret_cast<uint32_t*>(sq + at) = pack_bf16(dq[t][2 * hf], dq[t][2 * hf + 1]);
            *reinterpret_cast<uint32_t*>(sk + at) = pack_bf16(dk[t][2 * hf], dk[t][2 * hf + 1]);
        }
    __syncwarp();
    const int64_t ld = static_cast<int64_t>(p.seqs.Hk) * DK;
    for (int i = lane; i < 16 * (DK / 8); i += 32) {
        const int r = 16 * w + i / (DK / 8), cc = (i % (DK / 8)) * 8;
        if (r < valid && GLA_DCHECK(row + r < rows, p.status)) {
            const int64_t at = (row + r) * ld + hk * DK + cc;
            *reinterpret_cast<uint4*>(p.dq + at) = *reinterpret_cast<const uint4*>(sq + r * KS + cc);
            *reinterpret_cast<uint4*>(p.dkk + at) = *reinterpret_cast<const uint4*>(sk + r * KS + cc);
        }
    }
}

template <int DK, bool ONE>
gla_status launch(const GdParams& p, cudaStream_t st)
{
    constexpr int smem = GradSmem<DK>::bytes;
    cudaError_t e = cudaFuncSetAttribute(gd_grad_kernel<DK, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    trace_begin(st);
    gd_grad_kernel<DK, ONE><<<dim3(static_cast<unsigned>(p.slots), static_cast<unsigned>(p.seqs.Hk)), kThreads, smem, st>>>(p);
    trace_end(st, "gd_grad_kernel");
    count_launch();
    return check_launch("gd_grad_kernel");
}

template <int DK>
gla_status pick(const GdParams& p, cudaStream_t st)
{
    return p.seqs.H == p.seqs.Hk ? launch<DK, true>(p, st) : launch<DK, false>(p, st);
}

}  // namespace

gla_status gd_launch_grad(const GdParams& p, cudaStream_t st)
{
    if (p.slots == 0) return GLA_OK;
    switch (p.dk) {
    case 64: return pick<64>(p, st);
    case 96: return pick<96>(p, st);
    default: return pick<128>(p, st);
    }
}

}  // namespace gla
