// gated_delta_grad.cu -- dq, dk, da and dbeta of the gated delta rule, every
// chunk at once.  With X = dO, Y = dv, the state S that enters the chunk and the
// gradient E of the state that leaves it:
//
//   A_ij = scale X_i . v'_j D_ij (i >= j)      B_ij = -Y_i . v'_j D_ij (i > j)
//   dq = scale G X S^T + A K
//   dk = -G Y S^T + R V' E^T + (B + B^T) K + A^T Q
//   da_t = sum over i >= t of (o.dO - dv.y - dvs.z)_i up to the next <E, S'>
//          (every 128 tokens), and that
//
// The 64 rows of X stand over the 64 rows of Y in shared memory, so dq's tokens
// are lanes 0-63 of tensor memory and dk's lanes 64-127, and every product is
// one of 128 rows.  Per 64 columns of dv:
//
//   D1 += [X; Y] V'^T      D2 += [X; Y] S^T      D3 += [.; V'] E^T
//
// ([.; V']: its upper rows are whatever lies before V' in shared memory; what
// they give is not read).  Workers take scale G D2 and -G D2 + R D3 into their
// registers, turn D1, masked and decayed, into A over B (in shared memory), and
// the tensor core reads those as they stand and transposed:
//
//   D4 = [A; B] K + [0; B^T] K + [0; A^T] Q
//
// The value heads that share a q/k head are added up in the registers.  V', A and
// B are two bf16 terms, dO, K and Q are exact; S, E and dv are one term each: the
// parts that they give are the smaller ones unless decays are slow, and their
// second terms would double this kernel's bytes.  With the usual decays dq is off
// by 1.74e-3 and dk by 1.8e-3, of which 1.66e-3 is their own rounding (one term of
// V', A and B too: 2.9e-3; 147 us here and 304 in the reverse sweep where it is
// 168 and 325 so); with slow ones by 2.3e-3 and 2.5e-3.  The sums behind da and
// dbeta come in fp32 from the sweeps, and a warp of its own adds them up.
//
// The states and V' are read as the sweeps left them, in pieces of 16 values of
// 32 dv rows with the tensor core's 32-byte swizzle.  One CTA an SM walks over
// (chunk, head): a ring of stages of 64 dv columns keeps the loads going,
// and the products of the next unit start as soon as D2 and D3 are read (D1 has
// two buffers).  Every byte is read once, and HBM bounds it: 8 x 2,048 tokens,
// 16 heads of 96 x 192, 920 MB in 168 us, 5.5 TB/s.  (With one term each, mma.sync,
// two passes over dv and 12 warps an SM, latency did: 272 us against 146.)
#include "gated_delta_tc.cuh"

namespace gla {
namespace {

constexpr int kSms = 148;
constexpr int kThreads = (kGdWorkers + 4) * 32;      // + a slice, an issue, a sums and a tile warp
constexpr int kCols = 64;                            // dv columns of a stage
constexpr int kPieceBytes = kGdPiece * 2;
constexpr int kMaxWarps = 8;                         // of 32 dv rows (dv <= 256)

// Tensor memory columns.
template <int DK>
struct Cols {
    static constexpr int D1 = 0, D2 = 128, D3 = D2 + DK, D4 = D3 + DK, ALLOC = 512;       // D1: two buffers of 64
};
template <int DK>
struct Smem {
    using Rec = GdRec<DK, true>;
    static constexpr int VB = 8 * kPieceBytes, SB = DK / 16 * kPieceBytes;        // of 32 dv columns
    static constexpr int X = 0, Y = 8192, V = 16384, S = V + 2 * VB, E = S + 2 * SB, STAGE = E + 2 * SB;
    // a tile of zeros, A, B, their second terms; K and Q, later dk and dq; b of two units
    static constexpr int STAGES = DK == 64 ? 3 : 2, AB = 2 * 8192;
    static constexpr int Z = STAGES * STAGE, A = Z + 8192, K = A + 2 * AB, Q = K + kGdC * DK * 2, SC = Q + kGdC * DK * 2;
    static constexpr int SCB = 2 * kGdC * 4, BARS = SC + 2 * SCB, bytes = BARS + 256 + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of an SM");
};
template <int STAGES>
struct __align__(8) Bars {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t sc[2], sc_done[2];                      // b; workers -> copies
    uint64_t kq, kq_done;                            // K and Q; workers -> copies: free, or holding dk and dq
    uint64_t d123, d4, drain;                        // issuer -> workers, itself
    uint64_t w, read;                                // workers -> issuer: A and B are there; D2 and D3 are read
    uint32_t tmem;
};
struct Maps {
    CUtensorMap dO, dv, q, dq, dk;
};

// A (chunk, q/k head) of this CTA.
struct Unit {
    int64_t slot;
    int hk, row, valid;     // row: the chunk's first token
    bool between;           // <E, S'> is kept for the chunk behind this one, not for this one
    bool first;             // of its sequence
};
// Calls work for this CTA's units in turn, the same for all lanes, until it
// returns false.  32 units at a time are looked up, a lane each.
template <class F>
__device__ __forceinline__ void for_units(const GdParams& p, int lane, F work)
{
    const int64_t total = p.slots * p.seqs.Hk, step = gridDim.x;
    for (int64_t base = blockIdx.x; base < total; base += 32 * step) {
        const int64_t i = base + lane * step;
        int row = 0, valid = 0;
        int flags = 0;
        if (i < total) {
            const int64_t slot = i / p.seqs.Hk;
            const int n = gd_seq_of_slot(p.seqs, slot);
            int64_t row0;
            int len;
            p.seqs.span(n, row0, len);
            const int64_t c = slot - p.seqs.slot0(n, row0);
            if (len >= 0 && c >= 0 && c * kGdC < len) {      // else between two sequences
                row = static_cast<int>(row0 + c * kGdC);
                valid = min(kGdC, len - static_cast<int>(c) * kGdC);
                flags = ((c & 1) == 0 && (c + 1) * kGdC < len ? 1 : 0) | (c == 0 ? 2 : 0);
            }
        }
        for (uint32_t m = __ballot_sync(0xFFFFFFFFu, valid > 0); m; m &= m - 1) {
            const int l = __ffs(m) - 1;
            Unit u;
            u.slot = (base + l * step) / p.seqs.Hk;
            u.hk = static_cast<int>(base + l * step - u.slot * p.seqs.Hk);
            u.row = __shfl_sync(0xFFFFFFFFu, row, l);
            u.valid = __shfl_sync(0xFFFFFFFFu, valid, l);
            const int f = __shfl_sync(0xFFFFFFFFu, flags, l);
            u.between = (f & 1) != 0;
            u.first = (f & 2) != 0;
            if (!work(u)) return;
        }
    }
}

// da and dbeta of a (chunk, value head): one warp, two tokens a lane.
template <int DK>
__device__ __forceinline__ void sums(const GdParams& p, const Unit& x, int h, int lane)
{
    const int H = p.seqs.H, wtot = p.dv >> 5;
    const int64_t u = x.slot * H + h;
    const float* beta = reinterpret_cast<const float*>(p.rec + u * GdRec<DK, true>::BYTES + GdRec<DK, true>::SC) + kScBt * kGdC;
    // <E, S'> is there after every second chunk and the last; before the
    // others come the sums of the chunk in between
    const float* part = p.part + u * 3 * wtot * kGdC + 2 * lane;
    const float* pn = x.between ? part + static_cast<int64_t>(H) * 3 * wtot * kGdC : part;
    const float* an = p.anch + (x.between ? u + H : u) * wtot * 2;
    float2 od = make_float2(0.f, 0.f), s1 = od, s2 = od;
    float tail = 0.f, next = 0.f;
    // all loads at once: without branches, so that none waits for another
#pragma unroll
    for (int t = 0; t < kMaxWarps; ++t) {
        const bool on = t < wtot;
        const int tt = on ? t : 0;
        const float2 a = *reinterpret_cast<const float2*>(part + tt * kGdC);
        const float2 b = *reinterpret_cast<const float2*>(part + (wtot + tt) * kGdC);
        const float2 e = *reinterpret_cast<const float2*>(part + (2 * wtot + tt) * kGdC);
        const float2 f = *reinterpret_cast<const float2*>(pn + tt * kGdC);
        const float2 k = *reinterpret_cast<const float2*>(pn + (wtot + tt) * kGdC);
        const float2 n = *reinterpret_cast<const float2*>(an + tt * 2);
        od.x += on ? a.x : 0.f;
        od.y += on ? a.y : 0.f;
        s1.x += on ? b.x : 0.f;
        s1.y += on ? b.y : 0.f;
        s2.x += on ? e.x : 0.f;
        s2.y += on ? e.y : 0.f;
        tail += on ? n.x + n.y : 0.f;
        next += on && x.between ? (f.x - k.x) + (f.y - k.y) : 0.f;
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
    [[maybe_unused]] const int64_t rows = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;   // of the checking build
    const int64_t at = (static_cast<int64_t>(x.row) + 2 * lane) * H + h;
    if (2 * lane < x.valid && GLA_DCHECK(at >= 0 && at < rows * H, p.status)) {
        // nothing decays before a sequence's first token: what is left of its sum is
        // rounding (or not finite, and stays so)
        p.da[at] = x.first && lane == 0 && !p.s0 ? fmaf(0.f, s + tail, 0.f) : s + tail;
        p.dbeta[at] = s2.x / beta[2 * lane];
    }
    if (2 * lane + 1 < x.valid && GLA_DCHECK(at + H < rows * H, p.status)) {
        p.da[at + H] = later + d1 + tail;
        p.dbeta[at + H] = s2.y / beta[2 * lane + 1];
    }
}

template <int DK>
__global__ void __launch_bounds__(kThreads, 1) gd_grad_kernel(GdParams p, const __grid_constant__ Maps maps, WaitCtl ctl)
{
    using C = Cols<DK>;
    using M = Smem<DK>;
    using Rec = GdRec<DK, true>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int kStages = M::STAGES;
    Bars<kStages>& B = *reinterpret_cast<Bars<kStages>*>(smem + M::BARS);
    static_assert(sizeof(B) <= 256, "");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int H = p.seqs.H, group = H / p.seqs.Hk, ns = (p.dv + kCols - 1) / kCols;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&B.full[i], 1);
            mbar_init(&B.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.sc[i], 1);
            mbar_init(&B.sc_done[i], kGdWorkers);
        }
        uint64_t* one[4] = {&B.kq, &B.d123, &B.d4, &B.drain};
        for (uint64_t* b : one) mbar_init(b, 1);
        uint64_t* from_workers[3] = {&B.kq_done, &B.w, &B.read};
        for (uint64_t* b : from_workers) mbar_init(b, kGdWorkers);
        mbar_init_fence();
    }
    for (int i = tid; i < 8192 / 16; i += kThreads) reinterpret_cast<uint4*>(smem + M::Z)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    if (warp == kGdWorkers + 1) {
        tmem_alloc(&B.tmem, C::ALLOC);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = B.tmem;

    if (warp == kGdWorkers) {
        // ---- b; slices of dO, dv, V' and the states
        int step = 0, n = 0;
        for_units(p, lane, [&](const Unit& x) {
            bool ok = true;
            for (int j = 0; j < group && ok; ++j) {
                if (lane == 0) {
                    const int h = x.hk * group + j;
                    const int64_t u = x.slot * H + h;
                    const int b = step & 1;
                    ok = step < 2 || mbar_wait(&B.sc_done[b], ((step >> 1) - 1) & 1, ctl);
                    if (ok) {
                        mbar_arrive_expect_tx(&B.sc[b], M::SCB);
                        bulk_load(smem + M::SC + b * M::SCB, p.rec + u * Rec::BYTES + Rec::SC + kScBh * kGdC * 4, M::SCB, &B.sc[b]);
                        ++step;
                    }
                    for (int s = 0; s < ns && ok; ++s, ++n) {
                        const int st = n % kStages, col = s * kCols, left = min(kCols, p.dv - col);
                        ok = n < kStages || mbar_wait(&B.empty[st], (n / kStages - 1) & 1, ctl);
                        if (!ok) break;
                        unsigned char* at = smem + st * M::STAGE;
                        const uint32_t vb = left / 32 * M::VB, sb = left / 32 * M::SB;
                        const int64_t block = (u * p.dv + col) / 32;
                        mbar_arrive_expect_tx(&B.full[st], 16384 + vb + 2 * sb);
                        tma_load_2d(at + M::X, &maps.dO, &B.full[st], h * p.dv + col, x.row);
                        tma_load_2d(at + M::Y, &maps.dv, &B.full[st], h * p.dv + col, x.row);
                        bulk_load(at + M::V, p.vp + block * (M::VB / 2), vb, &B.full[st]);
                        bulk_load(at + M::S, p.sb + block * (M::SB / 2), sb, &B.full[st]);
                        bulk_load(at + M::E, p.eb + block * (M::SB / 2), sb, &B.full[st]);
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, static_cast<int>(ok), 0) != 0;
            }
            return ok;
        });
        // no copy may be in flight when the block ends
        if (lane == 0) {
            for (int i = max(0, n - kStages); i < n; ++i) mbar_wait(&B.full[i % kStages], (i / kStages) & 1, ctl);
            for (int i = max(0, step - 2); i < step; ++i) mbar_wait(&B.sc[i & 1], (i >> 1) & 1, ctl);
        }
        __syncwarp();
    } else if (warp == kGdWorkers + 3) {
        // ---- K and Q, and in their place dk and dq on the way out
        int step = 0, last_row = 0, last_hk = -1;             // heads so far; what waits to leave
        auto leave = [&]() {                                  // dq and dk of the step before, where whole
            if (step == 0) return true;
            if (!mbar_wait(&B.kq_done, (step - 1) & 1, ctl)) return false;
            if (last_hk >= 0) {
                for (int b = 0; b < DK / 32; ++b) {
                    tma_store_2d(&maps.dq, smem + M::Q + b * 4096, last_hk * DK + 32 * b, last_row);
                    tma_store_2d(&maps.dk, smem + M::K + b * 4096, last_hk * DK + 32 * b, last_row);
                }
                tma_store_commit();
                tma_store_wait_read();
            }
            return true;
        };
        for_units(p, lane, [&](const Unit& x) {
            bool ok = true;
            for (int j = 0; j < group && ok; ++j) {
                if (lane == 0) {
                    const unsigned char* rec = p.rec + (x.slot * H + x.hk * group + j) * Rec::BYTES;
                    bulk_prefetch_l2(rec, kGdC * DK * 2);
                    ok = leave();
                    if (ok) {
                        mbar_arrive_expect_tx(&B.kq, 2 * kGdC * DK * 2);
                        bulk_load(smem + M::K, rec, kGdC * DK * 2, &B.kq);
                        for (int b = 0; b < DK / 32; ++b)
                            tma_load_2d(smem + M::Q + b * 4096, &maps.q, &B.kq, x.hk * DK + 32 * b, x.row);
                        last_row = x.row;
                        last_hk = j + 1 == group && x.valid == kGdC ? x.hk : -1;
                        ++step;
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, static_cast<int>(ok), 0) != 0;
            }
            return ok;
        });
        if (lane == 0) {
            leave();
            tma_store_wait_read();
            if (step > 0) mbar_wait(&B.kq, (step - 1) & 1, ctl);
        }
        __syncwarp();
    } else if (warp == kGdWorkers + 1) {
        // ---- products
        int step = 0, n = 0;
        constexpr uint32_t id1 = idesc_bf16_f32(128, 64, 0, 1), id2 = idesc_bf16_f32(128, DK, 0, 1);
        constexpr uint32_t id3 = idesc_bf16_f32(128, DK, 1, 1);
        // A, B and the state's part of step t into dq and dk
        auto last_product = [&](int t) {
            if (!mbar_wait(&B.kq, t & 1, ctl) || !mbar_wait(&B.w, t & 1, ctl)) return false;
            tc_fence_after();
            const uint64_t k_n = smem_desc(smem_u32(smem + M::K), 4096, 512, kLayoutSW64);
            const uint64_t q_n = smem_desc(smem_u32(smem + M::Q), 4096, 512, kLayoutSW64);
            const uint64_t ab = smem_desc(smem_u32(smem + M::A), 16, 1024, kLayoutSW128);
            const uint64_t at = smem_desc(smem_u32(smem + M::Z), 8192, 1024, kLayoutSW128);         // zeros, then A
            const uint64_t bt = smem_desc(smem_u32(smem + M::Z), 16384, 1024, kLayoutSW128);        // zeros, then B
            const uint64_t atl = smem_desc(smem_u32(smem + M::Z), 8192 + M::AB, 1024, kLayoutSW128);
            const uint64_t btl = smem_desc(smem_u32(smem + M::Z), 16384 + M::AB, 1024, kLayoutSW128);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t kb = desc_add(k_n, 1024 * k), qb = desc_add(q_n, 1024 * k);
                umma_bf16(tm + C::D4, desc_add(ab, 32 * k), kb, id2, k > 0);
                umma_bf16(tm + C::D4, desc_add(ab, 32 * k + M::AB), kb, id2, 1);
                umma_bf16(tm + C::D4, desc_add(bt, 2048 * k), kb, id3, 1);
                umma_bf16(tm + C::D4, desc_add(btl, 2048 * k), kb, id3, 1);
                umma_bf16(tm + C::D4, desc_add(at, 2048 * k), qb, id3, 1);
                umma_bf16(tm + C::D4, desc_add(atl, 2048 * k), qb, id3, 1);
            }
            umma_commit(&B.d4);
            return true;
        };
        for_units(p, lane, [&](const Unit&) {
            bool ok = true;
            for (int j = 0; j < group && ok; ++j, ++step) {
                if (lane == 0) {
                    ok = step == 0 || mbar_wait(&B.read, (step - 1) & 1, ctl);
                    const uint32_t d1 = tm + C::D1 + 64 * (step & 1);
                    for (int s = 0; s < ns && ok; ++s, ++n) {
                        const int st = n % kStages, left = p.dv - s * kCols;
                        ok = mbar_wait(&B.full[st], (n / kStages) & 1, ctl);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t at = smem_u32(smem + st * M::STAGE);
                        const uint64_t xy = smem_desc(at + M::X, 16, 1024, kLayoutSW128);
                        const uint64_t v = smem_desc(at + M::V, kPieceBytes, 256, kLayoutSW32);
                        const uint64_t vm = smem_desc(at + M::V - M::VB / 2, kPieceBytes, 256, kLayoutSW32);
                        const uint64_t sd = smem_desc(at + M::S, kPieceBytes, 256, kLayoutSW32);
                        const uint64_t ed = smem_desc(at + M::E, kPieceBytes, 256, kLayoutSW32);
                        const uint32_t on = s > 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (k >= 2 && left == 32) break;
                            const uint32_t vo = (k >> 1) * M::VB + (k & 1) * 512, so = (k >> 1) * M::SB + (k & 1) * 512;
                            const uint32_t acc = k > 0 ? 1 : on;
                            const uint64_t a = desc_add(xy, 32 * k);
                            umma_bf16(d1, a, desc_add(v, vo), id1, acc);
                            umma_bf16(d1, a, desc_add(v, vo + M::VB / 2), id1, 1);
                            umma_bf16(tm + C::D2, a, desc_add(sd, so), id2, acc);
                            umma_bf16(tm + C::D3, desc_add(vm, vo), desc_add(ed, so), id3, acc);
                            umma_bf16(tm + C::D3, desc_add(vm, vo + M::VB / 2), desc_add(ed, so), id3, 1);
                        }
                        umma_commit(&B.empty[st]);
                        // while the workers get to this unit: the last product of the one before
                        if (s == 0 && step > 0) ok = last_product(step - 1);
                    }
                    if (ok) umma_commit(&B.d123);
                }
                ok = __shfl_sync(0xFFFFFFFFu, static_cast<int>(ok), 0) != 0;
            }
            return ok;
        });
        if (lane == 0) {
            if (step > 0) last_product(step - 1);
            umma_commit(&B.drain);
            mbar_wait(&B.drain, 0, ctl);
        }
        __syncwarp();
    } else if (warp == kGdWorkers + 2) {
        // ---- da and dbeta
        for_units(p, lane, [&](const Unit& x) {
            for (int j = 0; j < group; ++j) sums<DK>(p, x, x.hk * group + j, lane);
            return true;
        });
    } else {
        // ---- workers: lane = token of dq or of dk, half of the columns
        const int half = warp >> 2, i = (warp & 1) * 32 + lane;
        const bool is_k = (warp & 2) != 0;
        const uint32_t t0 = tm + (static_cast<uint32_t>(warp & 3) << 21);
        constexpr int HS = DK / 2;
        [[maybe_unused]] const int64_t rows = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;
        int step = 0;
        for_units(p, lane, [&](const Unit& x) {
            float acc[HS];
#pragma unroll
            for (int e = 0; e < HS; ++e) acc[e] = 0.f;
            for (int j = 0; j < group; ++j, ++step) {
                const float* own = reinterpret_cast<const float*>(p.rec + (x.slot * H + x.hk * group + j) * Rec::BYTES + Rec::SC) + i;
                const float g = own[kScG * kGdC], f2 = is_k ? -g : p.scale * g, f3 = own[kScR * kGdC];
                if (!warp_wait(&B.d123, step & 1, ctl)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < HS / 16; ++k) {
                    uint32_t d[16], e[16];
                    tmem_ld16(t0 + C::D2 + half * HS + 16 * k, d);
                    if (is_k) tmem_ld16(t0 + C::D3 + half * HS + 16 * k, e);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        acc[16 * k + t] = fmaf(f2, __uint_as_float(d[t]), acc[16 * k + t]);
                        if (is_k) acc[16 * k + t] = fmaf(f3, __uint_as_float(e[t]), acc[16 * k + t]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.read);
                if (!warp_wait(&B.sc[step & 1], (step >> 1) & 1, ctl)) return false;
                // A or B, 16 columns at a time: up to the diagonal, in the sequence
                // (a loop: a first pass waits for every line of its code)
                {
                    const float* sc = reinterpret_cast<const float*>(smem + M::SC + (step & 1) * M::SCB);     // b, high and low
                    const float bh = sc[i], bl = sc[kGdC + i], f = is_k ? -1.f : p.scale;
                    const int end = i >= x.valid ? 0 : i + !is_k;                 // columns of this row
                    unsigned char* tile = smem + M::A + (is_k ? 8192 : 0);
#pragma unroll 1
                    for (int c = 2 * half; c < 2 * half + 2; ++c) {
                        uint32_t w[8], l[8];
                        if (16 * c > (warp & 1) * 32 + 31) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = l[e] = 0u;
                        } else {
                            uint32_t d[16];
                            tmem_ld16(t0 + C::D1 + 64 * (step & 1) + 16 * c, d);
                            float m[16];
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const float4 jh = *reinterpret_cast<const float4*>(sc + 16 * c + e);
                                const float4 jl = *reinterpret_cast<const float4*>(sc + kGdC + 16 * c + e);
                                m[e] = f * gd_exp2((bh - jh.x) + (bl - jl.x));
                                m[e + 1] = f * gd_exp2((bh - jh.y) + (bl - jl.y));
                                m[e + 2] = f * gd_exp2((bh - jh.z) + (bl - jl.z));
                                m[e + 3] = f * gd_exp2((bh - jh.w) + (bl - jl.w));
                            }
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                m[e] *= __uint_as_float(d[e]);
                                if (16 * c + e >= end) m[e] = 0.f;
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                w[e] = pack_bf16(m[2 * e], m[2 * e + 1]);
                                l[e] = pack_bf16(m[2 * e] - bf16_lo(w[e]), m[2 * e + 1] - bf16_hi(w[e]));
                            }
                        }
                        *reinterpret_cast<uint4*>(tile + swz_off(i, 2 * c, 128)) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(tile + swz_off(i, 2 * c + 1, 128)) = make_uint4(w[4], w[5], w[6], w[7]);
                        *reinterpret_cast<uint4*>(tile + M::AB + swz_off(i, 2 * c, 128)) = make_uint4(l[0], l[1], l[2], l[3]);
                        *reinterpret_cast<uint4*>(tile + M::AB + swz_off(i, 2 * c + 1, 128)) = make_uint4(l[4], l[5], l[6], l[7]);
                    }
                }
                if (x.valid < kGdC && (warp & 3) == 0) {
                    // rows of Q behind the sequence's end are another's: zeros times them need not be zeros
                    if (!warp_wait(&B.kq, step & 1, ctl)) return false;
                    for (int r = x.valid + half; r < kGdC; r += 2)
                        for (int b = lane; b < DK / 8; b += 32)
                            *reinterpret_cast<uint4*>(smem + M::Q + (b >> 2) * 4096 + r * 64 + (b & 3) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&B.w);
                    mbar_arrive(&B.sc_done[step & 1]);
                }
                if (!warp_wait(&B.d4, step & 1, ctl)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < HS / 16; ++k) {
                    uint32_t d[16];
                    tmem_ld16(t0 + C::D4 + half * HS + 16 * k, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 16; ++t) acc[16 * k + t] += __uint_as_float(d[t]);
                }
                if (j + 1 == group) {
                    // out: through K's and Q's place where the chunk is whole
                    unsigned char* tile = smem + (is_k ? M::K : M::Q);
                    __nv_bfloat16* out = is_k ? p.dkk : p.dq;
                    const int64_t at = (static_cast<int64_t>(x.row) + i) * p.seqs.Hk * DK + x.hk * DK + half * HS;
#pragma unroll
                    for (int e = 0; e < HS; e += 8) {
                        uint4 w;
                        w.x = pack_bf16(acc[e], acc[e + 1]);
                        w.y = pack_bf16(acc[e + 2], acc[e + 3]);
                        w.z = pack_bf16(acc[e + 4], acc[e + 5]);
                        w.w = pack_bf16(acc[e + 6], acc[e + 7]);
                        const int k = (half * HS + e) >> 3;
                        if (x.valid == kGdC) *reinterpret_cast<uint4*>(tile + (k >> 2) * 4096 + swz_off(i, k & 3, 64)) = w;
                        else if (i < x.valid && GLA_DCHECK(x.row + i < rows, p.status)) *reinterpret_cast<uint4*>(out + at + e) = w;
                    }
                    fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.kq_done);
            }
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kGdWorkers + 1) tmem_dealloc(tm, C::ALLOC);
}

template <int DK>
gla_status launch(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    const int64_t tokens = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;
    const int64_t wv = static_cast<int64_t>(p.seqs.H) * p.dv, wk = static_cast<int64_t>(p.seqs.Hk) * DK;
    auto map = [&](CUtensorMap* m, const void* base, int64_t width, int64_t ld, int box, int swizzle) {
        return gd_block_map(m, base, width, ld, tokens, box, swizzle);
    };
    Maps maps;
    gla_status s;
    if ((s = map(&maps.dO, p.dO, wv, p.ld_do, kCols, 128)) != GLA_OK || (s = map(&maps.dv, p.dvv, wv, wv, kCols, 128)) != GLA_OK ||
        (s = map(&maps.q, p.q, wk, p.ld_qk, 32, 64)) != GLA_OK || (s = map(&maps.dq, p.dq, wk, wk, 32, 64)) != GLA_OK ||
        (s = map(&maps.dk, p.dkk, wk, wk, 32, 64)) != GLA_OK)
        return s;
    constexpr int smem = Smem<DK>::bytes;
    cudaError_t e = cudaFuncSetAttribute(gd_grad_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return status_of(e);
    const int64_t units = p.slots * p.seqs.Hk;
    trace_begin(st);
    gd_grad_kernel<DK><<<static_cast<unsigned>(units < kSms ? units : kSms), kThreads, smem, st>>>(p, maps, ctl);
    trace_end(st, "gd_grad_kernel");
    count_launch();
    return check_launch("gd_grad_kernel");
}

}  // namespace

gla_status gd_launch_grad(const GdParams& p, const WaitCtl& ctl, cudaStream_t st)
{
    if (p.slots == 0) return GLA_OK;
    switch (p.dk) {
    case 64: return launch<64>(p, ctl, st);
    case 96: return launch<96>(p, ctl, st);
    default: return launch<128>(p, ctl, st);
    }
}

}  // namespace gla
