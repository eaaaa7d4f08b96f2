// gated_delta_host.cu -- the C entry points of the gated delta rule and of the
// group norm with an activation: argument checks, workspace layout, dispatch.
// As everywhere in this library nothing is allocated and nothing waits.
#include <cmath>

#include "gated_delta.cuh"

namespace gla {

gla_status gd_launch_step(float* state, const int32_t* slot_idx, int n_slots, const void* q, const void* k,
                          const void* v, const float* a, const float* beta, float* o, int N, int T, int Hk, int H,
                          int dk, int dv, int64_t ld_qk, int64_t ld_v, float scale, bool f32, int* status,
                          cudaStream_t st);
size_t group_norm_bwd_workspace_bytes(int M, int G, int d);
gla_status launch_group_norm(const void* x, bool f32, const void* gate, const float* weight, const float* bias, void* y,
                             int M, int G, int d, int64_t ld_x, int64_t ld_gate, bool shared_w, bool center, bool act,
                             float eps, cudaStream_t st);
gla_status launch_group_norm_bwd(const void* x, bool f32, const void* gate, const float* weight, const float* bias,
                                 const void* dy, void* dx, void* dgate, float* dweight, float* dbias, float* ws, int M,
                                 int G, int d, int64_t ld_x, int64_t ld_gate, bool shared_w, bool center, bool act,
                                 float eps, cudaStream_t st);

namespace {

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool gd_dims_ok(int dk, int dv)
{
    return (dk == 64 || dk == 96 || dk == 128) && dv >= 32 && dv <= 256 && dv % 32 == 0;
}

// Sizes, head layout and token strides shared by the chunked calls and the step.
gla_status gd_check(int N, int T, int Hk, int H, int dk, int dv, int64_t ld_qkv, int esz, float scale, bool packed,
                    int64_t* ld_qk, int64_t* ld_v)
{
    if (N < 0 || T < 0 || H < 0 || Hk < 0 || dk <= 0 || dv <= 0 || ld_qkv < 0) return GLA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return GLA_ERR_INVALID_ARG;
    if (H > 0 && (Hk == 0 || H % Hk != 0)) return GLA_ERR_INVALID_ARG;
    if (!gd_dims_ok(dk, dv)) return GLA_ERR_UNSUPPORTED;
    if (H > 65535 || static_cast<int64_t>(N) * H > 0x3FFFFFFF) return GLA_ERR_UNSUPPORTED;
    const int64_t pq = static_cast<int64_t>(Hk) * dk, pv = static_cast<int64_t>(H) * dv;
    if (ld_qkv == 0) {
        *ld_qk = pq;
        *ld_v = pv;
    } else {
        if (ld_qkv < pq || ld_qkv < pv) return GLA_ERR_INVALID_ARG;
        if ((ld_qkv * esz) % 16 != 0) return GLA_ERR_MISALIGNED;
        *ld_qk = *ld_v = ld_qkv;
    }
    const int64_t rows = packed ? T : static_cast<int64_t>(N) * T;
    const int64_t widest = *ld_qk > *ld_v ? *ld_qk : *ld_v;
    if (widest > 0 && rows > (int64_t(1) << 40) / widest) return GLA_ERR_UNSUPPORTED;
    if (rows > 0x7FFFFFFF || gd_slots(packed, N, T) > 0x7FFFFFFF) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

// Segments of long sequences: as many as fill the SMs once (two CTAs each in
// the forward up to dk = 96, else one), where one CTA an SM leaves room for three
// (a pass over them costs about what the sweep does, so two would gain nothing).
// And no more than 2 sqrt(chunks) backward, sqrt(2 chunks) forward: the hand-over
// takes some 2 us a segment, passes and sweeps 15 and 6.5 a chunk (4 heads of 96 x
// 192, forward: 16,384 tokens in 37 segments 219 us, in 22 200; 4,096 tokens of 8
// heads in 14 132 us, in 11 122).  One piece against segments: 768 tokens of 8 heads
// of 96 x 192 backward 136 and 111 us, 1,024 tokens of 8 heads of 64 x 64 151 and
// 93, forward 60 and 47; but 4,096 tokens of two sequences of 16 heads of 96 x 192
// forward 257 and 270.  Below 12 chunks both happen backward, by the number of
// segments that fit: 640 tokens of 16 heads of 96 x 192 (four) 129 and 146, 555
// tokens of two sequences of 8 heads of 128 x 128 (nine) 142 and 129; forward, 500
// tokens of 8 heads of 96 x 192, 39 and 42.  The backward's have an even number of
// chunks: it keeps the state after every second one.
void gd_segments(GdParams& p, bool bwd)
{
    constexpr int64_t kSms = 148;
    const int64_t chunks = (static_cast<int64_t>(p.seqs.T) + kGdC - 1) / kGdC;
    const int64_t ctas = static_cast<int64_t>(p.seqs.N) * p.seqs.H * ((p.dv + 127) / 128);
    int64_t n = 1;
    if (ctas > 0 && 3 * ctas <= kSms && chunks >= 12) {
        n = kSms * (p.dk <= 96 && !bwd ? 2 : 1) / ctas;
        while (n * n > (bwd ? 4 : 2) * chunks) --n;
    }
    int64_t c = (chunks + n - 1) / n;
    if (bwd && n > 1) c += c & 1;
    if (c < 1) c = 1;
    p.seg_chunks = static_cast<int>(c);
    p.nseg = static_cast<int>(chunks > c ? (chunks + c - 1) / c : 1);
}

// The workspace: parts one behind the other, 256-byte aligned.  With base
// null only the size is found.
size_t gd_layout(GdParams& p, bool bwd, unsigned char* base)
{
    const size_t u = static_cast<size_t>(p.slots) * p.seqs.H, dk = p.dk, dv = p.dv;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* q = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    p.rec = take(u * gd_rec_bytes(p.dk, bwd));
    gd_segments(p, bwd);
    const size_t segs = p.nseg > 1 ? static_cast<size_t>(p.seqs.N) * p.seqs.H * p.nseg : 0;
    p.seg_l = reinterpret_cast<float*>(take(segs * dk * dv * 4));
    p.seg_a = reinterpret_cast<float*>(take(segs * dk * dk * 4));
    if (bwd) p.seg_e = reinterpret_cast<float*>(take(segs * dk * dv * 4));
    if (bwd) {
        p.sb = reinterpret_cast<__nv_bfloat16*>(take(u * dk * dv * 2));
        p.eb = reinterpret_cast<__nv_bfloat16*>(take(u * dk * dv * 2));
        p.sn = reinterpret_cast<float*>(take(u * dk * dv * 4));
        p.sn_last = reinterpret_cast<float*>(take(static_cast<size_t>(p.seqs.N) * p.seqs.H * dk * dv * 4));
        p.yn = reinterpret_cast<float*>(take(u * kGdC * dv * 4));
        p.vp = reinterpret_cast<__nv_bfloat16*>(take(u * 2 * kGdC * dv * 2));
        p.part = reinterpret_cast<float*>(take(u * 3 * (dv / 32) * kGdC * 4));
        p.anch = reinterpret_cast<float*>(take(u * (dv / 32) * 2 * 4));
    }
    return at;
}

GdParams gd_params(const void* q, const void* k, const void* v, const float* a, const float* beta,
                   const int32_t* cu_seqlens, const float* s0, int N, int T, int Hk, int H, int dk, int dv,
                   int64_t ld_qk, int64_t ld_v, float scale)
{
    GdParams p{};
    p.seqs = GdSeqs{cu_seqlens, N, T, H, Hk};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.a = a;
    p.beta = beta;
    p.s0 = s0;
    p.ld_qk = ld_qk;
    p.ld_v = ld_v;
    p.ld_do = static_cast<int64_t>(H) * dv;
    p.dk = dk;
    p.dv = dv;
    p.scale = scale;
    p.slots = gd_slots(cu_seqlens != nullptr, N, T);
    return p;
}

// The checking build's scan of the inputs (nothing in the normal build).  f32: the
// type of q, k and v; pool: the step's states.
gla_status gd_scan(const GdParams& p, cudaStream_t st, bool f32 = false, const float* pool = nullptr,
                   const int32_t* slot_idx = nullptr, int n_slots = 0)
{
    DebugScan d;
    const int64_t rows = p.seqs.cu ? p.seqs.T : static_cast<int64_t>(p.seqs.N) * p.seqs.T;
    const int64_t wq = static_cast<int64_t>(p.seqs.Hk) * p.dk, wv = static_cast<int64_t>(p.seqs.H) * p.dv;
    d.cu = p.seqs.cu;
    d.n_seq = p.seqs.N;
    d.heads = p.seqs.H;
    d.a = p.a;
    d.na = rows * p.seqs.H;
    DebugScan::Rows* qkv = f32 ? d.tokens_f32 + 1 : d.bf16;
    qkv[0] = {p.q, rows, p.ld_qk, wq};
    qkv[1] = {p.k, rows, p.ld_qk, wq};
    qkv[2] = {p.v, rows, p.ld_v, wv};
    d.bf16[3] = {p.dO, rows, p.ld_do, wv};
    d.tokens_f32[0] = {p.beta, rows, p.seqs.H, p.seqs.H};
    const int64_t per = static_cast<int64_t>(p.seqs.H) * p.dk * p.dv, ns = p.seqs.N * per;
    d.f32[0] = p.s0;
    d.nf32[0] = p.s0 ? ns : 0;
    d.f32[1] = p.ds_final;
    d.nf32[1] = p.ds_final ? ns : 0;
    d.pool = pool;
    d.slot_idx = slot_idx;
    d.n = p.seqs.N;
    d.n_slots = n_slots;
    d.per_slot = per;
    return debug_scan(d, p.status, st);
}

gla_status norm_check(const void* x, gla_dtype dt, const void* gate, const float* weight, const float* bias, int M,
                      int G, int d, int64_t* ld_x, int64_t* ld_gate, float eps)
{
    if (M < 0 || G < 0 || d <= 0 || *ld_x < 0 || *ld_gate < 0) return GLA_ERR_INVALID_ARG;
    if (dt != GLA_BF16 && dt != GLA_F32) return GLA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return GLA_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > 1024 || static_cast<int64_t>(G) * d > (1 << 20)) return GLA_ERR_UNSUPPORTED;
    const int64_t C = static_cast<int64_t>(G) * d;
    if (*ld_x == 0) *ld_x = C;
    if (*ld_gate == 0) *ld_gate = C;
    if (*ld_x < C || *ld_gate < C) return GLA_ERR_INVALID_ARG;
    if (*ld_x % (dt == GLA_F32 ? 4 : 8) != 0 || *ld_gate % 8 != 0) return GLA_ERR_MISALIGNED;
    if (!a16(weight) || !a16(bias)) return GLA_ERR_MISALIGNED;
    if (M > 0 && G > 0 && !x) return GLA_ERR_INVALID_ARG;
    if (!a16(x) || !a16(gate)) return GLA_ERR_MISALIGNED;
    return GLA_OK;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gated_delta_chunk_workspace_bytes(int N, int T, int H, int dk, int dv, int packed, int for_bwd)
{
    if (N <= 0 || T <= 0 || H <= 0 || !gd_dims_ok(dk, dv)) return 0;
    GdParams p{};
    p.seqs = GdSeqs{nullptr, N, T, H, H};
    p.dk = dk;
    p.dv = dv;
    p.slots = gd_slots(packed != 0, N, T);
    return gd_layout(p, for_bwd != 0, nullptr);
}

gla_status gated_delta_chunk_fwd(const void* q, const void* k, const void* v, const float* a, const float* beta,
                                 const int32_t* cu_seqlens, const float* s0, void* o, float* s_final, void* ws,
                                 size_t ws_bytes, int N, int T, int Hk, int H, int dk, int dv, int64_t ld_qkv,
                                 float scale, gla_dtype dt, cudaStream_t stream)
{
    int64_t ld_qk, ld_v;
    if (dt != GLA_BF16 && dt != GLA_F32) return GLA_ERR_INVALID_ARG;
    gla_status s = gd_check(N, T, Hk, H, dk, dv, ld_qkv, 2, scale, cu_seqlens != nullptr, &ld_qk, &ld_v);
    if (s != GLA_OK) return s;
    if (dt != GLA_BF16) return GLA_ERR_UNSUPPORTED;
    if (N == 0 || H == 0) return GLA_OK;
    if (T > 0 && (!q || !k || !v || !a || !beta || !o)) return GLA_ERR_INVALID_ARG;
    if (!a16(q) || !a16(k) || !a16(v) || !a16(a) || !a16(beta) || !a16(cu_seqlens) || !a16(s0) || !a16(o) ||
        !a16(s_final) || !a16(ws))
        return GLA_ERR_MISALIGNED;
    GdParams p = gd_params(q, k, v, a, beta, cu_seqlens, s0, N, T, Hk, H, dk, dv, ld_qk, ld_v, scale);
    if (T == 0) p.slots = 0;
    if (T > 0 && (!ws || ws_bytes < gd_layout(p, false, nullptr))) return GLA_ERR_INVALID_ARG;
    const WaitCtl ctl = wait_ctl_for_current_device(&s);
    if (s != GLA_OK) return s;
    p.status = ctl.status;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.s_final = s_final;
    gd_layout(p, false, static_cast<unsigned char*>(ws));
    if (T > 0 && (s = gd_scan(p, stream)) != GLA_OK) return s;
    if ((s = gd_launch_chunks(p, false, stream)) != GLA_OK) return s;
    return gd_launch_sweep_fwd(p, ctl, stream);
}

gla_status gated_delta_chunk_bwd(const void* q, const void* k, const void* v, const float* a, const float* beta,
                                 const int32_t* cu_seqlens, const float* s0, const void* dO, const float* ds_final,
                                 void* grad_q, void* grad_k, void* grad_v, float* grad_a, float* grad_beta,
                                 float* grad_s0, void* ws, size_t ws_bytes, int N, int T, int Hk, int H, int dk,
                                 int dv, int64_t ld_qkv, float scale, gla_dtype dt, cudaStream_t stream)
{
    int64_t ld_qk, ld_v;
    if (dt != GLA_BF16 && dt != GLA_F32) return GLA_ERR_INVALID_ARG;
    gla_status s = gd_check(N, T, Hk, H, dk, dv, ld_qkv, 2, scale, cu_seqlens != nullptr, &ld_qk, &ld_v);
    if (s != GLA_OK) return s;
    if (dt != GLA_BF16) return GLA_ERR_UNSUPPORTED;
    if (N == 0 || H == 0) return GLA_OK;
    if (T > 0 && (!q || !k || !v || !a || !beta || !dO || !grad_q || !grad_k || !grad_v || !grad_a || !grad_beta))
        return GLA_ERR_INVALID_ARG;
    if (!a16(q) || !a16(k) || !a16(v) || !a16(a) || !a16(beta) || !a16(cu_seqlens) || !a16(s0) || !a16(dO) ||
        !a16(ds_final) || !a16(grad_q) || !a16(grad_k) || !a16(grad_v) || !a16(grad_a) || !a16(grad_beta) ||
        !a16(grad_s0) || !a16(ws))
        return GLA_ERR_MISALIGNED;
    GdParams p = gd_params(q, k, v, a, beta, cu_seqlens, s0, N, T, Hk, H, dk, dv, ld_qk, ld_v, scale);
    if (T == 0) {
        // no token: the gradient of the state passes through
        if (!grad_s0) return GLA_OK;
        const size_t bytes = static_cast<size_t>(N) * H * dk * dv * sizeof(float);
        return status_of(ds_final ? cudaMemcpyAsync(grad_s0, ds_final, bytes, cudaMemcpyDeviceToDevice, stream)
                                  : cudaMemsetAsync(grad_s0, 0, bytes, stream));
    }
    if (!ws || ws_bytes < gd_layout(p, true, nullptr)) return GLA_ERR_INVALID_ARG;
    const WaitCtl ctl = wait_ctl_for_current_device(&s);
    if (s != GLA_OK) return s;
    p.status = ctl.status;
    p.dO = static_cast<const __nv_bfloat16*>(dO);
    p.ds_final = ds_final;
    p.dq = static_cast<__nv_bfloat16*>(grad_q);
    p.dkk = static_cast<__nv_bfloat16*>(grad_k);
    p.dvv = static_cast<__nv_bfloat16*>(grad_v);
    p.da = grad_a;
    p.dbeta = grad_beta;
    p.ds0 = grad_s0;
    gd_layout(p, true, static_cast<unsigned char*>(ws));
    if ((s = gd_scan(p, stream)) != GLA_OK) return s;
    if ((s = gd_launch_chunks(p, true, stream)) != GLA_OK) return s;
    if (p.nseg > 1 && (s = gd_launch_segment_states(p, ctl, stream)) != GLA_OK) return s;
    if ((s = gd_launch_sweeps_bwd(p, ctl, stream)) != GLA_OK) return s;
    return gd_launch_grad(p, ctl, stream);
}

gla_status gated_delta_decode_step(float* state, const int32_t* slot_idx, int n_slots, const void* q, const void* k,
                                   const void* v, const float* a, const float* beta, float* o, int N, int T, int Hk,
                                   int H, int dk, int dv, int64_t ld_qkv, float scale, gla_dtype dt,
                                   cudaStream_t stream)
{
    int64_t ld_qk, ld_v;
    if (dt != GLA_BF16 && dt != GLA_F32) return GLA_ERR_INVALID_ARG;
    const bool f32 = dt == GLA_F32;
    gla_status s = gd_check(N, T, Hk, H, dk, dv, ld_qkv, f32 ? 4 : 2, scale, false, &ld_qk, &ld_v);
    if (s != GLA_OK) return s;
    if (n_slots < 0 || (!slot_idx && n_slots < N)) return GLA_ERR_INVALID_ARG;
    if (N == 0 || H == 0 || T == 0) return GLA_OK;
    if (!state || !q || !k || !v || !a || !beta || !o) return GLA_ERR_INVALID_ARG;
    if (!a16(state) || !a16(slot_idx) || !a16(q) || !a16(k) || !a16(v) || !a16(a) || !a16(beta) || !a16(o))
        return GLA_ERR_MISALIGNED;
    const WaitCtl ctl = wait_ctl_for_current_device(&s);
    if (s != GLA_OK) return s;
    GdParams p = gd_params(q, k, v, a, beta, nullptr, nullptr, N, T, Hk, H, dk, dv, ld_qk, ld_v, scale);
    p.status = ctl.status;
    if ((s = gd_scan(p, stream, f32, state, slot_idx, n_slots)) != GLA_OK) return s;
    return gd_launch_step(state, slot_idx, n_slots, q, k, v, a, beta, o, N, T, Hk, H, dk, dv, ld_qk, ld_v, scale, f32,
                          ctl.status, stream);
}

size_t group_norm_silu_bwd_workspace_bytes(int M, int G, int d)
{
    if (M <= 0 || G <= 0 || d <= 0 || d % 8 != 0 || d > 1024 || static_cast<int64_t>(G) * d > (1 << 20)) return 0;
    return group_norm_bwd_workspace_bytes(M, G, d);
}

gla_status group_norm_silu(const void* x, const void* gate, const float* weight, const float* bias, void* y, int M,
                           int G, int d, int64_t ld_x, int64_t ld_gate, int shared_weight, int center, int act,
                           float eps, gla_dtype dt, cudaStream_t stream)
{
    gla_status s = norm_check(x, dt, gate, weight, bias, M, G, d, &ld_x, &ld_gate, eps);
    if (s != GLA_OK) return s;
    if (M == 0 || G == 0) return GLA_OK;
    if (!y) return GLA_ERR_INVALID_ARG;
    if (!a16(y)) return GLA_ERR_MISALIGNED;
    return launch_group_norm(x, dt == GLA_F32, gate, weight, bias, y, M, G, d, ld_x, ld_gate, shared_weight != 0,
                             center != 0, act != 0, eps, stream);
}

gla_status group_norm_silu_bwd(const void* x, const void* gate, const float* weight, const float* bias, const void* dy,
                               void* grad_x, void* grad_gate, float* grad_weight, float* grad_bias, void* ws,
                               size_t ws_bytes, int M, int G, int d, int64_t ld_x, int64_t ld_gate, int shared_weight,
                               int center, int act, float eps, gla_dtype dt, cudaStream_t stream)
{
    gla_status s = norm_check(x, dt, gate, weight, bias, M, G, d, &ld_x, &ld_gate, eps);
    if (s != GLA_OK) return s;
    if (G == 0) M = 0;                          // no group: the gradients of shared parameters are zeros
    if (M > 0 && (!dy || !grad_x || (gate && !grad_gate))) return GLA_ERR_INVALID_ARG;
    if (!a16(dy) || !a16(grad_x) || !a16(grad_gate) || !a16(grad_weight) || !a16(grad_bias) || !a16(ws))
        return GLA_ERR_MISALIGNED;
    if (M > 0 && (grad_weight || grad_bias) && (!ws || ws_bytes < group_norm_silu_bwd_workspace_bytes(M, G, d)))
        return GLA_ERR_INVALID_ARG;
    return launch_group_norm_bwd(x, dt == GLA_F32, gate, weight, bias, dy, grad_x, grad_gate, grad_weight, grad_bias,
                                 static_cast<float*>(ws), M, G, d, ld_x, ld_gate, shared_weight != 0, center != 0,
                                 act != 0, eps, stream);
}

}  // extern "C"
