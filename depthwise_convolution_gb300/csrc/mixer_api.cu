// C ABI of the token mixer: argument validation and kernel selection for the
// causal convolution, the block norms and the gated delta rule.  As in
// dwconv_api.cu, every argument is checked on the host before the CUDA runtime
// is touched.
#include <cmath>

#include "delta_chunk_host.cuh"

namespace dwc {

namespace {

bool float_dtype(dwconv_dtype dt) { return dt == DWCONV_FP32 || dt == DWCONV_FP16 || dt == DWCONV_BF16; }
dwconv_status check_dtype(dwconv_dtype dt) {
    if (float_dtype(dt)) return DWCONV_OK;
    return dt >= DWCONV_INT8 && dt <= DWCONV_FP8_E4M3 ? DWCONV_ERR_UNSUPPORTED : DWCONV_ERR_INVALID_ARG;
}
size_t float_size(dwconv_dtype dt) { return dt == DWCONV_FP32 ? 4 : 2; }

bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
dwconv_status cuda_to_status(cudaError_t e) {
    return e == cudaSuccess ? DWCONV_OK : e == cudaErrorNotSupported ? DWCONV_ERR_UNSUPPORTED : DWCONV_ERR_CUDA;
}

constexpr int kMaxRows = 65535;      // rows of a batch (a grid dimension)
constexpr int kMaxTokens = 1 << 24;  // tokens of a sequence
constexpr int kMaxWidth = 1 << 20;   // channels
constexpr int kMaxTaps = 8;

dwconv_status check_causal(int B, int T, int C, int W, dwconv_dtype dtype, dwconv_activation act) {
    const dwconv_status st = check_dtype(dtype);
    if (st != DWCONV_OK) return st;
    if (B < 0 || T < 0 || C <= 0 || W <= 0 || B > kMaxRows || T > kMaxTokens || C > kMaxWidth || W > kMaxTaps)
        return DWCONV_ERR_INVALID_ARG;
    if (act < DWCONV_ACT_NONE || act > DWCONV_ACT_GELU) return DWCONV_ERR_INVALID_ARG;
    return act == DWCONV_ACT_NONE || act == DWCONV_ACT_SILU ? DWCONV_OK : DWCONV_ERR_UNSUPPORTED;
}

dwconv_status check_norm(long long rows_outer, int rows_inner, int C, dwconv_dtype dtype, dwconv_norm norm,
                         dwconv_gate gate_act, float eps) {
    const dwconv_status st = check_dtype(dtype);
    if (st != DWCONV_OK) return st;
    if (rows_outer < 0 || rows_inner <= 0 || C <= 0 || C > kMaxNormWidth || rows_outer > (1LL << 40) / rows_inner / C)
        return DWCONV_ERR_INVALID_ARG;
    if (norm != DWCONV_NORM_RMS && norm != DWCONV_NORM_LAYER) return DWCONV_ERR_INVALID_ARG;
    if (gate_act < DWCONV_GATE_NONE || gate_act > DWCONV_GATE_SIGMOID) return DWCONV_ERR_INVALID_ARG;
    return eps >= 0.f && std::isfinite(eps) ? DWCONV_OK : DWCONV_ERR_INVALID_ARG;
}

dwconv_status check_delta(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype, dwconv_dtype gate_dtype,
                          float scale) {
    const dwconv_status st = check_dtype(dtype);
    if (st != DWCONV_OK) return st;
    if (gate_dtype != dtype && gate_dtype != DWCONV_FP32) return DWCONV_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || Hk <= 0 || Hv <= 0 || K <= 0 || V <= 0 || B > kMaxRows || T > kMaxTokens ||
        Hv > kMaxRows || V > kMaxWidth || Hv % Hk)
        return DWCONV_ERR_INVALID_ARG;
    if (K > kDeltaMaxK) return DWCONV_ERR_UNSUPPORTED;
    if ((long long)B * T > (1LL << 40) / Hv / (K > V ? K : V)) return DWCONV_ERR_INVALID_ARG;
    return std::isfinite(scale) ? DWCONV_OK : DWCONV_ERR_INVALID_ARG;
}

// Strides must not be negative; returns false on one that is.
bool good_strides(const long long *s, int n) {
    for (int i = 0; s && i < n; ++i)
        if (s[i] < 0) return false;
    return true;
}

// Whether two buffers of `bytes` bytes share one.
bool overlap(const void *p, const void *q, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && (a < b ? b - a : a - b) < bytes;
}

struct Sized {
    const void *p;
    size_t size;
};
bool all_aligned(std::initializer_list<Sized> ps) {
    for (const Sized &s : ps)
        if (!aligned_to(s.p, s.size)) return false;
    return true;
}

// Argument block of a sequence pass; strides of q, k, v, g, beta in threes (or dense).
DeltaArgs delta_args(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype, dwconv_dtype gate_dtype,
                     const void *q, const void *k, const void *v, const void *g, const void *beta,
                     const long long *strides, float scale, int qk_norm) {
    DeltaArgs a{};
    a.B = B; a.T = T; a.Hk = Hk; a.Hv = Hv; a.K = K; a.V = V;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    const long long dense[15] = {(long long)T * Hk * K, (long long)Hk * K, K, (long long)T * Hk * K,
                                 (long long)Hk * K,     K,                 (long long)T * Hv * V, (long long)Hv * V,
                                 V,                     (long long)T * Hv, Hv, 1, (long long)T * Hv, Hv, 1};
    const long long *s = strides ? strides : dense;
    long long *to[5] = {a.q_s, a.k_s, a.v_s, a.g_s, a.b_s};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < 3; ++j) to[i][j] = s[3 * i + j];
    a.gate_f32 = gate_dtype == DWCONV_FP32;
    a.scale = scale;
    a.qk_norm = qk_norm != 0;
    a.N = B;
    return a;
}

// The chunked kernels take K <= 128; up to kShort tokens the token-by-token
// kernel is faster than a padded chunk (two launches).  K = V = 128, bf16, 32 x 16
// heads: 8 tokens 60 us against 79, 16 tokens 104 against 81, 64 tokens 376
// against 85; one row of 8 heads, K = V = 64: 15.5 against 17.5, 24 against 20,
// 77 against 20.
constexpr int kShort = 10;
bool chunked(int T, int K) { return K <= chunk::kMaxK && T > kShort; }

// Buffers of the chunked kernels, laid out one behind the other (every part a
// multiple of 512 bytes): what is prepared, what the forward walk saves for the
// backward pass, what the backward walk leaves.
struct ChunkSizes {
    size_t kq16, mp16, vec16, kq, mp, vec, s, u, f, d_o, totals;
    size_t prepared() const { return kq16 + mp16 + vec16; }
    size_t saved() const { return prepared() + kq + mp + vec + s + u; }
    size_t walked() const { return s + f + d_o + totals; }
};
ChunkSizes chunk_sizes(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype) {
    const size_t n = (T + chunk::kC - 1) / chunk::kC, kd = K <= 64 ? 64 : 128, nt = dtype == DWCONV_BF16 ? 1 : 2;
    const size_t v16 = (size_t)(V + 15) / 16 * 16, vc = (size_t)B * Hv * n, kc = (size_t)B * Hk * n;
    ChunkSizes z;
    z.kq16 = kc * 2 * (dtype == DWCONV_FP32 ? 2 : 1) * chunk::kC * kd * 2;
    z.mp16 = vc * chunk::kMpElems * 2;
    z.vec16 = vc * chunk::kVec16Elems * 4;
    z.kq = kc * 2 * nt * chunk::kC * kd * 2;
    z.mp = vc * chunk::kMpElems * 2;
    z.vec = vc * chunk::kVecElems * 4;
    z.s = vc * nt * v16 * kd * 2;
    z.u = z.f = vc * 2 * v16 * chunk::kC * 2;
    z.d_o = vc * nt * v16 * chunk::kC * 2;
    z.totals = Hv > Hk ? kc * 2 * chunk::kC * kd * 4 : 0;
    return z;
}
template <typename P> P *at_byte(const void *p, size_t n) {
    return reinterpret_cast<P *>(const_cast<unsigned char *>(static_cast<const unsigned char *>(p)) + n);
}
// train: with the images of the backward pass, behind those of the forward pass.
chunk::Prepared prepared_at(const void *p, const ChunkSizes &z, bool train) {
    chunk::Prepared w{};
    size_t at = 0;
    w.kq16 = at_byte<__half>(p, at);
    w.mp16 = at_byte<__half>(p, at += z.kq16);
    w.vec16 = at_byte<float>(p, at += z.mp16);
    if (!train) return w;
    w.kq = at_byte<__nv_bfloat16>(p, at += z.vec16);
    w.mp = at_byte<__nv_bfloat16>(p, at += z.kq);
    w.vec = at_byte<float>(p, at += z.mp);
    return w;
}
chunk::Saved saved_at(const void *p, const ChunkSizes &z) {
    const size_t at = z.prepared() + z.kq + z.mp + z.vec;
    return {at_byte<__nv_bfloat16>(p, at), at_byte<__nv_bfloat16>(p, at + z.s)};
}

}  // namespace
}  // namespace dwc

using namespace dwc;

extern "C" {

dwconv_status dwconv_causal_fwd(int B, int T, int C, int W, dwconv_dtype dtype, const void *x, long long x_batch,
                                long long x_row, const void *w, const float *bias, dwconv_activation act,
                                const void *state, const int *lengths, void *y, void *state_out,
                                dwconv_stream stream) {
    const dwconv_status st = check_causal(B, T, C, W, dtype, act);
    if (st != DWCONV_OK) return st;
    if (x_batch < 0 || x_row < 0) return DWCONV_ERR_INVALID_ARG;
    const bool some = B > 0 && T > 0;
    if (some && (!x || !w || !y)) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype);
    // a row's last segment writes its window while the first may still read the one before
    if (overlap(state, state_out, es * B * (W - 1) * C)) return DWCONV_ERR_INVALID_ARG;
    if (!all_aligned({{x, es}, {w, es}, {bias, 4}, {state, es}, {lengths, 4}, {y, es}, {state_out, es}}))
        return DWCONV_ERR_MISALIGNED;
    if (B == 0 || (T == 0 && (!state_out || W == 1))) return DWCONV_OK;
    return cuda_to_status(launch_causal_fwd(B, T, C, W, dtype, x, x_batch, x_row, w, bias, act, state, lengths, y,
                                            state_out, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dwconv_causal_bwd_workspace_size(int B, int T, int C, int W, dwconv_dtype dtype) {
    if (check_causal(B, T, C, W, dtype, DWCONV_ACT_NONE) != DWCONV_OK || B == 0 || T == 0) return 0;
    return (size_t)causal_bwd_slices(B, T, C) * (W + 1) * C * sizeof(float);
}

dwconv_status dwconv_causal_bwd(int B, int T, int C, int W, dwconv_dtype dtype, const void *dy, long long dy_batch,
                                long long dy_row, const void *x, long long x_batch, long long x_row, const void *w,
                                const float *bias, dwconv_activation act, const void *state, const int *lengths,
                                void *dx, float *dw, float *db, void *dstate, void *workspace,
                                size_t workspace_bytes, dwconv_stream stream) {
    const dwconv_status st = check_causal(B, T, C, W, dtype, act);
    if (st != DWCONV_OK) return st;
    if (x_batch < 0 || x_row < 0 || dy_batch < 0 || dy_row < 0 || !dw) return DWCONV_ERR_INVALID_ARG;
    const bool some = B > 0 && T > 0;
    if (some && (!dy || !x || !w || !dx)) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype), need = dwconv_causal_bwd_workspace_size(B, T, C, W, dtype);
    if (some && (need == 0 || !workspace || workspace_bytes < need)) return DWCONV_ERR_INVALID_ARG;
    if (!all_aligned({{dy, es}, {x, es}, {w, es}, {bias, 4}, {state, es}, {lengths, 4}, {dx, es}, {dw, 4}, {db, 4},
                      {dstate, es}, {workspace, 16}}))
        return DWCONV_ERR_MISALIGNED;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (!some) {  // no token: every gradient is zero
        cudaError_t e = cudaMemsetAsync(dw, 0, sizeof(float) * W * C, cs);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, sizeof(float) * C, cs);
        if (e == cudaSuccess && dstate && B > 0 && W > 1)
            e = cudaMemsetAsync(dstate, 0, es * B * (W - 1) * C, cs);
        return cuda_to_status(e);
    }
    return cuda_to_status(launch_causal_bwd(B, T, C, W, dtype, dy, dy_batch, dy_row, x, x_batch, x_row, w, bias, act,
                                            state, lengths, dx, dstate, dw, db, static_cast<float *>(workspace),
                                            cs));
}

dwconv_status dwconv_causal_step(int B, int slots, int C, int W, dwconv_dtype dtype, const void *x, long long x_row,
                                 const void *w, const float *bias, dwconv_activation act, void *state,
                                 const int *slot_of, void *y, dwconv_stream stream) {
    const dwconv_status st = check_causal(B, 1, C, W, dtype, act);
    if (st != DWCONV_OK) return st;
    if (x_row < 0 || slots < 0 || (!slot_of && slots < B)) return DWCONV_ERR_INVALID_ARG;
    if (B > 0 && (!x || !w || !y || (!state && W > 1 && slots > 0))) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype);
    if (!all_aligned({{x, es}, {w, es}, {bias, 4}, {state, es}, {slot_of, 4}, {y, es}})) return DWCONV_ERR_MISALIGNED;
    if (B == 0) return DWCONV_OK;
    return cuda_to_status(launch_causal_step(B, slots, C, W, dtype, x, x_row, w, bias, act, state, slot_of, y,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

dwconv_status dwconv_block_norm_fwd(long long rows_outer, int rows_inner, int C, dwconv_dtype dtype,
                                    dwconv_norm norm, dwconv_gate gate_act, float eps, const void *y,
                                    const void *residual, const void *gate, const long long *strides,
                                    const float *w_post, const float *scale, const float *w_pre, void *h, void *n,
                                    dwconv_stream stream) {
    const dwconv_status st = check_norm(rows_outer, rows_inner, C, dtype, norm, gate_act, eps);
    if (st != DWCONV_OK) return st;
    if (!good_strides(strides, 6)) return DWCONV_ERR_INVALID_ARG;
    if (rows_outer > 0 && (!y || !h || !w_pre != !n)) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype);
    if (!all_aligned({{y, es}, {residual, es}, {gate, es}, {w_post, 4}, {scale, 4}, {w_pre, 4}, {h, es}, {n, es}}))
        return DWCONV_ERR_MISALIGNED;
    if (rows_outer == 0) return DWCONV_OK;
    return cuda_to_status(launch_block_norm_fwd(rows_outer, rows_inner, C, dtype, norm, gate_act, eps, y, residual,
                                                gate, strides, w_post, scale, w_pre, h, n,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

size_t dwconv_block_norm_bwd_workspace_size(long long rows_outer, int rows_inner, int C, dwconv_dtype dtype) {
    if (check_norm(rows_outer, rows_inner, C, dtype, DWCONV_NORM_RMS, DWCONV_GATE_NONE, 0.f) != DWCONV_OK) return 0;
    return (size_t)block_norm_slices(rows_outer * rows_inner, C) * 3 * C * sizeof(float);
}

dwconv_status dwconv_block_norm_bwd(long long rows_outer, int rows_inner, int C, dwconv_dtype dtype,
                                    dwconv_norm norm, dwconv_gate gate_act, float eps, const void *y,
                                    const void *residual, const void *gate, const void *dh, const void *dn,
                                    const long long *strides, const float *w_post, const float *scale,
                                    const float *w_pre, void *dy, void *dresidual, void *dgate, float *dw_post,
                                    float *dscale, float *dw_pre, void *workspace, size_t workspace_bytes,
                                    dwconv_stream stream) {
    const dwconv_status st = check_norm(rows_outer, rows_inner, C, dtype, norm, gate_act, eps);
    if (st != DWCONV_OK) return st;
    if (!good_strides(strides, 10) || (!w_pre && dn) || (dw_post && !w_post) || (dw_pre && !w_pre) ||
        (dgate && !gate))
        return DWCONV_ERR_INVALID_ARG;
    const bool some = rows_outer > 0;
    if (some && (!y || !dy || (!dh && !dn))) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype);
    const size_t need = dwconv_block_norm_bwd_workspace_size(rows_outer, rows_inner, C, dtype);
    if (some && (!workspace || workspace_bytes < need)) return DWCONV_ERR_INVALID_ARG;
    if (!all_aligned({{y, es}, {residual, es}, {gate, es}, {dh, es}, {dn, es}, {w_post, 4}, {scale, 4}, {w_pre, 4},
                      {dy, es}, {dresidual, es}, {dgate, es}, {dw_post, 4}, {dscale, 4}, {dw_pre, 4},
                      {workspace, 16}}))
        return DWCONV_ERR_MISALIGNED;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (!some) {
        for (float *p : {dw_post, dscale, dw_pre}) {
            if (!p) continue;
            const cudaError_t e = cudaMemsetAsync(p, 0, sizeof(float) * C, cs);
            if (e != cudaSuccess) return cuda_to_status(e);
        }
        return DWCONV_OK;
    }
    return cuda_to_status(launch_block_norm_bwd(rows_outer, rows_inner, C, dtype, norm, gate_act, eps, y, residual,
                                                gate, dh, dn, strides, w_post, scale, w_pre, dy, dresidual, dgate,
                                                dw_post, dscale, dw_pre, static_cast<float *>(workspace), cs));
}

size_t dwconv_delta_fwd_workspace_size(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype) {
    if (check_delta(B, T, Hk, Hv, K, V, dtype, dtype, 1.f) != DWCONV_OK || B == 0 || !chunked(T, K)) return 0;
    return chunk_sizes(B, T, Hk, Hv, K, V, dtype).prepared();
}

size_t dwconv_delta_saved_size(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype) {
    if (check_delta(B, T, Hk, Hv, K, V, dtype, dtype, 1.f) != DWCONV_OK || B == 0 || T == 0 || K > chunk::kMaxK)
        return 0;
    return chunk_sizes(B, T, Hk, Hv, K, V, dtype).saved();
}

size_t dwconv_delta_bwd_workspace_size(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype, int saved) {
    const size_t need = dwconv_delta_saved_size(B, T, Hk, Hv, K, V, dtype);
    return need == 0 ? 0 : chunk_sizes(B, T, Hk, Hv, K, V, dtype).walked() + (saved ? 0 : need);
}

dwconv_status dwconv_delta_fwd(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype,
                               dwconv_dtype gate_dtype, const void *q, const void *k, const void *v, const void *g,
                               const void *beta, const long long *strides, float scale, int qk_norm,
                               const float *state, const int *lengths, void *out, float *state_out, void *saved,
                               void *workspace, size_t workspace_bytes, dwconv_stream stream) {
    const dwconv_status st = check_delta(B, T, Hk, Hv, K, V, dtype, gate_dtype, scale);
    if (st != DWCONV_OK) return st;
    if (!good_strides(strides, 15)) return DWCONV_ERR_INVALID_ARG;
    if (B > 0 && T > 0 && (!q || !k || !v || !g || !beta || !out)) return DWCONV_ERR_INVALID_ARG;
    if (state != state_out && overlap(state, state_out, sizeof(float) * B * Hv * K * V)) return DWCONV_ERR_INVALID_ARG;
    if (saved && K > chunk::kMaxK) return DWCONV_ERR_UNSUPPORTED;
    const size_t need = saved ? 0 : dwconv_delta_fwd_workspace_size(B, T, Hk, Hv, K, V, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype), gs = float_size(gate_dtype);
    if (!all_aligned({{q, es}, {k, es}, {v, es}, {g, gs}, {beta, gs}, {state, 4}, {lengths, 4}, {out, es},
                      {state_out, 4}, {saved, 16}, {workspace, 16}}))
        return DWCONV_ERR_MISALIGNED;
    if (B == 0 || (T == 0 && (!state_out || state_out == state))) return DWCONV_OK;
    DeltaArgs a = delta_args(B, T, Hk, Hv, K, V, dtype, gate_dtype, q, k, v, g, beta, strides, scale, qk_norm);
    a.state = state; a.state_out = state_out; a.lengths = lengths; a.out = out;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0 || (!saved && !chunked(T, K))) return cuda_to_status(launch_delta_recurrent(a, dtype, cs));
    const ChunkSizes z = chunk_sizes(B, T, Hk, Hv, K, V, dtype);
    const chunk::Prepared w = prepared_at(saved ? saved : workspace, z, saved != nullptr);
    const cudaError_t e = chunk::launch_prep(a, dtype, w, cs);
    if (e != cudaSuccess) return cuda_to_status(e);
    return cuda_to_status(chunk::launch_chunk_fwd(a, dtype, w, saved ? saved_at(saved, z) : chunk::Saved{}, cs));
}

dwconv_status dwconv_delta_bwd(int B, int T, int Hk, int Hv, int K, int V, dwconv_dtype dtype,
                               dwconv_dtype gate_dtype, const void *d_out, const void *q, const void *k,
                               const void *v, const void *g, const void *beta, const long long *strides, float scale,
                               int qk_norm, const float *state, const int *lengths, const float *dstate_out, void *dq,
                               void *dk, void *dv, void *dg, void *dbeta, float *dstate, const void *saved,
                               void *workspace, size_t workspace_bytes, dwconv_stream stream) {
    const dwconv_status st = check_delta(B, T, Hk, Hv, K, V, dtype, gate_dtype, scale);
    if (st != DWCONV_OK) return st;
    if (K > chunk::kMaxK) return DWCONV_ERR_UNSUPPORTED;
    if (!good_strides(strides, 18)) return DWCONV_ERR_INVALID_ARG;
    const bool some = B > 0 && T > 0;
    if (some && (!d_out || !q || !k || !v || !g || !beta || !dq || !dk || !dv || !dg || !dbeta))
        return DWCONV_ERR_INVALID_ARG;
    const size_t need = dwconv_delta_bwd_workspace_size(B, T, Hk, Hv, K, V, dtype, saved != nullptr);
    if (some && (!workspace || workspace_bytes < need)) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype), gs = float_size(gate_dtype);
    if (!all_aligned({{d_out, es}, {q, es}, {k, es}, {v, es}, {g, gs}, {beta, gs}, {state, 4}, {lengths, 4},
                      {dstate_out, 4}, {dq, es}, {dk, es}, {dv, es}, {dg, gs}, {dbeta, gs}, {dstate, 4}, {saved, 16},
                      {workspace, 16}}))
        return DWCONV_ERR_MISALIGNED;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (!some) {  // no token: the state passes through
        const size_t bytes = sizeof(float) * B * Hv * K * V;
        if (!dstate || bytes == 0) return DWCONV_OK;
        return cuda_to_status(dstate_out ? cudaMemcpyAsync(dstate, dstate_out, bytes, cudaMemcpyDeviceToDevice, cs)
                                         : cudaMemsetAsync(dstate, 0, bytes, cs));
    }
    DeltaArgs a = delta_args(B, T, Hk, Hv, K, V, dtype, gate_dtype, q, k, v, g, beta, strides, scale, qk_norm);
    a.state = state; a.lengths = lengths;
    chunk::DeltaGrads d{};
    d.d_o = d_out;
    const long long dense[3] = {(long long)T * Hv * V, (long long)Hv * V, V};
    for (int i = 0; i < 3; ++i) d.do_s[i] = strides ? strides[15 + i] : dense[i];
    d.dstate_out = dstate_out;
    d.dq = dq; d.dk = dk; d.dv = dv; d.dg = dg; d.dbeta = dbeta; d.dstate = dstate;
    const ChunkSizes z = chunk_sizes(B, T, Hk, Hv, K, V, dtype);
    const chunk::Walked walked{at_byte<__nv_bfloat16>(workspace, 0), at_byte<__nv_bfloat16>(workspace, z.s),
                               at_byte<__nv_bfloat16>(workspace, z.s + z.f)};
    d.totals = z.totals ? at_byte<float>(workspace, z.s + z.f + z.d_o) : nullptr;
    const void *have = saved ? saved : at_byte<unsigned char>(workspace, z.walked());
    const chunk::Prepared w = prepared_at(have, z, true);
    cudaError_t e = cudaSuccess;
    if (!saved) {
        e = chunk::launch_prep(a, dtype, w, cs);
        if (e == cudaSuccess) e = chunk::launch_chunk_fwd(a, dtype, w, saved_at(have, z), cs);
    }
    if (e == cudaSuccess) e = chunk::launch_chunk_walk_back(a, d, dtype, w, walked, cs);
    if (e == cudaSuccess) e = chunk::launch_chunk_grads(a, d, dtype, w, saved_at(have, z), walked, cs);
    return cuda_to_status(e);
}

dwconv_status dwconv_delta_step(int B, int slots, int Hk, int Hv, int K, int V, dwconv_dtype dtype,
                                dwconv_dtype gate_dtype, const void *q, const void *k, const void *v, const void *g,
                                const void *beta, const long long *strides, float scale, int qk_norm, float *state,
                                const int *slot_of, void *out, dwconv_stream stream) {
    const dwconv_status st = check_delta(B, 1, Hk, Hv, K, V, dtype, gate_dtype, scale);
    if (st != DWCONV_OK) return st;
    if (!good_strides(strides, 10) || slots < 0 || (!slot_of && slots < B)) return DWCONV_ERR_INVALID_ARG;
    if (B > 0 && (!q || !k || !v || !g || !beta || !out || (!state && slots > 0))) return DWCONV_ERR_INVALID_ARG;
    const size_t es = float_size(dtype), gs = float_size(gate_dtype);
    if (!all_aligned({{q, es}, {k, es}, {v, es}, {g, gs}, {beta, gs}, {state, 4}, {slot_of, 4}, {out, es}}))
        return DWCONV_ERR_MISALIGNED;
    if (B == 0) return DWCONV_OK;
    long long s[15];
    if (strides)
        for (int i = 0; i < 5; ++i) {
            s[3 * i] = strides[2 * i];
            s[3 * i + 1] = 0;
            s[3 * i + 2] = strides[2 * i + 1];
        }
    DeltaArgs a = delta_args(B, 1, Hk, Hv, K, V, dtype, gate_dtype, q, k, v, g, beta, strides ? s : nullptr, scale,
                             qk_norm);
    a.state = state; a.state_out = state; a.slots = slot_of; a.N = slots; a.out = out;
    return cuda_to_status(launch_delta_recurrent(a, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
