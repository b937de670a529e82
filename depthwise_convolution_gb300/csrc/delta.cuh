// The gated delta rule: arguments shared by its kernels and their launchers.
//
// Per value head, with a = e^g and a state S [K][V]:
//   S_t = a_t S_(t-1) + beta_t k_t (v_t - a_t S_(t-1)^T k_t)^T,   o_t = scale S_t^T q_t.
// q and k may be used as they are or divided by their norm
// sqrt(sum x^2 + kDeltaEps).  Hv value heads share Hk key heads: value head h
// reads key head h / (Hv / Hk).
#pragma once

#include "mixer_common.cuh"

namespace dwc {

constexpr float kDeltaEps = 1e-6f;
constexpr int kDeltaMaxK = 256;       // recurrent kernel
constexpr int kDeltaChunk = 64;       // tokens of a chunk
// Log decays below this reset the state just as well (e^g is zero in fp32 from
// -104 on), and sums of them leave what stands beside them in the sum intact:
// 64 of them as hi + lo floats are good to 2^-28.  Minus infinity would not be
// (its differences are not numbers), nor the lowest float (it swallows the rest).
constexpr float kDeltaReset = -1e4f;

struct DeltaArgs {
    int B, T, Hk, Hv, K, V;
    const void *q, *k, *v, *g, *beta;
    long long q_s[3], k_s[3], v_s[3], g_s[3], b_s[3];  // batch, token, head strides in elements
    int gate_f32;                                      // g and beta are float, whatever q's type
    float scale;
    int qk_norm;
    const float *state;      // [B][Hv][K][V] (null: zeros), or [N][Hv][K][V] with slots
    float *state_out;        // the same layout; null: dropped
    const int *slots;        // state slot per row (null: row b); outside [0, N): the row is idle
    int N;
    const int *lengths;      // live tokens per row (null: T)
    void *out;               // [B][T][Hv][V], dense; null (chunked kernels): no output wanted
};

template <typename T> __device__ __forceinline__ float gate_at(const void *p, long long i, int f32) {
    return f32 ? static_cast<const float *>(p)[i] : to_f32(static_cast<const T *>(p)[i]);
}

// Token-by-token form: any T, K <= kDeltaMaxK.
cudaError_t launch_delta_recurrent(const DeltaArgs &a, dwconv_dtype dt, cudaStream_t st);

}  // namespace dwc
