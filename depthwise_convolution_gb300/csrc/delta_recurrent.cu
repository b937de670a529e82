// The gated delta rule token by token: single tokens against cached states,
// short sequences, and keys wider than the chunked kernels take.
//
// A CTA holds K x 32 values of one head's state in registers (16 row groups of
// 8 lanes, 4 columns a lane), so a state is read once and written once
// whatever the number of tokens.  Columns of the state are independent given q
// and k; rows meet in two sums per token.  Both are taken over the old state,
//
//   y = S^T k, z = S^T q  ->  u = beta (v - a y),  o = scale (a z + (q.k) u),
//
// which is the output of the new state without a second pass over it.  A
// single token moves 8 K V bytes of state per head and little else: the floor
// is memory.  240 live rows of 250, 16 heads, K = V = 128: 88 us, 5.7 TB/s of 506 MB;
// one row 4.7 us, a chain of latencies.
#include "delta.cuh"

namespace dwc {

namespace {

constexpr int kLanes = 8, kGroups = 16, kRecThreads = kLanes * kGroups;

template <typename T, int NR, int CV>
__global__ void __launch_bounds__(kRecThreads) delta_recurrent_kernel(DeltaArgs a) {
    __shared__ float ks[2][NR * kGroups], qs[2][NR * kGroups];
    __shared__ float sums[2][3][kRecThreads / 32];
    __shared__ float yz[2][kRecThreads / 32][kLanes][2 * CV];
    const int tid = threadIdx.x, lane = tid % kLanes, rg = tid / kLanes, warp = tid / 32;
    const int c = (blockIdx.x * kLanes + lane) * CV, h = blockIdx.y, b = blockIdx.z;
    const int hk = h / (a.Hv / a.Hk);
    after_previous();
    const int slot = a.slots ? a.slots[b] : b;
    const bool idle = slot < 0 || slot >= a.N;
    const int n = idle ? 0 : live_length(a.lengths, b, a.T);
    T *out = static_cast<T *>(a.out) + ((long long)b * a.T * a.Hv + h) * a.V + c;
    const long long o_row = (long long)a.Hv * a.V;

    float s[NR][CV];
    const long long at = ((long long)slot * a.Hv + h) * a.K * a.V + c;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = r * kGroups + rg;
        Pack<float, CV> p = zero_pack<float, CV>();
        if (!idle && a.state && row < a.K && c < a.V) p = load_pack<float, CV>(a.state + at + (long long)row * a.V);
#pragma unroll
        for (int i = 0; i < CV; ++i) s[r][i] = p.get(i);
    }
    const T *q = static_cast<const T *>(a.q) + b * a.q_s[0] + hk * a.q_s[2];
    const T *k = static_cast<const T *>(a.k) + b * a.k_s[0] + hk * a.k_s[2];
    const T *v = static_cast<const T *>(a.v) + b * a.v_s[0] + h * a.v_s[2] + c;

    for (int t = 0; t < n; ++t) {
        const int f = t & 1;
        // q and k of the token into shared memory, with |k|^2, |q|^2 and q.k
        float m[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = tid; i < NR * kGroups; i += kRecThreads) {
            const float kv = i < a.K ? to_f32(k[t * a.k_s[1] + i]) : 0.f;
            const float qv = i < a.K ? to_f32(q[t * a.q_s[1] + i]) : 0.f;
            ks[f][i] = kv;
            qs[f][i] = qv;
            m[0] = fmaf(kv, kv, m[0]);
            m[1] = fmaf(qv, qv, m[1]);
            m[2] = fmaf(qv, kv, m[2]);
        }
        float vv[CV];
#pragma unroll
        for (int i = 0; i < CV; ++i) vv[i] = c + i < a.V ? to_f32(v[t * a.v_s[1] + i]) : 0.f;
        const float alpha = __expf(gate_at<T>(a.g, b * a.g_s[0] + t * a.g_s[1] + h * a.g_s[2], a.gate_f32));
        const float beta = gate_at<T>(a.beta, b * a.b_s[0] + t * a.b_s[1] + h * a.b_s[2], a.gate_f32);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
#pragma unroll
            for (int o = 16; o; o >>= 1) m[j] += __shfl_xor_sync(0xFFFFFFFFu, m[j], o);
            if (tid % 32 == 0) sums[f][j][warp] = m[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            m[j] = 0.f;
#pragma unroll
            for (int w = 0; w < kRecThreads / 32; ++w) m[j] += sums[f][j][w];
        }
        const float kn = a.qk_norm ? rsqrtf(m[0] + kDeltaEps) : 1.f;
        const float qn = (a.qk_norm ? rsqrtf(m[1] + kDeltaEps) : 1.f) * a.scale;
        float y[CV], z[CV];
#pragma unroll
        for (int i = 0; i < CV; ++i) y[i] = z[i] = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float kv = ks[f][r * kGroups + rg], qv = qs[f][r * kGroups + rg];
#pragma unroll
            for (int i = 0; i < CV; ++i) {
                y[i] = fmaf(s[r][i], kv, y[i]);
                z[i] = fmaf(s[r][i], qv, z[i]);
            }
        }
        // over the warp's 4 row groups, then over the warps
#pragma unroll
        for (int i = 0; i < CV; ++i) {
#pragma unroll
            for (int o = kLanes; o < 32; o *= 2) {
                y[i] += __shfl_xor_sync(0xFFFFFFFFu, y[i], o);
                z[i] += __shfl_xor_sync(0xFFFFFFFFu, z[i], o);
            }
            if (tid % 32 < kLanes) {
                yz[f][warp][lane][i] = y[i];
                yz[f][warp][lane][CV + i] = z[i];
            }
        }
        __syncthreads();
        float u[CV];
        float o[CV];
#pragma unroll
        for (int i = 0; i < CV; ++i) {
            float ys = 0.f, zs = 0.f;
#pragma unroll
            for (int w = 0; w < kRecThreads / 32; ++w) {
                ys += yz[f][w][lane][i];
                zs += yz[f][w][lane][CV + i];
            }
            u[i] = beta * (vv[i] - alpha * kn * ys) * kn;
            o[i] = qn * fmaf(m[2], u[i], alpha * zs);
        }
        if (rg == 0 && c < a.V) store_pack<T, CV>(out + t * o_row, Pack<T, CV>::of(o));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float kv = ks[f][r * kGroups + rg];
#pragma unroll
            for (int i = 0; i < CV; ++i) s[r][i] = fmaf(kv, u[i], alpha * s[r][i]);
        }
    }
    if (c < a.V)
        for (int t = n + rg; t < a.T; t += kGroups) store_pack<T, CV>(out + t * o_row, zero_pack<T, CV>());
    if (idle || !a.state_out || (n == 0 && a.state == a.state_out)) return;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = r * kGroups + rg;
        const Pack<float, CV> p = Pack<float, CV>::of(s[r]);
        if (row < a.K && c < a.V) store_pack<float, CV>(a.state_out + at + (long long)row * a.V, p);
    }
}

template <typename T, int CV> cudaError_t run(const DeltaArgs &a, cudaStream_t st) {
    const dim3 grid((a.V + kLanes * CV - 1) / (kLanes * CV), a.Hv, a.B);
    note_launches(1);
    note_kernel("delta_recurrent");
    auto kern = a.K <= 64    ? delta_recurrent_kernel<T, 4, CV>
                : a.K <= 128 ? delta_recurrent_kernel<T, 8, CV>
                             : delta_recurrent_kernel<T, 16, CV>;
    return launch_after(kern, grid, kRecThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs &a, dwconv_dtype dt, cudaStream_t st) {
    auto pick = [&](auto t) {
        using E = decltype(t);
        // four columns a lane where rows of the state and of the output are whole vectors
        auto ok = [](const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
        const bool vec = a.V % 4 == 0 && ok(a.state, 16) && ok(a.state_out, 16) && ok(a.out, 4 * sizeof(E));
        return vec ? run<E, 4>(a, st) : run<E, 1>(a, st);
    };
    switch (dt) {
        case DWCONV_FP32: return pick(float{});
        case DWCONV_FP16: return pick(__half{});
        default: return pick(__nv_bfloat16{});
    }
}

}  // namespace dwc
