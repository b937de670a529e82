// Pieces shared by the token mixer's translation units (causal convolution,
// gated delta rule, block norms): vectors of channels, the split-sum pass and
// launch helpers.
#pragma once

#include "common.cuh"

namespace dwc {

constexpr int kMaxNormWidth = 16384;  // values of a row that the norms take

// VEC adjacent values of one storage type, moved as one access: 16 bytes for
// VEC = 8 (16-bit) and 4 (fp32), 8 bytes for VEC = 4 (16-bit), one element for
// VEC = 1.  Pairs of 16-bit values stay packed in words until get() widens
// them: taken apart as elements, a load would be waited for where it is made
// instead of where its values are used.
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Pack {
    static constexpr int WORDS = sizeof(T) * VEC / 4;
    unsigned w[WORDS];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[i]);
        } else {
            const float2 f = unpack2<T>(w[i / 2]);
            return i & 1 ? f.y : f.x;
        }
    }
    static __device__ __forceinline__ Pack of(const float (&x)[VEC]) {
        Pack r;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) r.w[i] = __float_as_uint(x[i]);
            else r.w[i] = pack2<T>(make_float2(x[2 * i], x[2 * i + 1]));
        }
        return r;
    }
    static __device__ __forceinline__ Pack zero() {
        Pack r;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.w[i] = 0u;
        return r;
    }
};
template <typename T> struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
    static __device__ __forceinline__ Pack of(const float (&x)[1]) { return Pack{from_f32<T>(x[0])}; }
    static __device__ __forceinline__ Pack zero() { return Pack{from_f32<T>(0.f)}; }
};
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, VEC> *>(p);
}
template <typename T, int VEC> __device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &v) {
    *reinterpret_cast<Pack<T, VEC> *>(p) = v;
}
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> zero_pack() { return Pack<T, VEC>::zero(); }

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// Launches a kernel whose blocks may be set up while the one before it in the
// stream ends; every thread calls after_previous before it touches memory, which
// it then reads with plain loads (read-only ones could be moved ahead of it).  The
// delta rule's four kernels of a training step took 8 us more without.
template <typename... A>
cudaError_t launch_after(void (*kern)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                                   A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) (void)cudaGetLastError();  // told here, not to who asks next
    return e;
}
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// Length of row b: the whole T without a lengths vector, else its entry
// brought into [0, T] (it lives on the device, so the host cannot refuse it).
__device__ __forceinline__ int live_length(const int *lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : n > T ? T : n;
}

// Sums Z slices part[z][count] in a fixed order into up to three float
// vectors: columns [0, n0) go to out0, the next n1 to out1, the rest to out2
// (a null vector's columns are dropped).  Same split as launch_wgrad_reduce.
cudaError_t launch_split_sums(const float *part, int Z, long long count, float *out0, long long n0, float *out1,
                              long long n1, float *out2, cudaStream_t st);

}  // namespace dwc
