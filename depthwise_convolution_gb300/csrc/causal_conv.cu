// Short causal depthwise convolution along time, with bias and SiLU:
//
//   z[b,t,c] = bias[c] + sum_{j<W} w[j,c] x[b, t-(W-1)+j, c],   y = act(z),
//
// where positions before the sequence come from a window state [B][W-1][C] or
// read as zero.  W multiply-adds per element against four bytes moved: the floor
// is memory, so a thread owns a few adjacent channels and walks down the tokens
// with the window in registers, and each x is read once apart from the W-1 tokens
// that neighbouring segments share.  4 x 4096 x 4096 bf16, W = 4, SiLU: forward 52
// us (5.1 TB/s), backward 98 us (4.1 TB/s: 122 registers leave 16 warps an SM, which
// issue 0.5 instructions a cycle and scheduler, 27 an element, five of them the two
// special functions of a sigmoid).  fp32: 89 us (6.0 TB/s) and 132 us (6.1 TB/s).
#include <algorithm>

#include "mixer_common.cuh"

namespace dwc {

namespace {

constexpr int kThreads = 128;

struct CausalArgs {
    int B, T, C, W;
    int act;
    const void *x, *w, *state, *dy;
    const float *bias;
    const int *lengths;
    void *y, *state_out;
    long long x_batch, x_row, dy_batch, dy_row;
    float *part;
    void *dx, *dstate;
    int seg;  // tokens a thread walks
};

// Arithmetic on a thread's channels in pairs (packed fp32 instructions: half the
// issue slots) or, where rows are no whole vectors, one by one.
__device__ __forceinline__ float2 fma_(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul_(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add_(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 sigmoid_(float2 a) { return make_float2(sigmoid(a.x), sigmoid(a.y)); }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ float sigmoid_(float a) { return sigmoid(a); }
template <int VEC> struct Chan {
    using E = std::conditional_t<VEC == 1, float, float2>;
    static constexpr int N = VEC == 1 ? 1 : VEC / 2;
    static __device__ __forceinline__ E all(float v) {
        if constexpr (VEC == 1) return v;
        else return make_float2(v, v);
    }
    template <typename P> static __device__ __forceinline__ E get(const P &p, int i) {
        if constexpr (VEC == 1) return p.get(0);
        else return make_float2(p.get(2 * i), p.get(2 * i + 1));
    }
    static __device__ __forceinline__ float at(const E (&x)[N], int i) {
        if constexpr (VEC == 1) return x[0];
        else return i & 1 ? x[i / 2].y : x[i / 2].x;
    }
    template <typename T> static __device__ __forceinline__ Pack<T, VEC> pack(const E (&x)[N]) {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = at(x, i);
        return Pack<T, VEC>::of(f);
    }
};

template <typename T, int VEC, int W> struct Taps {
    using X = Chan<VEC>;
    typename X::E w[W][X::N], bias[X::N];
    __device__ __forceinline__ Taps(const CausalArgs &a, int c) {
        const T *wp = static_cast<const T *>(a.w) + c;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const Pack<T, VEC> p = load_pack<T, VEC>(wp + (long long)j * a.C);
#pragma unroll
            for (int i = 0; i < X::N; ++i) w[j][i] = X::get(p, i);
        }
#pragma unroll
        for (int i = 0; i < X::N; ++i) {
            if constexpr (VEC == 1) bias[i] = a.bias ? a.bias[c] : 0.f;
            else bias[i] = a.bias ? make_float2(a.bias[c + 2 * i], a.bias[c + 2 * i + 1]) : X::all(0.f);
        }
    }
};

// x of row b at token t (may be negative: the window state, or zero).
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> token(const CausalArgs &a, const T *x, const T *state, int t, int W1) {
    if (t >= 0) return load_pack<T, VEC>(x + (long long)t * a.x_row);
    if (state) return load_pack<T, VEC>(state + (long long)(t + W1) * a.C);
    return zero_pack<T, VEC>();
}

// Forward: grid (channel vectors x segments, B).  Eight tokens are loaded
// before any of them is used.  Tokens at and beyond the row's length are
// written as zero and never read.  The threads of the extra last segment write
// the window that the row leaves.  Batches of live tokens run without a check
// per token: with one the passes were bound by instructions, not memory.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) causal_fwd_kernel(CausalArgs a) {
    constexpr int W1 = W - 1, U = 8;
    after_previous();
    const int nvec = a.C / VEC;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int s = (int)(id / nvec), c = (int)(id - (long long)s * nvec) * VEC, b = blockIdx.y;
    const int nseg = (a.T + a.seg - 1) / a.seg;
    if (s > nseg || (s == nseg && !a.state_out)) return;
    const int n = live_length(a.lengths, b, a.T);
    const T *x = static_cast<const T *>(a.x) + (long long)b * a.x_batch + c;
    const T *state = a.state ? static_cast<const T *>(a.state) + (long long)b * W1 * a.C + c : nullptr;
    if (s == nseg) {
        T *so = static_cast<T *>(a.state_out) + (long long)b * W1 * a.C + c;
#pragma unroll
        for (int i = 0; i < W1; ++i)
            store_pack<T, VEC>(so + (long long)i * a.C, token<T, VEC>(a, x, state, n - W1 + i, W1));
        return;
    }
    const int t0 = s * a.seg, t1 = min(a.T, t0 + a.seg), live = min(t1, n);
    T *y = static_cast<T *>(a.y) + ((long long)b * a.T + t0) * a.C + c;
    int t = t0;
    if (t0 < n) {
        const Taps<T, VEC, W> k(a, c);
        using X = Chan<VEC>;
        typename X::E win[W][X::N];  // win[j]: x of token t - W1 + j; the last slot is the newest
#pragma unroll
        for (int j = 0; j < W1; ++j) {
            const Pack<T, VEC> p = token<T, VEC>(a, x, state, t0 - W1 + j, W1);
#pragma unroll
            for (int i = 0; i < X::N; ++i) win[j + 1][i] = X::get(p, i);
        }
        auto step = [&](const Pack<T, VEC> &in) {
            typename X::E out[X::N];
#pragma unroll
            for (int i = 0; i < X::N; ++i) {
#pragma unroll
                for (int j = 0; j < W1; ++j) win[j][i] = win[j + 1][i];
                win[W1][i] = X::get(in, i);
                out[i] = k.bias[i];
#pragma unroll
                for (int j = 0; j < W; ++j) out[i] = fma_(k.w[j][i], win[j][i], out[i]);
                if (a.act == DWCONV_ACT_SILU) out[i] = mul_(out[i], sigmoid_(out[i]));
            }
            store_pack<T, VEC>(y, X::template pack<T>(out));
            y += a.C;
        };
        const T *xp = x + (long long)t * a.x_row;
        for (; t + U <= live; t += U) {
            Pack<T, VEC> in[U];
#pragma unroll
            for (int u = 0; u < U; ++u, xp += a.x_row) in[u] = load_pack<T, VEC>(xp);
#pragma unroll
            for (int u = 0; u < U; ++u) step(in[u]);
        }
        for (; t < live; ++t, xp += a.x_row) step(load_pack<T, VEC>(xp));
    }
    for (; t < t1; ++t, y += a.C) store_pack<T, VEC>(y, zero_pack<T, VEC>());
}

// Backward: dz = dy act'(z) with z recomputed, dx[t] = sum_j w[j] dz[t+W-1-j],
// dw[j] = sum_t dz[t] x[t-(W-1)+j], db = sum_t dz[t].  A thread walks its
// segment plus the W-1 tokens after it (their dz reach back into the segment)
// with the x window and the last W values of dz in registers.  A block holds
// 32 channel vectors times kRows segments; their weight sums are added in
// segment order in shared memory and written as one slice, so the result does
// not depend on scheduling.  dx of the tokens before the sequence is the
// window's gradient.
constexpr int kRows = 4;

// Asynchronous copy of one lane's vector into its place in shared memory.
template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src),
                     "n"(BYTES)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// The tokens of a segment between its edges arrive through a queue of 4 batches
// (2 of 16-byte vectors: 32 KB either way) of 4 tokens in shared memory, every
// lane copying and reading its own vectors: loads straight into registers left
// the memory idle while a batch was worked on.  Five blocks an SM instead of four
// (96 registers, with a few spilled) take as long, six twice as long.
constexpr int kBatch = 4;
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(32 * kRows, W <= 4 ? 4 : 1) causal_bwd_kernel(CausalArgs a) {
    constexpr int W1 = W - 1, U = kBatch;
    constexpr bool ASYNC = sizeof(T) * VEC >= 4;
    constexpr int kQueue = sizeof(T) * VEC == 16 ? 2 : 4;
    using X = Chan<VEC>;
    using E = typename X::E;
    __shared__ Pack<T, VEC> queue[ASYNC ? kQueue : 1][ASYNC ? U : 1][2][ASYNC ? kRows : 1][ASYNC ? 32 : 1];
    after_previous();
    const int lane = threadIdx.x, r = threadIdx.y, b = blockIdx.z;
    const int c = (blockIdx.x * 32 + lane) * VEC;
    const int n = live_length(a.lengths, b, a.T);
    const int t0 = (blockIdx.y * kRows + r) * a.seg, t1 = min(a.T, t0 + a.seg);
    const bool on = c < a.C;
    E dw[W][X::N], db[X::N];
#pragma unroll
    for (int i = 0; i < X::N; ++i) {
        db[i] = X::all(0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = X::all(0.f);
    }
    if (on && t0 < a.T) {
        const T *x = static_cast<const T *>(a.x) + (long long)b * a.x_batch + c;
        const T *dy = static_cast<const T *>(a.dy) + (long long)b * a.dy_batch + c;
        const T *state = a.state ? static_cast<const T *>(a.state) + (long long)b * W1 * a.C + c : nullptr;
        T *dx = static_cast<T *>(a.dx) + (long long)b * a.T * a.C + c;
        const Taps<T, VEC, W> k(a, c);
        E win[W][X::N], dz[W][X::N];  // dz[j]: dz of token t - W1 + j
        const int last = min(t1 + W1, n);  // beyond the tokens whose dz this thread needs
#pragma unroll
        for (int j = 0; j < W1; ++j) {
            const Pack<T, VEC> p = t0 < n ? token<T, VEC>(a, x, state, t0 - W1 + j, W1) : zero_pack<T, VEC>();
#pragma unroll
            for (int i = 0; i < X::N; ++i) win[j + 1][i] = X::get(p, i);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < X::N; ++i) dz[j][i] = X::all(0.f);
        // Token t gives dz[t] (none beyond the live ones) and completes dx[t - W1];
        // its dz counts for the weights where the segment owns it.
        auto step = [&](const Pack<T, VEC> &xi, const Pack<T, VEC> &di, auto has_dz, bool mine) {
            E out[X::N];
#pragma unroll
            for (int i = 0; i < X::N; ++i) {
#pragma unroll
                for (int j = 0; j < W1; ++j) {
                    win[j][i] = win[j + 1][i];
                    dz[j][i] = dz[j + 1][i];
                }
                E d = X::all(0.f);
                if (decltype(has_dz)::value) {
                    win[W1][i] = X::get(xi, i);
                    d = X::get(di, i);
                    if (a.act == DWCONV_ACT_SILU) {
                        E z = k.bias[i];
#pragma unroll
                        for (int j = 0; j < W; ++j) z = fma_(k.w[j][i], win[j][i], z);
                        // slope: s (1 + z (1 - s))
                        const E s = sigmoid_(z);
                        const E t = fma_(z, fma_(s, X::all(-1.f), X::all(1.f)), X::all(1.f));
                        d = mul_(d, mul_(s, t));
                    }
                    if (mine) {
                        db[i] = add_(db[i], d);
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][i] = fma_(d, win[j][i], dw[j][i]);
                    }
                }
                dz[W1][i] = d;
                out[i] = mul_(k.w[0][i], dz[W1][i]);
#pragma unroll
                for (int j = 1; j < W; ++j) out[i] = fma_(k.w[j][i], dz[W1 - j][i], out[i]);
            }
            return X::template pack<T>(out);
        };
        auto edge = [&](int t) {  // one token with every check
            const bool in = t < last;
            const Pack<T, VEC> xi = in ? load_pack<T, VEC>(x + (long long)t * a.x_row) : zero_pack<T, VEC>();
            const Pack<T, VEC> di = in ? load_pack<T, VEC>(dy + (long long)t * a.dy_row) : zero_pack<T, VEC>();
            const Pack<T, VEC> out = in ? step(xi, di, std::true_type{}, t < t1) : step(xi, di, std::false_type{}, false);
            const int s = t - W1;  // the token whose gradient is now complete
            if (s >= t0) store_pack<T, VEC>(dx + (long long)s * a.C, out);
            else if (s < 0 && a.dstate)
                store_pack<T, VEC>(static_cast<T *>(a.dstate) + ((long long)b * W1 + s + W1) * a.C + c, out);
        };
        int t = min(t0 + W1, t1 + W1);
        const int batches = max(0, (min(t1, n) - t) / U);
        const T *xp = x + (long long)t * a.x_row, *dp = dy + (long long)t * a.dy_row;
        auto fetch = [&](int g) {
            if (ASYNC && g < batches) {
#pragma unroll
                for (int u = 0; u < U; ++u, xp += a.x_row, dp += a.dy_row) {
                    copy_async<sizeof(Pack<T, VEC>)>(&queue[g % kQueue][u][0][r][lane], xp);
                    copy_async<sizeof(Pack<T, VEC>)>(&queue[g % kQueue][u][1][r][lane], dp);
                }
            }
            if (ASYNC) copy_commit();
        };
#pragma unroll
        for (int g = 0; g < kQueue - 1; ++g) fetch(g);
        for (int e = t0; e < t; ++e) edge(e);
        T *out = dx + (long long)(t - W1) * a.C;
        for (int g = 0; g < batches; ++g, t += U) {
            Pack<T, VEC> xi[U], di[U];
            if (ASYNC) copy_wait<kQueue - 2>();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if constexpr (ASYNC) {
                    xi[u] = queue[g % kQueue][u][0][r][lane];
                    di[u] = queue[g % kQueue][u][1][r][lane];
                } else {
                    xi[u] = load_pack<T, VEC>(xp + u * a.x_row);
                    di[u] = load_pack<T, VEC>(dp + u * a.dy_row);
                }
            }
            if (!ASYNC) {
                xp += U * a.x_row;
                dp += U * a.dy_row;
            }
            fetch(g + kQueue - 1);
#pragma unroll
            for (int u = 0; u < U; ++u, out += a.C) store_pack<T, VEC>(out, step(xi[u], di[u], std::true_type{}, true));
        }
        for (; t < t1 + W1; ++t) edge(t);
    }
    // One slice per block: rows added in segment order, one quantity at a time.
    __shared__ float sums[kRows][32][VEC + 1];
    const long long slice = (long long)blockIdx.z * gridDim.y + blockIdx.y;
    float *part = a.part + slice * (long long)(W + 1) * a.C;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) sums[r][lane][i] = j < W ? X::at(dw[j < W ? j : 0], i) : X::at(db, i);
        __syncthreads();
        for (int e = r * 32 + lane; e < 32 * VEC; e += 32 * kRows) {
            const int l = e / VEC, i = e % VEC, ch = (blockIdx.x * 32 + l) * VEC + i;
            float t = sums[0][l][i];
#pragma unroll
            for (int q = 1; q < kRows; ++q) t += sums[q][l][i];
            if (ch < a.C) part[(long long)j * a.C + ch] = t;
        }
        __syncthreads();
    }
}

// One token per row against the window in slot slots[b] (b without a slots
// vector), which is shifted in place; a slot outside [0, N) leaves the row
// idle: its y is zero and no window changes.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
    causal_step_kernel(int B, int N, int C, int act, const T *x, long long x_row,
                       const T *w, const float *bias, T *state,
                       const int *slots, T *y) {
    constexpr int W1 = W - 1;
    after_previous();
    const int nvec = C / VEC;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int b = (int)(id / nvec), c = (int)(id - (long long)b * nvec) * VEC;
    if (b >= B) return;
    const int slot = slots ? slots[b] : b;
    T *yo = y + (long long)b * C + c;
    if (slot < 0 || slot >= N) {
        store_pack<T, VEC>(yo, zero_pack<T, VEC>());
        return;
    }
    T *st = state + (long long)slot * W1 * C + c;
    Pack<T, VEC> win[W], wk[W];
    float out[VEC];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        win[j] = j < W1 ? load_pack<T, VEC>(st + (long long)j * C) : load_pack<T, VEC>(x + (long long)b * x_row + c);
        wk[j] = load_pack<T, VEC>(w + (long long)j * C + c);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float z = bias ? bias[c + i] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) z = fmaf(wk[j].get(i), win[j].get(i), z);
        if (act == DWCONV_ACT_SILU) z *= sigmoid(z);
        out[i] = z;
    }
    store_pack<T, VEC>(yo, Pack<T, VEC>::of(out));
#pragma unroll
    for (int j = 0; j < W1; ++j) store_pack<T, VEC>(st + (long long)j * C, win[j + 1]);
}

template <typename F> cudaError_t with_width(int W, F &&f) {
    switch (W) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 5: return f(std::integral_constant<int, 5>{});
        case 6: return f(std::integral_constant<int, 6>{});
        case 7: return f(std::integral_constant<int, 7>{});
        case 8: return f(std::integral_constant<int, 8>{});
        default: return cudaErrorNotSupported;
    }
}

bool is16(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whole vectors of `bytes` bytes everywhere: channel rows, strides and bases.
bool vector_rows(size_t es, int bytes, int C, std::initializer_list<const void *> bases,
                 std::initializer_list<long long> strides) {
    if ((C * es) % bytes) return false;
    for (const void *p : bases)
        if (!is16(p, bytes)) return false;
    for (long long s : strides)
        if ((s * (long long)es) % bytes) return false;
    return true;
}

void note_call(const char *family) {
    note_launches(1);
    note_kernel(family);
}

// Tokens a forward thread walks: long segments re-read fewer of the W-1 shared
// tokens, but about 2,000 threads an SM have to have work.
int fwd_segment(long long vectors, int T) {
    int seg = 64;
    while (seg > 8 && vectors * ((T + seg - 1) / seg) < 2048LL * sm_count()) seg /= 2;
    return seg;
}

template <typename T, int VEC> cudaError_t fwd_launch(CausalArgs a, cudaStream_t st) {
    const long long nvec = a.C / VEC;
    a.seg = fwd_segment(nvec * a.B, a.T);
    const long long segs = (a.T + a.seg - 1) / a.seg + (a.state_out ? 1 : 0);
    const long long blocks = (nvec * segs + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    return with_width(a.W, [&](auto w) {
        note_call("causal_fwd");
        return launch_after(causal_fwd_kernel<T, VEC, decltype(w)::value>, dim3((unsigned)blocks, a.B), kThreads, 0, st, a);
    });
}

template <typename T, int VEC> cudaError_t bwd_launch(const CausalArgs &a, float *dw, float *db, cudaStream_t st) {
    const int groups = (a.T + a.seg * kRows - 1) / (a.seg * kRows);
    const dim3 grid((a.C / VEC + 31) / 32, groups, a.B);
    return with_width(a.W, [&](auto w) {
        note_call("causal_bwd");
        cudaError_t e = launch_after(causal_bwd_kernel<T, VEC, decltype(w)::value>, grid, dim3(32, kRows), 0, st, a);
        if (e != cudaSuccess) return e;
        const long long taps = (long long)a.W * a.C;
        return launch_split_sums(a.part, groups * a.B, taps + a.C, dw, taps, db, a.C, nullptr, st);
    });
}

}  // namespace

cudaError_t launch_causal_fwd(int B, int T, int C, int W, dwconv_dtype dt, const void *x, long long x_batch,
                              long long x_row, const void *w, const float *bias, int act, const void *state,
                              const int *lengths, void *y, void *state_out, cudaStream_t st) {
    CausalArgs a{};
    a.B = B; a.T = T; a.C = C; a.W = W; a.act = act;
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.lengths = lengths; a.y = y;
    a.state_out = W > 1 ? state_out : nullptr;
    a.x_batch = x_batch; a.x_row = x_row;
    auto run = [&](auto t) {
        using E = decltype(t);
        // four channels a thread: with eight, window and taps left 12 warps an SM
        const bool vec = vector_rows(sizeof(E), 4 * sizeof(E), C, {x, w, state, y, state_out}, {x_batch, x_row});
        return vec ? fwd_launch<E, 4>(a, st) : fwd_launch<E, 1>(a, st);
    };
    switch (dt) {
        case DWCONV_FP32: return run(float{});
        case DWCONV_FP16: return run(__half{});
        default: return run(__nv_bfloat16{});
    }
}

// Tokens a backward thread walks.  A pure function of the shape (the workspace
// holds one slice per kRows segments of a row): the length whose waves of blocks
// take the fewest steps, with the W-1 tokens that a segment re-reads and the
// checked ones at its ends counted as 12 more, on 152 SMs of 4 blocks (8 of
// single channels).  4 x 4096 x 4096 bf16: 114 tokens, 98 us (fp32 132); 16 take
// 162 (166), 64 102 (145), 128 94 (134), 147 92 (142), 256 100 (127), 512 118
// (156): the rule is within 7 % of the best.  2 x 4097 x 2304 bf16: 65 tokens, 35;
// 32 take 40, 128 45.  1 x 777 x 2304 fp16: 8 tokens, 10.6; 32 take 14, 64 19.
int causal_bwd_segment(long long B, long long T, long long C) {
    constexpr long long kLeast = 8;  // only the first segment reaches back before the sequence
    const bool whole = C % 4 == 0;
    const long long slots = 152 * (whole ? 4 : 8), columns = B * ((C + (whole ? 127 : 31)) / (whole ? 128 : 32));
    // Groups of kRows segments a row, at most: none of the shortest length is empty, and no more than eight waves
    // of segments up to 1024 tokens need.
    const long long full = (T + kRows * kLeast - 1) / (kRows * kLeast);
    const long long enough = std::max((T + kRows * 1024 - 1) / (kRows * 1024), 8 * slots / columns + 1);
    const long long most = std::max(std::min(full, enough), 1LL);
    // Of the numbers of groups that take the same waves the largest has the shortest segments: one try a wave.
    long long best = 0, seg = kLeast;
    for (long long groups = 0, waves = (columns + slots - 1) / slots; groups < most; ++waves) {
        if (waves * slots < (groups + 1) * columns) waves = ((groups + 1) * columns + slots - 1) / slots;
        groups = std::min(waves * slots / columns, most);
        const long long s = std::max((T + groups * kRows - 1) / (groups * kRows), kLeast);
        const long long cost = waves * (s + 12);
        if (best == 0 || cost < best) {
            best = cost;
            seg = s;
        }
    }
    return (int)seg;
}
int causal_bwd_slices(long long B, long long T, long long C) {
    const long long group = (long long)causal_bwd_segment(B, T, C) * kRows;
    const long long n = B * ((T + group - 1) / group);
    return n > 0x7FFFFFFFLL ? 0 : (int)n;
}

cudaError_t launch_causal_bwd(int B, int T, int C, int W, dwconv_dtype dt, const void *dy, long long dy_batch,
                              long long dy_row, const void *x, long long x_batch, long long x_row, const void *w,
                              const float *bias, int act, const void *state, const int *lengths, void *dx,
                              void *dstate, float *dw, float *db, float *part, cudaStream_t st) {
    CausalArgs a{};
    a.B = B; a.T = T; a.C = C; a.W = W; a.act = act;
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.lengths = lengths; a.dy = dy;
    a.x_batch = x_batch; a.x_row = x_row; a.dy_batch = dy_batch; a.dy_row = dy_row;
    a.dx = dx; a.dstate = W > 1 ? dstate : nullptr; a.part = part;
    a.seg = causal_bwd_segment(B, T, C);
    auto run = [&](auto t) {
        using E = decltype(t);
        const bool vec = vector_rows(sizeof(E), 4 * sizeof(E), C, {x, w, state, dy, dx, dstate},
                                     {x_batch, x_row, dy_batch, dy_row});
        return vec ? bwd_launch<E, 4>(a, dw, db, st) : bwd_launch<E, 1>(a, dw, db, st);
    };
    switch (dt) {
        case DWCONV_FP32: return run(float{});
        case DWCONV_FP16: return run(__half{});
        default: return run(__nv_bfloat16{});
    }
}

cudaError_t launch_causal_step(int B, int N, int C, int W, dwconv_dtype dt, const void *x, long long x_row,
                               const void *w, const float *bias, int act, void *state, const int *slots, void *y,
                               cudaStream_t st) {
    auto run = [&](auto t, auto vec) {
        using E = decltype(t);
        constexpr int V = decltype(vec)::value;
        const long long blocks = ((long long)B * (C / V) + kThreads - 1) / kThreads;
        if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
        return with_width(W, [&](auto w_) {
            note_call("causal_step");
            return launch_after(causal_step_kernel<E, V, decltype(w_)::value>, dim3((unsigned)blocks), kThreads, 0, st, B,
                                N, C, act, static_cast<const E *>(x), x_row, static_cast<const E *>(w), bias,
                                static_cast<E *>(state), slots, static_cast<E *>(y));
        });
    };
    auto pick = [&](auto t) {
        using E = decltype(t);
        // 8-byte vectors: a step is a few thousand channels, and twice the threads of 16-byte ones
        if (vector_rows(sizeof(E), 4 * sizeof(E), C, {x, w, state, y}, {x_row}))
            return run(t, std::integral_constant<int, 4>{});
        return run(t, std::integral_constant<int, 1>{});
    };
    switch (dt) {
        case DWCONV_FP32: return pick(float{});
        case DWCONV_FP16: return pick(__half{});
        default: return pick(__nv_bfloat16{});
    }
}

}  // namespace dwc
