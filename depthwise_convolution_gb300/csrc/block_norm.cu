// The norms before and after a block, fused with its gate, residual scale and
// residual.  Per row of C values:
//
//   z = post(y) act(gate),   h = residual + scale z,   n = pre(h),
//
// post and pre either x / sqrt(mean x^2 + eps) or (x - mean) / sqrt(var + eps),
// times a weight vector; each part may be absent.  Rows are independent and a
// row's work is a few operations per value, so every pass is bound by memory:
// a group of G threads holds a whole row in registers, each input is read once
// and each output written once.  Means, squares and column sums are fp32.
//
// The backward pass recomputes the forward row instead of reading saved
// statistics or h (the inputs are all in registers anyway):
//   dh' = dh + pre_back(dn w_pre),  dscale = sum dh' z,  dz = dh' scale,
//   dgate = dz post(y) act'(gate),  dp = dz act(gate),  dy = post_back(dp w_post),
// with, for x^ = (x - m) r and u the gradient of x^,
//   back(u) = r (u - x^ mean(u x^) [- mean(u) for the layer norm]).
// Column sums stay in the threads' registers over all rows of a CTA and leave
// it as one slice; the slices are added in a fixed order by a second kernel.
#include <algorithm>

#include "mixer_common.cuh"
#include "tma.cuh"

namespace dwc {

namespace {

constexpr int NV_MAX = 2;  // sums that one exchange carries

// Row inputs, in the order of the strides at the interface.
enum { IN_Y, IN_RESIDUAL, IN_GATE, IN_DH, IN_DN, kInputs };

struct NormArgs {
    long long rows;
    long long inner;  // row r is (r / inner, r % inner)
    int C, G;         // row width, threads per row
    int flat;         // rows are evenly spaced in every tensor
    int stages;       // rounds of rows that the ring holds
    int layer, act;
    float eps, inv_c;
    int want;         // column sums wanted: 1 w_post, 2 scale, 4 w_pre
    const void *in[kInputs];      // null: absent
    long long st[kInputs][2];     // outer, inner row strides in elements
    const float *w_post, *scale, *w_pre;
    void *h, *n, *dy, *dresidual, *dgate;
    float *part;  // [CTAs][3][C]
    unsigned *err;
    __device__ __forceinline__ bool has(int t) const { return in[t] != nullptr; }
};

// (outer, inner) index of row r; (0, r) where one stride steps through all rows
// of every tensor, which spares the division.
template <typename T> __device__ __forceinline__ const T *row_at(const NormArgs &a, int t, long long r) {
    const long long o = a.flat ? 0 : r / a.inner, i = a.flat ? r : r - o * a.inner;
    return static_cast<const T *>(a.in[t]) + o * a.st[t][0] + i * a.st[t][1];
}

// Sums over the G threads of a row group (a power of two up to 512; every thread
// of the CTA takes part), the same value in all of them; NV sums at once.
// Groups of more than a warp exchange their warps' sums through shared memory,
// whose two halves alternate so that one barrier a sum is enough.  A row's sums
// cost as much as its values do: no divisions and no loops here.
struct Group {
    float (&red)[2][NV_MAX][32];
    int G, phase, put, get;
    bool any;  // this lane reads another warp's sum
    __device__ __forceinline__ Group(float (&red_)[2][NV_MAX][32], int G_) : red(red_), G(G_), phase(0) {
        const int warps = G / 32, lane = threadIdx.x % 32;
        put = threadIdx.x / 32;
        any = (lane & 15) < warps;
        get = any ? (put & ~(warps - 1)) + (lane & 15) : 0;
    }
    template <int NV, int O> static __device__ __forceinline__ void fold(float (&v)[NV]) {
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] += __shfl_xor_sync(0xFFFFFFFFu, v[q], O);
    }
    template <int NV> __device__ __forceinline__ void sum(float (&v)[NV]) {
        if (G >= 32) fold<NV, 16>(v);
        if (G >= 16) fold<NV, 8>(v);
        if (G >= 8) fold<NV, 4>(v);
        fold<NV, 2>(v);
        fold<NV, 1>(v);
        if (G <= 32) return;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int q = 0; q < NV; ++q) red[phase][q][put] = v[q];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] = any ? red[phase][q][get] : 0.f;
        fold<NV, 8>(v);
        fold<NV, 4>(v);
        fold<NV, 2>(v);
        fold<NV, 1>(v);
        phase ^= 1;
    }
};

// act(gate) and its slope; with_act compiles a loop over a row for each act (a
// choice per value took half of the backward pass's instructions).
template <int ACT> __device__ __forceinline__ float gate_value(float g) {
    if (ACT == DWCONV_GATE_NONE) return g;
    const float s = sigmoid(g);
    return ACT == DWCONV_GATE_SIGMOID ? s : g * s;
}
template <int ACT> __device__ __forceinline__ void gate_both(float g, float &value, float &slope) {
    value = g;
    slope = 1.f;
    if (ACT == DWCONV_GATE_NONE) return;
    const float s = sigmoid(g);
    value = ACT == DWCONV_GATE_SIGMOID ? s : g * s;
    slope = ACT == DWCONV_GATE_SIGMOID ? s * (1.f - s) : s * fmaf(g, 1.f - s, 1.f);
}
template <typename F> __device__ __forceinline__ void with_act(int act, F &&f) {
    if (act == DWCONV_GATE_SILU) f(std::integral_constant<int, DWCONV_GATE_SILU>{});
    else if (act == DWCONV_GATE_SIGMOID) f(std::integral_constant<int, DWCONV_GATE_SIGMOID>{});
    else f(std::integral_constant<int, DWCONV_GATE_NONE>{});
}

// A thread's columns of a row of any tensor, and of the weight vectors; `ends`: the
// row's end where a vector of its lies beyond.
template <int VEC, int NV> struct Cols {
    int c[NV];
    bool in[NV];
    __device__ __forceinline__ Cols(const NormArgs &a, int g, bool ends = false) {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            c[q] = (q * a.G + g) * VEC;
            in[q] = c[q] < a.C;
            if (ends) c[q] = min(c[q], a.C);
        }
    }
    // One vector's worth of a weight vector (ones where it is absent); all CTAs of
    // an SM share it in L1.
    __device__ __forceinline__ Pack<float, VEC> weight(const float *w, int q) const {
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 1.f;
        if (!w) return Pack<float, VEC>::of(v);
        Pack<float, VEC> r = zero_pack<float, VEC>();
        if (!in[q]) return r;
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(w + c[q] + i);
                r.w[i] = u.x; r.w[i + 1] = u.y; r.w[i + 2] = u.z; r.w[i + 3] = u.w;
            }
        } else {
            r.v = w[c[q]];
        }
        return r;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, bool on, Pack<T, VEC> (&v)[NV]) const {
#pragma unroll
        for (int q = 0; q < NV; ++q)
            v[q] = on && in[q] ? load_pack<T, VEC>(row + c[q]) : zero_pack<T, VEC>();
    }
    template <typename T> __device__ __forceinline__ void store(T *row, bool on, const float (&x)[NV][VEC]) const {
        if (!on) return;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const Pack<T, VEC> out = Pack<T, VEC>::of(x[q]);
            if (in[q]) store_pack<T, VEC>(row + c[q], out);
        }
    }
};

// A weight vector (the product of two) at the thread's columns: HOLD keeps it in registers for all
// rows, otherwise it is read for each.
template <int VEC, int NV, bool HOLD> struct Weight {
    const float *w, *by;
    Pack<float, VEC> held[HOLD ? NV : 1];
    __device__ __forceinline__ Weight(const Cols<VEC, NV> &cols, const float *w_, const float *by_ = nullptr)
        : w(w_), by(by_) {
        if (HOLD) {
#pragma unroll
            for (int q = 0; q < NV; ++q) held[q] = read(cols, q);
        }
    }
    __device__ __forceinline__ Pack<float, VEC> read(const Cols<VEC, NV> &cols, int q) const {
        const Pack<float, VEC> v = cols.weight(w, q);
        if (!by) return v;
        const Pack<float, VEC> u = cols.weight(by, q);
        float x[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = v.get(i) * u.get(i);
        return Pack<float, VEC>::of(x);
    }
    __device__ __forceinline__ Pack<float, VEC> at(const Cols<VEC, NV> &cols, int q) const {
        if constexpr (HOLD) return held[q];
        else return read(cols, q);
    }
};

// The same out of shared memory, where the backward pass, which has no
// registers left for them, keeps its weight vectors: ones where a vector is
// absent, zeros beyond the row.  Beside a ring all columns beyond share one vector
// of zeros behind the row; elsewhere, where there is room, each has its own (the
// widest rows' form spills, and the shared one's addresses cost it 4 %).
template <int VEC, int NV, bool RING> struct SharedWeight {
    const float *w;
    static __host__ __device__ int size(int C, int G) { return RING ? C + VEC : G * NV * VEC; }
    __device__ __forceinline__ SharedWeight(const NormArgs &a, const float *from, float *to) : w(to) {
        for (int c = threadIdx.x; c < size(a.C, a.G); c += blockDim.x) to[c] = c < a.C ? (from ? from[c] : 1.f) : 0.f;
    }
    __device__ __forceinline__ Pack<float, VEC> at(const Cols<VEC, NV> &cols, int q) const {
        if constexpr (VEC == 1) {
            return Pack<float, 1>{w[cols.c[q]]};
        } else {
            Pack<float, VEC> r;
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(w + cols.c[q] + i);
                r.w[i] = u.x; r.w[i + 1] = u.y; r.w[i + 2] = u.z; r.w[i + 3] = u.w;
            }
            return r;
        }
    }
};

// Mean (0 for the rms norm) and reciprocal root of a row held as x[NV][VEC],
// zero outside the row.  The variance is summed about the mean: no cancellation
// for a large mean.
template <int NV, int VEC>
__device__ __forceinline__ void row_stats(const float (&x)[NV][VEC], const Cols<VEC, NV> &cols, const NormArgs &a,
                                          Group &group, float &mean, float &rstd) {
    float s[1] = {0.f};
    mean = 0.f;
    if (a.layer) {
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] += x[q][i];
        group.sum<1>(s);
        mean = s[0] * a.inv_c;
        s[0] = 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if (cols.in[q])
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[0] = fmaf(x[q][i] - mean, x[q][i] - mean, s[0]);
    } else {
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = fmaf(x[q][i], x[q][i], s[0]);
    }
    group.sum<1>(s);
    rstd = rsqrtf(fmaf(s[0], a.inv_c, a.eps));
}

// x -> (x - mean) rstd; the rms norm has no mean to take off.
template <int NV, int VEC>
__device__ __forceinline__ void normalise(float (&x)[NV][VEC], const NormArgs &a, float mean, float rstd) {
    if (a.layer) {
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[q][i] = (x[q][i] - mean) * rstd;
    } else {
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[q][i] *= rstd;
    }
}

// The walk of a CTA over its rows: round k is rows r0 .. r0 + per - 1, a group
// of G threads each.
struct Walk {
    long long r0, step;
    int per, mine, rounds;
    __device__ __forceinline__ Walk(const NormArgs &a) {
        per = blockDim.x / a.G;
        mine = threadIdx.x / a.G;
        step = (long long)gridDim.x * per;
        r0 = (long long)blockIdx.x * per;
        rounds = (int)((a.rows - r0 + step - 1) / step);  // a CTA has at least one row
    }
    __device__ __forceinline__ int live(const NormArgs &a, int k) const {
        const long long left = a.rows - (r0 + k * step);
        return left < per ? (int)left : per;
    }
};

// Whole-vector rows come through a ring of 2 or 3 rounds in shared memory,
// filled by bulk copies (one for all rows of a round where they are dense):
// with loads straight into registers a CTA had nothing on its way while it
// exchanged sums and stored (2.9 TB/s of 6.8).
constexpr int kMostStages = 3;
struct RowRing {
    uint64_t full[kMostStages], empty[kMostStages];
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int s = 0; s < kMostStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], blockDim.x / 32);
        }
        mbar_fence_init();
    }
};
__device__ __forceinline__ void bulk_rows(void *dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// Reads the rows of the walk's rounds, one round after the other: from the ring
// (RING) or straight from memory.
template <typename T, bool RING> struct Rows {
    const NormArgs &a;
    const Walk &walk;
    RowRing &ring;
    unsigned char *smem;
    const unsigned bytes, slot, stage;  // of a row, of one tensor's rows, of a round
    const long long own;                // of this thread's row in a round
    unsigned here, there;               // offsets of the stage being read and of the one being filled
    int at, turn, next, lap;            // stage and parity being read; stage and lap being filled
    bool ok;                            // false once a wait gave up: the kernel goes on without waiting
    bool apart;                         // rows of some tensor are not dense: a copy each
    const T *from;                      // lane t of the first warp: tensor t where its rows are dense
    unsigned to;                        // its place in a stage
    __device__ __forceinline__ Rows(const NormArgs &a_, const Walk &w, RowRing &r, unsigned char *s, int inputs)
        : a(a_), walk(w), ring(r), smem(s), bytes(a_.C * sizeof(T)), slot(w.per * bytes), stage(slot * inputs),
          own((long long)w.mine * a_.C), here(0), there(0), at(0), turn(0), next(0), lap(0), ok(true), apart(false),
          from(nullptr), to(0) {
        if (!RING) return;
        unsigned offset = 0;
#pragma unroll
        for (int t = 0; t < kInputs; ++t) {
            if (!a.has(t)) continue;
            const bool dense = a.flat && a.st[t][1] == a.C;
            if (!dense) apart = true;
            if (dense && threadIdx.x == t) {
                from = static_cast<const T *>(a.in[t]);
                to = offset;
            }
            offset += slot;
        }
        if (threadIdx.x == 0) ring.init();
        __syncthreads();
        for (int k = 0; k < a.stages; ++k) fetch(k);
    }
    // Starts the copies of round k, once the round before it there has been read.
    __device__ __forceinline__ void fetch(int k) {
        if (!RING || threadIdx.x >= 32 || k >= walk.rounds) return;
        const int n = walk.live(a, k);
        uint64_t *bar = &ring.full[next];
        if (ok && lap > 0 && !mbar_wait(&ring.empty[next], (lap - 1) & 1)) lost();
        unsigned char *stage_at = smem + there;
        there += stage;
        if (++next == a.stages) {
            next = 0;
            there = 0;
            ++lap;
        }
        if (!ok) return;
        if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, n == walk.per ? stage : stage / slot * n * bytes);
        __syncwarp();
        const long long r = walk.r0 + k * walk.step;
        if (from) bulk_rows(stage_at + to, from + r * a.C, n * bytes, bar);
        if (!apart) return;
#pragma unroll
        for (int t = 0; t < kInputs; ++t) {
            if (!a.has(t)) continue;
            if (!a.flat || a.st[t][1] != a.C)
                for (int i = threadIdx.x; i < n; i += 32)
                    bulk_rows(stage_at + i * bytes, row_at<T>(a, t, r + i), bytes, bar);
            stage_at += slot;
        }
    }
    __device__ __forceinline__ void lost() {
        report_timeout(a.err);
        ok = false;
    }
    __device__ __forceinline__ void wait() {
        if (RING && ok && !mbar_wait(&ring.full[at], turn)) lost();
    }
    __device__ __forceinline__ void done() {  // this warp needs the round no more
        if (!RING) return;
        __syncwarp();
        if (threadIdx.x % 32 == 0) mbar_arrive(&ring.empty[at]);
        here += stage;
        if (++at == a.stages) {
            at = 0;
            here = 0;
            turn ^= 1;
        }
    }
    // This thread's row of the round being read (row r) of tensor t, the nth of those present.
    __device__ __forceinline__ const T *row(long long r, int t, int nth) const {
        if (RING) return reinterpret_cast<const T *>(smem + here + nth * slot) + own;
        return row_at<T>(a, t, r);
    }
};

// A thread's part of a row of one tensor: with the ring it is read where it is
// used, as often as that is, and holds no registers.
template <typename T, int VEC, int NV, bool RING> struct Input {
    const T *row;
    bool on;
    Pack<T, VEC> v[RING ? 1 : NV];
    __device__ __forceinline__ Input(const Cols<VEC, NV> &cols, const T *row_, bool on_) : row(row_), on(on_) {
        if constexpr (!RING) cols.load(row, on, v);
    }
    __device__ __forceinline__ Pack<T, VEC> at(const Cols<VEC, NV> &cols, int q) const {
        if constexpr (!RING) return v[q];
        else return on && cols.in[q] ? load_pack<T, VEC>(row + cols.c[q]) : zero_pack<T, VEC>();
    }
};

// Forward.  A thread holds 16 values of a row and the weights for them.  What
// bounds it is instructions (about 30 a value at 4096 columns, half of them for
// the row: sums, addresses, barriers): 16384 rows of 4096 in bf16 with residual,
// scale and both norms take 97 us, 5.55 TB/s; with three weight vectors and the
// inputs in registers 109, with 32 values a thread and the weights read from L1
// for each row 118, and with divisions and loops in the sums 132.  Three CTAs of
// 256 threads an SM instead of two spill at 80 registers: 127.
template <typename T, int VEC, int NV, int MAXT, bool RING>
__global__ void __launch_bounds__(MAXT, MAXT == 128 ? 4 : 1) block_norm_fwd_kernel(NormArgs a) {
    __shared__ float red[2][NV_MAX][32];
    __shared__ RowRing ring;
    extern __shared__ __align__(128) unsigned char stages[];
    after_previous();
    Group group(red, a.G);
    const Cols<VEC, NV> cols(a, threadIdx.x % a.G);
    constexpr bool HOLD = NV * VEC <= 16;
    // w_post and the residual scale meet in one product
    const Weight<VEC, NV, HOLD> post(cols, a.w_post, a.scale), pre(cols, a.w_pre);
    const Walk walk(a);
    const int nr = 1, ng = nr + a.has(IN_RESIDUAL);
    Rows<T, RING> rows(a, walk, ring, stages, ng + a.has(IN_GATE));
    long long r = walk.r0 + walk.mine, to = r * a.C;
    for (int k = 0; k < walk.rounds; ++k, r += walk.step, to += walk.step * a.C) {
        const bool live = r < a.rows;
        rows.wait();
        using In = Input<T, VEC, NV, RING>;
        const In yv(cols, rows.row(r, IN_Y, 0), live),
            rv(cols, rows.row(r, IN_RESIDUAL, nr), live && a.has(IN_RESIDUAL)),
            gv(cols, rows.row(r, IN_GATE, ng), live && a.has(IN_GATE));
        float x[NV][VEC];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const Pack<T, VEC> v = yv.at(cols, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[q][i] = v.get(i);
        }
        float mean, rstd;
        if (a.w_post) {
            row_stats<NV, VEC>(x, cols, a, group, mean, rstd);
            normalise<NV, VEC>(x, a, mean, rstd);
        }
        if (a.w_post || a.scale) {
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const Pack<float, VEC> w = post.at(cols, q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[q][i] *= w.get(i);
            }
        }
        if (a.has(IN_GATE))
            with_act(a.act, [&](auto act) {
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const Pack<T, VEC> v = gv.at(cols, q);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) x[q][i] *= gate_value<decltype(act)::value>(v.get(i));
                }
            });
        if (a.has(IN_RESIDUAL)) {
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const Pack<T, VEC> v = rv.at(cols, q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[q][i] += v.get(i);
            }
        }
        rows.done();
        cols.store(static_cast<T *>(a.h) + to, live, x);
        rows.fetch(k + a.stages);
        if (!a.w_pre) continue;
        row_stats<NV, VEC>(x, cols, a, group, mean, rstd);
        normalise<NV, VEC>(x, a, mean, rstd);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const Pack<float, VEC> w = pre.at(cols, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[q][i] *= w.get(i);
        }
        cols.store(static_cast<T *>(a.n) + to, live, x);
    }
}

// u -> back(u) for the normalised row hat: needs mean(u hat) and, for the layer
// norm, mean(u); both in one exchange.  u is zero outside the row.
template <int NV, int VEC>
__device__ __forceinline__ void norm_back(float (&u)[NV][VEC], const float (&hat)[NV][VEC], const NormArgs &a,
                                          float rstd, Group &group) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[0] = fmaf(u[q][i], hat[q][i], s[0]);
    if (a.layer) {
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[1] += u[q][i];
        group.sum<2>(s);
    } else {
        float only[1] = {s[0]};
        group.sum<1>(only);
        s[0] = only[0];
    }
    const float c0 = -rstd * s[0] * a.inv_c, c1 = -rstd * s[1] * a.inv_c;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) u[q][i] = fmaf(u[q][i], rstd, fmaf(hat[q][i], c0, c1));
}

// Backward: CTAs stay like the forward's, with their column sums in registers,
// the weights in shared memory and the inputs read from the ring where they are
// used.  8192 rows of 2048 in bf16 with all parts and a sigmoid gate take 103 us
// (2.6 TB/s): four sums of a row follow one another, on 12 warps an SM, with some
// 95 instructions a value, half of them arithmetic (the gate is evaluated twice:
// no registers are left to keep it).  Choices per value took 129; a fourth
// CTA an SM spills at 128 registers (133), except with eight values a thread
// (fp32, 16384 x 768: 81 us instead of 97).  From 256 threads a row on 128
// registers are the limit of 512 threads: 16-bit rows of more than 2048 columns
// spill a little (8192 x 4096 bf16 292 us, fp32 196; 4096 x 7040 218), the widest
// rows' form a lot (4096 x 8192 bf16 515, fp32 658; 2048 x 16384 522, 668).
template <typename T, int VEC, int NV, int MAXT, bool RING>
__global__ void __launch_bounds__(MAXT, MAXT == 128 ? (NV * VEC <= 8 ? 4 : 3) : 1) block_norm_bwd_kernel(NormArgs a) {
    __shared__ float red[2][NV_MAX][32];
    __shared__ RowRing ring;
    extern __shared__ __align__(128) unsigned char smem[];  // weights, then the ring; afterwards [rows per CTA][C] column sums
    float *shared_cols = reinterpret_cast<float *>(smem), *weights = shared_cols;
    const int width = SharedWeight<VEC, NV, RING>::size(a.C, a.G);
    unsigned char *stages = smem + 3 * width * sizeof(float);
    after_previous();
    Group group(red, a.G);
    const Cols<VEC, NV> cols(a, threadIdx.x % a.G, RING);
    const SharedWeight<VEC, NV, RING> post(a, a.w_post, weights), scale(a, a.scale, weights + width),
        pre(a, a.w_pre, weights + 2 * width);
    __syncthreads();
    float s_post[NV][VEC], s_scale[NV][VEC], s_pre[NV][VEC];
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s_post[q][i] = s_scale[q][i] = s_pre[q][i] = 0.f;
    const Walk walk(a);
    const bool with_n = a.has(IN_DN);
    const int nr = 1, ng = nr + a.has(IN_RESIDUAL), nh = ng + a.has(IN_GATE), nn = nh + a.has(IN_DH);
    Rows<T, RING> rows(a, walk, ring, stages, nn + with_n);
    long long r = walk.r0 + walk.mine, to = r * a.C;
    for (int k = 0; k < walk.rounds; ++k, r += walk.step, to += walk.step * a.C) {
        const bool live = r < a.rows;
        rows.wait();
        using In = Input<T, VEC, NV, RING>;
        const In yv(cols, rows.row(r, IN_Y, 0), live), rv(cols, rows.row(r, IN_RESIDUAL, nr), live && a.has(IN_RESIDUAL)),
            gv(cols, rows.row(r, IN_GATE, ng), live && a.has(IN_GATE)), hv(cols, rows.row(r, IN_DH, nh), live && a.has(IN_DH)),
            nv(cols, rows.row(r, IN_DN, nn), live && with_n);
        // hat: the normalised row (or the row itself); z: what the residual scale multiplies
        float hat[NV][VEC], z[NV][VEC], d[NV][VEC];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const Pack<T, VEC> v = yv.at(cols, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) hat[q][i] = v.get(i);
        }
        float mean = 0.f, rstd = 1.f;
        if (a.w_post) {
            row_stats<NV, VEC>(hat, cols, a, group, mean, rstd);
            if (!live) rstd = 0.f;  // zeros stand in for a missing row: nothing for the column sums, whatever eps
            normalise<NV, VEC>(hat, a, mean, rstd);
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const Pack<float, VEC> w = post.at(cols, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                z[q][i] = hat[q][i] * w.get(i);
                d[q][i] = 0.f;
            }
        }
        if (a.has(IN_GATE))
            with_act(a.act, [&](auto act) {
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const Pack<T, VEC> v = gv.at(cols, q);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) z[q][i] *= gate_value<decltype(act)::value>(v.get(i));
                }
            });
        if (with_n) {
            float x[NV][VEC];
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const Pack<float, VEC> w = scale.at(cols, q);
                const Pack<T, VEC> from = rv.at(cols, q), v = nv.at(cols, q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    x[q][i] = fmaf(z[q][i], w.get(i), from.get(i));
                    d[q][i] = v.get(i);
                }
            }
            float hm, hr;
            row_stats<NV, VEC>(x, cols, a, group, hm, hr);
            if (!live) hr = 0.f;
            normalise<NV, VEC>(x, a, hm, hr);
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const Pack<float, VEC> w = pre.at(cols, q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    s_pre[q][i] = fmaf(d[q][i], x[q][i], s_pre[q][i]);
                    d[q][i] *= w.get(i);
                }
            }
            norm_back<NV, VEC>(d, x, a, hr, group);
        }
        if (a.has(IN_DH)) {
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const Pack<T, VEC> v = hv.at(cols, q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[q][i] += v.get(i);
            }
        }
        if (a.dresidual) cols.store(static_cast<T *>(a.dresidual) + to, live, d);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const Pack<float, VEC> w = scale.at(cols, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s_scale[q][i] = fmaf(d[q][i], z[q][i], s_scale[q][i]);
                d[q][i] *= w.get(i);
            }
        }
        if (a.has(IN_GATE)) {
            with_act(a.act, [&](auto act) {
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const Pack<float, VEC> w = post.at(cols, q);
                    const Pack<T, VEC> v = gv.at(cols, q);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        float value, slope;
                        gate_both<decltype(act)::value>(v.get(i), value, slope);
                        z[q][i] = d[q][i] * hat[q][i] * w.get(i) * slope;  // dgate
                        d[q][i] *= value;
                    }
                }
            });
            if (a.dgate) cols.store(static_cast<T *>(a.dgate) + to, live, z);
        }
        rows.done();
        if (a.w_post) {
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const Pack<float, VEC> w = post.at(cols, q);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    s_post[q][i] = fmaf(d[q][i], hat[q][i], s_post[q][i]);
                    d[q][i] *= w.get(i);
                }
            }
            norm_back<NV, VEC>(d, hat, a, rstd, group);
        }
        cols.store(static_cast<T *>(a.dy) + to, live, d);
        rows.fetch(k + a.stages);
    }
    // Columns over the CTA's row slots, in slot order, one vector at a time.
    float *part = a.part + (long long)blockIdx.x * 3 * a.C;
    auto leave = [&](const float(&s)[NV][VEC], float *to) {
        if (walk.per == 1) {
#pragma unroll
            for (int q = 0; q < NV; ++q)
                if (cols.in[q])
#pragma unroll
                    for (int i = 0; i < VEC; ++i) to[cols.c[q] + i] = s[q][i];
            return;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if (cols.in[q])
#pragma unroll
                for (int i = 0; i < VEC; ++i) shared_cols[walk.mine * a.C + cols.c[q] + i] = s[q][i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            float t = shared_cols[c];
            for (int p = 1; p < walk.per; ++p) t += shared_cols[p * a.C + c];
            to[c] = t;
        }
    };
    if (a.want & 1) leave(s_post, part);
    if (a.want & 2) leave(s_scale, part + a.C);
    if (a.want & 4) leave(s_pre, part + 2LL * a.C);
}

constexpr int kSumWarps = 32;

// Column sums over slices: a block takes 32 columns, its warps the slices in
// turn (eight loads in flight), and the warps' sums are added in warp order.
__global__ void __launch_bounds__(32 * kSumWarps)
    split_sums_kernel(const float *part, int Z, long long count, float *out0, long long n0, float *out1,
                      long long n1, float *out2) {
    __shared__ float acc[kSumWarps][32];
    const int lane = threadIdx.x % 32, r = threadIdx.x / 32, warps = blockDim.x / 32;
    const long long i = blockIdx.x * 32LL + lane;
    after_previous();
    float *to = i < n0 ? out0 : i < n0 + n1 ? out1 : out2;
    const long long at = i < n0 ? i : i < n0 + n1 ? i - n0 : i - n0 - n1;
    const bool on = i < count && to;
    float sum = 0.f;
    if (on) {
        int z = r;
        for (; z + 7 * warps < Z; z += 8 * warps) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = part[(long long)(z + q * warps) * count + i];
#pragma unroll
            for (int q = 0; q < 8; ++q) sum += v[q];
        }
        float v[7];
#pragma unroll
        for (int q = 0; q < 7; ++q) v[q] = z + q * warps < Z ? part[(long long)(z + q * warps) * count + i] : 0.f;
#pragma unroll
        for (int q = 0; q < 7; ++q) sum += v[q];
    }
    acc[r][lane] = sum;
    __syncthreads();
    if (r == 0 && on) {
        float t = acc[0][lane];
        for (int q = 1; q < warps; ++q) t += acc[q][lane];
        to[at] = t;
    }
}

// Threads per row: the smallest power of two that holds the row in `most`
// vectors a thread.
int group_size(int vectors, int most) {
    int G = 4;
    while (G * most < vectors) G *= 2;
    return G;
}

// Shared memory of a round of `per` rows of every input.
template <typename T> size_t round_bytes(const NormArgs &a, int per) {
    size_t inputs = 0;
    for (const void *p : a.in) inputs += p != nullptr;
    return inputs * per * a.C * sizeof(T);
}

// CTAs of one wave, at most one per `per` rows.
template <typename K> cudaError_t wave(K kern, int threads, size_t smem, long long rows, int per, long long &grid) {
    int per_sm = 0;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), threads, smem, &per_sm);
    grid = std::min<long long>((rows + per - 1) / per, (long long)std::max(1, per_sm) * plan_sms(true));
    return e;
}

template <typename T, int VEC, int NV, int MAXT, bool RING>
cudaError_t fwd_run(const NormArgs &a, int threads, cudaStream_t st) {
    auto kern = block_norm_fwd_kernel<T, VEC, NV, MAXT, RING>;
    long long grid = 0;
    const size_t smem = RING ? a.stages * round_bytes<T>(a, threads / a.G) : 0;
    const cudaError_t e = wave(kern, threads, smem, a.rows, threads / a.G, grid);
    if (e != cudaSuccess) return e;
    note_launches(1);
    note_kernel("block_norm_fwd");
    return launch_after(kern, dim3((unsigned)grid), threads, smem, st, a);
}

template <typename T, int VEC, int NV, int MAXT, bool RING>
cudaError_t bwd_run(const NormArgs &a, int threads, float *dwp, float *dsc, float *dwr, cudaStream_t st) {
    const int per = threads / a.G;
    const size_t smem = std::max(3 * sizeof(float) * SharedWeight<VEC, NV, RING>::size(a.C, a.G) + (RING ? a.stages * round_bytes<T>(a, per) : 0),
                                 per > 1 ? (size_t)per * a.C * sizeof(float) : 0);
    auto kern = block_norm_bwd_kernel<T, VEC, NV, MAXT, RING>;
    long long grid = 0;
    cudaError_t e = wave(kern, threads, smem, a.rows, per, grid);
    if (e != cudaSuccess) return e;
    grid = std::min<long long>(grid, block_norm_slices(a.rows, a.C));
    note_launches(1);
    note_kernel("block_norm_bwd");
    e = launch_after(kern, dim3((unsigned)grid), threads, smem, st, a);
    if (e != cudaSuccess || !a.want) return e;
    return launch_split_sums(a.part, (int)grid, 3LL * a.C, dwp, a.C, dsc, a.C, dwr, st);
}

// Vectors a thread takes of a row.  FEW where there are rows for the whole
// machine (16 values forward, with the weights in registers; 32 bytes backward,
// with the column sums), in CTAs of 128 threads, which narrow rows share, or of
// up to 512.  One, straight from memory and a CTA a row, where all rows together
// are at most 512 threads an SM and a call is a chain of latencies: 7 rows of 768
// in fp32 take 5.2 us instead of 15.4, 152 rows of 4096 in bf16 9.3 instead of
// 10.4, and 304 rows of 4096, beyond the rule, would take 12.4 instead of 11.4.
// MOST, without a ring, for the widest rows and those whose ring has no room
// beside `fixed` bytes.
template <typename T, int VEC, int FEW, typename F> cudaError_t with_shape(NormArgs &a, size_t fixed, F &&f) {
    constexpr bool RING = VEC > 1;
    constexpr int MOST = kMaxNormWidth / 512 / VEC;
    const int nvec = (a.C + VEC - 1) / VEC;
    auto fits = [&](int nv, int most, int threads) {
        a.G = group_size(nvec, nv);
        if (a.G > most) return false;
        const size_t round = round_bytes<T>(a, std::max(threads, a.G) / a.G);
        // three rounds while that leaves room for four CTAs an SM
        a.stages = 3 * round <= 56 * 1024 ? 3 : 2;
        return !RING || a.stages * round + fixed <= 224 * 1024;
    };
    using std::integral_constant;
    using Ring = std::bool_constant<RING>;
    if ((a.G = group_size(nvec, 1)) <= 512 && a.rows * a.G <= 512LL * plan_sms(true))
        return f(integral_constant<int, 1>{}, integral_constant<int, 512>{}, std::false_type{}, std::max(a.G, 32));
    if (fits(FEW, 128, 128)) return f(integral_constant<int, FEW>{}, integral_constant<int, 128>{}, Ring{}, 128);
    if (fits(FEW, 512, 0)) return f(integral_constant<int, FEW>{}, integral_constant<int, 512>{}, Ring{}, a.G);
    a.G = group_size(nvec, MOST);
    return f(integral_constant<int, MOST>{}, integral_constant<int, 512>{}, std::false_type{}, std::max(a.G, 32));
}

template <typename T, int VEC> cudaError_t fwd_launch(NormArgs a, cudaStream_t st) {
    return with_shape<T, VEC, 16 / VEC>(a, 0, [&](auto nv, auto most, auto ring, int threads) {
        return fwd_run<T, VEC, decltype(nv)::value, decltype(most)::value, decltype(ring)::value>(a, threads, st);
    });
}

template <typename T, int VEC>
cudaError_t bwd_launch(NormArgs a, float *dwp, float *dsc, float *dwr, cudaStream_t st) {
    return with_shape<T, VEC, (VEC == 1 ? 8 : 2)>(a, 3 * sizeof(float) * (a.C + VEC), [&](auto nv, auto most, auto ring, int threads) {
        return bwd_run<T, VEC, decltype(nv)::value, decltype(most)::value, decltype(ring)::value>(a, threads, dwp, dsc, dwr,
                                                                                                 st);
    });
}

// Whole 16-byte vectors in every row of every tensor, and in the weights.
bool vector_rows(const NormArgs &a, size_t es) {
    if ((a.C * es) % 16) return false;
    const void *bases[] = {a.h, a.n, a.dy, a.dresidual, a.dgate, a.w_post, a.scale, a.w_pre};
    for (const void *p : bases)
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    for (int t = 0; t < kInputs; ++t) {
        if (reinterpret_cast<uintptr_t>(a.in[t]) % 16) return false;
        for (long long s : a.st[t])
            if ((s * (long long)es) % 16) return false;
    }
    return true;
}

// Inputs with their strides (null strides: dense); absent ones count as dense.
void set_inputs(NormArgs &a, long long rows_outer, std::initializer_list<const void *> in, const long long *strides) {
    int t = 0;
    a.flat = 1;
    for (const void *p : in) {
        a.in[t] = p;
        a.st[t][0] = p && strides ? strides[2 * t] : a.inner * a.C;
        a.st[t][1] = p && strides ? strides[2 * t + 1] : a.C;
        if (rows_outer > 1 && a.st[t][0] != a.inner * a.st[t][1]) a.flat = 0;
        ++t;
    }
    a.err = device_error_word();
}

NormArgs make_args(long long rows_outer, int rows_inner, int C, int layer, int act, float eps) {
    NormArgs a{};
    a.rows = rows_outer * rows_inner; a.inner = rows_inner; a.C = C;
    a.layer = layer; a.act = act; a.eps = eps; a.inv_c = 1.f / C;
    return a;
}
}  // namespace

// Slices of the backward pass's column sums: the CTAs of one wave at most (16
// of 128 threads an SM), never more than there are rows.
int block_norm_slices(long long rows, int C) {
    (void)C;
    return (int)std::min<long long>(rows, 16LL * kPlanMaxSms);
}

cudaError_t launch_split_sums(const float *part, int Z, long long count, float *out0, long long n0, float *out1,
                              long long n1, float *out2, cudaStream_t st) {
    const long long blocks = (count + 31) / 32;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const int warps = Z > 128 ? kSumWarps : 8;  // few slices: more blocks an SM
    note_launches(1);
    return launch_after(split_sums_kernel, dim3((unsigned)blocks), 32 * warps, 0, st, part, Z, count, out0, n0, out1, n1,
                        out2);
}

cudaError_t launch_block_norm_fwd(long long rows_outer, int rows_inner, int C, dwconv_dtype dt, int layer, int act,
                                  float eps, const void *y, const void *residual, const void *gate,
                                  const long long *strides, const float *w_post, const float *scale,
                                  const float *w_pre, void *h, void *n, cudaStream_t st) {
    NormArgs a = make_args(rows_outer, rows_inner, C, layer, act, eps);
    set_inputs(a, rows_outer, {y, residual, gate, nullptr, nullptr}, strides);
    a.w_post = w_post; a.scale = scale; a.w_pre = w_pre;
    a.h = h; a.n = n;
    auto run = [&](auto t) {
        using E = decltype(t);
        constexpr int V = 16 / sizeof(E);
        return vector_rows(a, sizeof(E)) ? fwd_launch<E, V>(a, st) : fwd_launch<E, 1>(a, st);
    };
    switch (dt) {
        case DWCONV_FP32: return run(float{});
        case DWCONV_FP16: return run(__half{});
        default: return run(__nv_bfloat16{});
    }
}

cudaError_t launch_block_norm_bwd(long long rows_outer, int rows_inner, int C, dwconv_dtype dt, int layer, int act,
                                  float eps, const void *y, const void *residual, const void *gate, const void *dh,
                                  const void *dn, const long long *strides, const float *w_post, const float *scale,
                                  const float *w_pre, void *dy, void *dresidual, void *dgate, float *dw_post,
                                  float *dscale, float *dw_pre, float *part, cudaStream_t st) {
    NormArgs a = make_args(rows_outer, rows_inner, C, layer, act, eps);
    // the residual matters only through the norm of h
    set_inputs(a, rows_outer, {y, dn ? residual : nullptr, gate, dh, dn}, strides);
    a.w_post = w_post; a.scale = scale; a.w_pre = w_pre;
    a.dy = dy; a.dresidual = dresidual; a.dgate = gate ? dgate : nullptr; a.part = part;
    a.want = (dw_post ? 1 : 0) | (dscale ? 2 : 0) | (dw_pre ? 4 : 0);
    auto run = [&](auto t) {
        using E = decltype(t);
        constexpr int V = 16 / sizeof(E);
        return vector_rows(a, sizeof(E)) ? bwd_launch<E, V>(a, dw_post, dscale, dw_pre, st)
                                             : bwd_launch<E, 1>(a, dw_post, dscale, dw_pre, st);
    };
    switch (dt) {
        case DWCONV_FP32: return run(float{});
        case DWCONV_FP16: return run(__half{});
        default: return run(__nv_bfloat16{});
    }
}

}  // namespace dwc
