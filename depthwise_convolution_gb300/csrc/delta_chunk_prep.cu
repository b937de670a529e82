// First kernel of the chunked gated delta rule: per chunk and value head the
// triangular system's inverse, the masked score matrix and the row factors,
// none of which depend on the state.
#include "delta_chunk.cuh"
#include "delta_chunk_host.cuh"

namespace dwc {
namespace chunk {

namespace {

constexpr int kPrepThreads = 128;

// Eight values of a token's row, as they are stored: whole vectors (VEC) or
// single values.
template <typename T, bool VEC> struct Row8 {
    static constexpr int N = VEC ? 16 / sizeof(T) : 1;
    Pack<T, N> v[8 / N];
    __device__ __forceinline__ float get(int i) const { return v[i / N].get(i % N); }
};

// Loads PART units of 8 values each (unit i: row i / UNITS) of a [tokens][K]
// tensor, all on their way at once.  VEC: every unit is a whole aligned vector
// (compiled in: behind a run-time choice each load is waited for where it is
// made, 16 thousand cycles for a chunk).
template <typename T, int PART, int UNITS, bool VEC>
__device__ __forceinline__ void load_units(Row8<T, VEC> (&r)[PART], const T *p, long long row, int i0, int t0, int n,
                                           int K) {
    constexpr int N = Row8<T, VEC>::N;
#pragma unroll
    for (int x = 0; x < PART; ++x) {
        const int i = i0 + x * kPrepThreads, c = i % UNITS * 8, t = t0 + i / UNITS;
        const T *at = p + (long long)t * row + c;
#pragma unroll
        for (int j = 0; j < 8 / N; ++j)
            r[x].v[j] = t < n && c + j * N < K ? load_pack<T, N>(at + j * N) : zero_pack<T, N>();
    }
}

// A gate as it is stored, widened where it is used.
struct GateBits {
    unsigned v;
    template <typename T> __device__ __forceinline__ void load(const void *p, long long at, int f32, bool live) {
        v = 0u;
        if (!live) return;
        if (f32 || sizeof(T) == 4) v = static_cast<const unsigned *>(p)[at];
        else v = static_cast<const unsigned short *>(p)[at];
    }
    template <typename T> __device__ __forceinline__ float get(int f32) const {
        if (f32 || sizeof(T) == 4) return __uint_as_float(v);
        const unsigned short h = (unsigned short)v;
        return to_f32(*reinterpret_cast<const T *>(&h));
    }
};

constexpr int kLP = kC + 4;  // row pitch of L: columns of 8 rows 2 apart fall in different banks

// Shared memory: K and Q tiles, whose place L (fp32) and A (fp16 hi, lo) take
// over once the products with them are done; row factors.  M^T and P go to
// memory straight from registers: without a place for them here four CTAs fit
// an SM instead of three.
template <typename T, int KD> __host__ __device__ constexpr int front_bytes() {
    return 2 * kq16_elems<T, KD>() > 4 * kC * kLP + 4 * kTile ? 2 * kq16_elems<T, KD>() : 4 * kC * kLP + 4 * kTile;
}
// Per token while the chunk is prepared: scale of the k and q rows, |q|^2 and
// |k|^2 of the scaled rows, beta, e^G, e^(G_last - G), 1/|k|, l_k, 1/|q|, l_q scale.
enum { W_UK, W_UQ, W_Q2, W_K2, W_BETA, W_EG, W_EW, W_RK, W_LK, W_RQ, W_FQ, kWork };

// Grid (chunks, Hv, B).  The first value head of a key head also writes the K
// and Q images.
//
// With unit keys and L' = D k_i.k_j / (|k_i| |k_j|), beta' = beta l_k^2, the
// inverse M' = (I + L' beta')^-1 L' is found as its transpose X, 16 rows a warp
// and block column by block column (blocks of 16):
//   X_I = (L'^T_I - sum_(J < I) X_J (L' beta')^T_IJ) D_I^-T,   D_I = (I + L' beta')_II,
// each X_J the left operand of matrix instructions straight from the
// accumulators it was computed in.  The four D_I^-1 come first, one column a
// thread by forward substitution in fp32 (16 dependent steps instead of 64);
// split operands throughout.  The lengths are taken from the diagonal of the
// same K K^T that L' is made of, so that equal keys give 1 to the last bits.
// 65 chunks x 32 heads (K = 128, bf16) read 17 MB, write 88 MB and take 45 us
// (2.3 TB/s): a CTA's phases wait for one another (four CTAs of 128 threads an SM,
// issue 0.45 a cycle; the four inverses keep half the threads), and 2080 CTAs are
// 3.4 waves.  Five CTAs at 96 registers take as long here and 35 us instead of 32
// for 32 chunks x 32 heads, which are two waves either way; whole rows of blocks a
// warp, 1 to 4 of them, took 48.6.
//
// A token's key, gate or beta may be no finite number.  Its row of K and its beta
// are then zeros, its sum of gates a low number in all that M and P are made of, so
// that rows of tokens before it stay as they are; e^G of its key is no number, by
// which the walk finds where outputs and state are lost.
template <typename T, int KD, bool VEC>
__global__ void __launch_bounds__(kPrepThreads, sizeof(T) == 4 ? 1 : 4) delta_prep_kernel(DeltaArgs a, Prepared w, int nchunks) {
    constexpr int NT = terms16<T>(), TILE = kC * KD, BT = terms(!std::is_same<T, __nv_bfloat16>::value);
    extern __shared__ __align__(128) unsigned char smem[];
    __half *kq = reinterpret_cast<__half *>(smem);        // K tiles, Q tiles
    float *L = reinterpret_cast<float *>(smem);           // [64][kLP]
    // (-L' beta')_IJ below the diagonal blocks, D_I^-1 in them; hi, lo
    __half *A = reinterpret_cast<__half *>(smem + 4 * kC * kLP);
    float *vec16 = reinterpret_cast<float *>(smem + front_bytes<T, KD>()), *vec = vec16 + kVec16Elems, *work = vec + kVecElems;
    float *gh = vec + V_GH * kC, *gl = vec + V_GL * kC;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int c = blockIdx.x, h = blockIdx.y, b = blockIdx.z, group = a.Hv / a.Hk, hk = h / group;
    after_previous();
    const int n = live_length(a.lengths, b, a.T);
    const int t0 = c * kC;
    if (t0 >= n) return;
    const T *q = static_cast<const T *>(a.q) + b * a.q_s[0] + hk * a.q_s[2];
    const T *k = static_cast<const T *>(a.k) + b * a.k_s[0] + hk * a.k_s[2];
    const long long hc = ((long long)b * a.Hv + h) * nchunks + c, kc = ((long long)b * a.Hk + hk) * nchunks + c;
    const bool lead = h % group == 0;
    __half *mp = w.mp16 + hc * kMpElems;  // l_k M'^T hi, lo, P hi, lo

    // The gates of two tokens a lane of the last warp, on their way before all else.
    GateBits g_bits[2], b_bits[2];
    if (warp == 3) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = t0 + 2 * lane + j;
            g_bits[j].load<T>(a.g, b * a.g_s[0] + t * a.g_s[1] + h * a.g_s[2], a.gate_f32, t < n);
            b_bits[j].load<T>(a.beta, b * a.b_s[0] + t * a.b_s[1] + h * a.b_s[2], a.gate_f32, t < n);
        }
    }
    // Tiles: a row's KD / 8 units are neighbouring lanes; a thread has the loads
    // of PART units of both tensors in flight.
    constexpr int UNITS = KD / 8, PART = 4;
#pragma unroll
    for (int i0 = 0; i0 < kC * UNITS; i0 += PART * kPrepThreads) {
        Row8<T, VEC> kr[PART], qr[PART];
        load_units<T, PART, UNITS, VEC>(kr, k, a.k_s[1], i0 + tid, t0, n, a.K);
        load_units<T, PART, UNITS, VEC>(qr, q, a.q_s[1], i0 + tid, t0, n, a.K);
        float mk[PART], mq[PART], sq[PART];
#pragma unroll
        for (int x = 0; x < PART; ++x) {
            mk[x] = mq[x] = sq[x] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                mk[x] = max_or_nan(mk[x], fabsf(kr[x].get(i)), fabsf(kr[x].get(i + 1)));
                mq[x] = fmaxf(fmaxf(mq[x], fabsf(qr[x].get(i))), fabsf(qr[x].get(i + 1)));
            }
        }
#pragma unroll
        for (int o = 1; o < UNITS; o *= 2)
#pragma unroll
            for (int x = 0; x < PART; ++x) {
                mk[x] = max_or_nan(mk[x], __shfl_xor_sync(0xFFFFFFFFu, mk[x], o), 0.f);
                mq[x] = fmaxf(mq[x], __shfl_xor_sync(0xFFFFFFFFu, mq[x], o));
            }
#pragma unroll
        for (int x = 0; x < PART; ++x) {
            const int i = i0 + x * kPrepThreads + tid, r = i / UNITS, u = i % UNITS, at = swz<KD>(r, u * 8);
            float dk, uk, dq, uq;
            pow2_scale(mk[x], dk, uk);
            pow2_scale(mq[x], dq, uq);
            Frag kh, kl, qh, ql;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float q0 = qr[x].get(2 * j) * dq, q1 = qr[x].get(2 * j + 1) * dq;
                split_half(kr[x].get(2 * j) * dk, kr[x].get(2 * j + 1) * dk, kh.r[j], kl.r[j]);
                split_half(q0, q1, qh.r[j], ql.r[j]);
                sq[x] = fmaf(q0, q0, fmaf(q1, q1, sq[x]));
            }
            *reinterpret_cast<uint4 *>(kq + at) = make_uint4(kh.r[0], kh.r[1], kh.r[2], kh.r[3]);
            *reinterpret_cast<uint4 *>(kq + NT * TILE + at) = make_uint4(qh.r[0], qh.r[1], qh.r[2], qh.r[3]);
            if (NT == 2) {
                *reinterpret_cast<uint4 *>(kq + TILE + at) = make_uint4(kl.r[0], kl.r[1], kl.r[2], kl.r[3]);
                *reinterpret_cast<uint4 *>(kq + (NT + 1) * TILE + at) = make_uint4(ql.r[0], ql.r[1], ql.r[2], ql.r[3]);
            }
            if (!is_finite(mk[x])) {
                *reinterpret_cast<uint4 *>(kq + at) = make_uint4(0, 0, 0, 0);
                if (NT == 2) *reinterpret_cast<uint4 *>(kq + TILE + at) = make_uint4(0, 0, 0, 0);
                uk = kNan;
            }
            if (u == 0) {
                work[W_UK * kC + r] = uk;
                work[W_UQ * kC + r] = uq;
            }
            if (w.kq && lead) {  // the backward pass's images
                __nv_bfloat16 *to = w.kq + kc * 2 * BT * TILE + at;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    split_bf16(kr[x].get(2 * j), kr[x].get(2 * j + 1), kh.r[j], kl.r[j]);
                    split_bf16(qr[x].get(2 * j), qr[x].get(2 * j + 1), qh.r[j], ql.r[j]);
                }
                *reinterpret_cast<uint4 *>(to) = make_uint4(kh.r[0], kh.r[1], kh.r[2], kh.r[3]);
                *reinterpret_cast<uint4 *>(to + BT * TILE) = make_uint4(qh.r[0], qh.r[1], qh.r[2], qh.r[3]);
                if (BT == 2) {
                    *reinterpret_cast<uint4 *>(to + TILE) = make_uint4(kl.r[0], kl.r[1], kl.r[2], kl.r[3]);
                    *reinterpret_cast<uint4 *>(to + (BT + 1) * TILE) = make_uint4(ql.r[0], ql.r[1], ql.r[2], ql.r[3]);
                }
            }
        }
#pragma unroll
        for (int o = 1; o < UNITS; o *= 2)
#pragma unroll
            for (int x = 0; x < PART; ++x) sq[x] += __shfl_xor_sync(0xFFFFFFFFu, sq[x], o);
#pragma unroll
        for (int x = 0; x < PART; ++x) {
            const int i = i0 + x * kPrepThreads + tid;
            if (i % UNITS == 0) work[W_Q2 * kC + i / UNITS] = sq[x];
        }
    }
    // Running sums of g in double, as hi + lo floats: differences of sums that a
    // strong decay made large stay exact to fp32.
    if (warp == 3) {
        double s[2];
        float be[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float g = g_bits[j].get<T>(a.gate_f32);
            s[j] = g < kDeltaReset ? kDeltaReset : g;
            be[j] = b_bits[j].get<T>(a.gate_f32);
        }
        double run = s[0] + s[1];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const double up = __shfl_up_sync(0xFFFFFFFFu, run, o);
            if (lane >= o) run += up;
        }
        const double before = __shfl_up_sync(0xFFFFFFFFu, run, 1);
        if (lane > 0) s[0] += before;  // not run - s[1], which need be no number where s[0] is one
        s[1] = run;
        const double last = __shfl_sync(0xFFFFFFFFu, run, 31);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 2 * lane + j;
            // a sum that is none stands below all others: decays from there are 0 or, among such, 1
            const bool sum = is_finite((float)s[j]);
            const float hi = sum ? (float)s[j] : 256 * kDeltaReset;
            gh[r] = hi;
            gl[r] = sum ? (float)(s[j] - hi) : 0.f;
            work[W_BETA * kC + r] = be[j];
            work[W_EG * kC + r] = __expf((float)s[j]);
            work[W_EW * kC + r] = __expf((float)(last - s[j]));
            vec[V_LAST * kC + r] = vec16[F_LAST * kC + r] = __expf((float)last);
        }
    }
    fence_async();
    __syncthreads();
    if (tid == 0 && lead) {
        constexpr int N = kq16_elems<T, KD>();
        bulk_store(w.kq16 + kc * N, kq, N * 2);
        bulk_commit();
    }

    // K K^T and Q K^T up to the diagonal, ten blocks of 16 x 16 each: a warp takes
    // two blocks of both, its diagonal block and one of the last row (or (2, 1)), and
    // a third of one of them, (1, 0) or (2, 0).
    const int br[3] = {warp, warp == 3 ? 2 : 3, warp / 2 + 1};     // block rows and columns
    const int bc[3] = {warp, warp == 3 ? 1 : warp, 0};
    const bool third_q = warp % 2;  // the third block is of Q K^T
    float kk[2][2][4], qk[2][2][4], third[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[0][t][j] = kk[1][t][j] = qk[0][t][j] = qk[1][t][j] = third[t][j] = 0.f;
#pragma unroll
    for (int s = 0; s < KD / 16; ++s) {
        auto left = [&](const __half *tile, int i) {  // rows of block i
            return ldsm(tile + swz<KD>(16 * br[i] + kn_row(lane), 16 * s + kn_col(lane)));
        };
        auto right = [&](const __half *tile, int i) {
            return ldsm(tile + swz<KD>(16 * bc[i] + nk_row(lane), 16 * s + nk_col(lane)));
        };
        auto times = [&](float (&d)[2][4], const Frag (&x)[NT], const Frag (&y)[NT]) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < NT - i; ++j)  // hi hi, hi lo, lo hi
                        mma16(d[t], x[i], y[j].r[2 * t], y[j].r[2 * t + 1]);
        };
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            Frag kb[NT], ka[NT], qa[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) kb[t] = right(kq + t * TILE, i);
            if (i == 2) {
#pragma unroll
                for (int t = 0; t < NT; ++t) ka[t] = left(kq + (third_q ? NT + t : t) * TILE, i);
                times(third, ka, kb);
            } else {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    ka[t] = left(kq + t * TILE, i);
                    qa[t] = left(kq + (NT + t) * TILE, i);
                }
                times(kk[i & 1], ka, kb);
                times(qk[i & 1], qa, kb);
            }
        }
    }
    const int r0 = lane / 4, c0 = 2 * (lane % 4);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (8 * t + c0 + (j & 1) == r0 + 8 * (j >> 1))
                work[W_K2 * kC + 16 * warp + r0 + 8 * (j >> 1)] = kk[0][t][j];
    if (tid == 0) bulk_wait_read();  // the tiles have left
    __syncthreads();
    if (tid < kC) {  // row factors
        auto at = [&](int i) -> float & { return work[i * kC + tid]; };
        const float k2 = at(W_K2), q2 = at(W_Q2), uk = at(W_UK), uq = at(W_UQ), be = at(W_BETA);
        const float rk = k2 > 0.f ? rsqrtf(k2) : 0.f, rq = q2 > 0.f ? rsqrtf(q2) : 0.f;
        // |k| = sqrt(k2) uk; the eps of the norms belongs to the unscaled sum
        const float nk = a.qk_norm ? rsqrtf(fmaf(k2 * uk, uk, kDeltaEps)) : 1.f;
        const float nq = a.qk_norm ? rsqrtf(fmaf(q2 * uq, uq, kDeltaEps)) : 1.f;
        const float fk = uk * nk, lk = finite_or_zero(k2 * rk * fk), lq = q2 * rq * uq * nq;
        const float eg = at(W_EG), ew = at(W_EW);
        at(W_RK) = rk;
        at(W_LK) = lk;
        at(W_RQ) = rq;
        at(W_FQ) = lq * a.scale;
        vec16[F_LB * kC + tid] = finite_or_zero(lk * be);
        vec16[F_EK * kC + tid] = fmaf(0.f, be, eg * fk);  // no number where beta is none
        vec16[F_EQ * kC + tid] = eg * rq;
        vec16[F_WB * kC + tid] = be * ew * fk;
        vec16[F_FQ * kC + tid] = lq * a.scale;
        vec[V_BETA * kC + tid] = be;
        vec[V_EK * kC + tid] = eg * nk;
        vec[V_EQ * kC + tid] = eg * nq * a.scale;
        vec[V_W * kC + tid] = ew * nk;
        vec[V_NK * kC + tid] = nk;
        vec[V_NQ * kC + tid] = nq * a.scale;
        vec[V_IQ * kC + tid] = nq;
    }
    __syncthreads();
    // L' (fp32), -L' beta' and P (hi, lo), block by block
    auto each = [&](int R, int C, auto &&f) {  // f(tile, half, row, column, decays over both key lengths)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int col = 16 * C + 8 * t + c0;
            const float2 rj = *reinterpret_cast<const float2 *>(work + W_RK * kC + col);
            const float2 gj = *reinterpret_cast<const float2 *>(gh + col), hj = *reinterpret_cast<const float2 *>(gl + col);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = 16 * R + r0 + 8 * half;
                const float g = gh[r], gg = gl[r];
                f(t, half, r, col, col <= r ? __expf((g - gj.x) + (gg - hj.x)) * rj.x : 0.f,
                  col + 1 <= r ? __expf((g - gj.y) + (gg - hj.y)) * rj.y : 0.f);
            }
        }
    };
    auto put_l = [&](const float (&d)[2][4], int R, int C, int t, int half, int r, int col, float d0, float d1) {
        const float rk = work[W_RK * kC + r];
        const float l0 = col < r ? d0 * rk * d[t][2 * half] : 0.f, l1 = col + 1 < r ? d1 * rk * d[t][2 * half + 1] : 0.f;
        *reinterpret_cast<float2 *>(L + r * kLP + col) = make_float2(l0, l1);
        if (C < R) {
            const float2 bj = *reinterpret_cast<const float2 *>(vec16 + F_LB * kC + col);
            const float2 lj = *reinterpret_cast<const float2 *>(work + W_LK * kC + col);
            const int at = swz<kC>(r, col);
            unsigned hi, lo;
            split_half(-l0 * bj.x * lj.x, -l1 * bj.y * lj.y, hi, lo);
            *reinterpret_cast<unsigned *>(A + at) = hi;
            *reinterpret_cast<unsigned *>(A + kTile + at) = lo;
        }
    };
    auto put_p = [&](const float (&d)[2][4], int t, int half, int r, int col, float d0, float d1) {
        const float rq = work[W_RQ * kC + r], p0 = d[t][2 * half] * d0 * rq, p1 = d[t][2 * half + 1] * d1 * rq;
        const int at = swz<kC>(r, col);
        unsigned hi, lo;
        split_half(p0, p1, hi, lo);
        *reinterpret_cast<unsigned *>(mp + 2 * kTile + at) = hi;
        if (fine_out<T>()) *reinterpret_cast<unsigned *>(mp + 3 * kTile + at) = lo;
        if (w.mp) {
            const float fq = work[W_FQ * kC + r];
            const float2 lj = *reinterpret_cast<const float2 *>(work + W_LK * kC + col);
            split_bf16(p0 * fq * lj.x, p1 * fq * lj.y, hi, lo);
            *reinterpret_cast<unsigned *>(w.mp + hc * kMpElems + 2 * kTile + at) = hi;
            *reinterpret_cast<unsigned *>(w.mp + hc * kMpElems + 3 * kTile + at) = lo;
        }
    };
#pragma unroll
    for (int i = 0; i < 2; ++i)
        each(br[i], bc[i], [&](int t, int half, int r, int col, float d0, float d1) {
            put_l(kk[i], br[i], bc[i], t, half, r, col, d0, d1);
            put_p(qk[i], t, half, r, col, d0, d1);
        });
    each(br[2], bc[2], [&](int t, int half, int r, int col, float d0, float d1) {
        if (third_q) put_p(third, t, half, r, col, d0, d1);
        else put_l(third, br[2], bc[2], t, half, r, col, d0, d1);
    });
    __syncthreads();
    if (tid < kC) {
        // column tid % 16 of D^-1 of block tid / 16; the block's rows are read ahead
        // of the chain, which is stored at its end
        const int first = tid / 16 * 16, cc = tid % 16;
        float x[16], y[16], be[16];  // y = beta' x
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(vec16 + F_LB * kC + first + i);
            const float4 l = *reinterpret_cast<const float4 *>(work + W_LK * kC + first + i);
            be[i] = v.x * l.x; be[i + 1] = v.y * l.y; be[i + 2] = v.z * l.z; be[i + 3] = v.w * l.w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s[2] = {i == cc ? 1.f : 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(L + (first + i) * kLP + first + m);
                const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (m + j < i) s[j & 1] = fmaf(-l[j], y[m + j], s[j & 1]);
            }
            x[i] = s[0] + s[1];
            y[i] = x[i] * be[i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __half hi = __float2half_rn(x[i]);
            const int at = swz<kC>(first + i, first + cc);
            A[at] = hi;
            A[kTile + at] = __float2half_rn(x[i] - __half2float(hi));
        }
    }
    __syncthreads();
    const float lr[2] = {work[W_LK * kC + 16 * warp + r0], work[W_LK * kC + 16 * warp + r0 + 8]};
    // X: rows j = 16 warp .. + 15, blocks I from the diagonal on (those before are zero).
    Frag xh[4], xl[4];
#pragma unroll
    for (int I = 0; I < 4; ++I) {
        if (I < warp) continue;
        float acc[2][4], x[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[t][j] = L[(16 * I + 8 * t + c0 + (j & 1)) * kLP + 16 * warp + r0 + 8 * (j >> 1)];
                x[t][j] = 0.f;
            }
        auto times = [&](float (&d)[2][4], const Frag &hi, const Frag &lo, int J) {
            const int at = swz<kC>(16 * I + nk_row(lane), 16 * J + nk_col(lane));
            const Frag bh = ldsm(A + at), bl = ldsm(A + kTile + at);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma16(d[t], hi, bh.r[2 * t], bh.r[2 * t + 1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma16(d[t], lo, bh.r[2 * t], bh.r[2 * t + 1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma16(d[t], hi, bl.r[2 * t], bl.r[2 * t + 1]);
        };
#pragma unroll
        for (int J = 0; J < I; ++J)
            if (J >= warp) times(acc, xh[J], xl[J], J);
        Frag hi, lo;
        to_frags16(acc[0], acc[1], hi, lo);
        times(x, hi, lo, I);
        to_frags16(x[0], x[1], xh[I], xl[I]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {  // l_i X (and l_i l_j X for the backward pass), i along the columns
            const int col = 16 * I + 8 * t + c0;
            const float2 li = *reinterpret_cast<const float2 *>(work + W_LK * kC + col);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float x0 = x[t][2 * half] * li.x, x1 = x[t][2 * half + 1] * li.y;
                const int at = swz<kC>(16 * warp + r0 + 8 * half, col);
                unsigned uh, ul;
                split_half(x0, x1, uh, ul);
                *reinterpret_cast<unsigned *>(mp + at) = uh;
                *reinterpret_cast<unsigned *>(mp + kTile + at) = ul;
                if (w.mp) {
                    split_bf16(x0 * lr[half], x1 * lr[half], uh, ul);
                    *reinterpret_cast<unsigned *>(w.mp + hc * kMpElems + at) = uh;
                    *reinterpret_cast<unsigned *>(w.mp + hc * kMpElems + kTile + at) = ul;
                }
            }
        }
    }
    fence_async();
    __syncthreads();
    if (tid == 0) {
        bulk_store(w.vec16 + hc * kVec16Elems, vec16, kVec16Elems * 4);
        if (w.vec) bulk_store(w.vec + hc * kVecElems, vec, kVecElems * 4);
        bulk_commit();
        bulk_wait_read();
    }
}

template <typename T, int KD> cudaError_t run(const DeltaArgs &a, const Prepared &w, cudaStream_t st) {
    constexpr size_t smem = front_bytes<T, KD>() + 4 * (kVec16Elems + kVecElems + kWork * kC);
    // whole aligned vectors of 8 in every row of q and k
    auto whole = [&](const void *p, const long long(&s)[3]) {
        bool ok = reinterpret_cast<uintptr_t>(p) % 16 == 0 && a.K % 8 == 0;
        for (long long v : s) ok = ok && v * (long long)sizeof(T) % 16 == 0;
        return ok;
    };
    auto kern = whole(a.k, a.k_s) && whole(a.q, a.q_s) ? delta_prep_kernel<T, KD, true> : delta_prep_kernel<T, KD, false>;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), kPrepThreads, smem, nullptr);
    if (e != cudaSuccess) return e;
    const int n = (a.T + kC - 1) / kC;
    note_launches(1);
    return launch_after(kern, dim3(n, a.Hv, a.B), kPrepThreads, smem, st, a, w, n);
}

}  // namespace

cudaError_t launch_prep(const DeltaArgs &a, dwconv_dtype dt, const Prepared &w, cudaStream_t st) {
    auto width = [&](auto t) {
        using E = decltype(t);
        return a.K <= 64 ? run<E, 64>(a, w, st) : run<E, 128>(a, w, st);
    };
    switch (dt) {
        case DWCONV_FP32: return width(float{});
        case DWCONV_FP16: return width(__half{});
        default: return width(__nv_bfloat16{});
    }
}

}  // namespace chunk
}  // namespace dwc
