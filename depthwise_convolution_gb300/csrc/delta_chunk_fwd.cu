// Second kernel of the chunked gated delta rule: the state's walk over the
// chunks of one head, with outputs.
//
// Columns of the state are independent, so a team of four warps owns 16 of them
// and keeps S^T [16][K] in the accumulators of its matrix instructions for the
// whole sequence, each warp a quarter of the keys.  Everything it multiplies is
// a tile of tokens x keys or tokens x tokens that all warps of the head share:
//   (K S)^T = S^T K^T,  R^T = V^T - (e^G K S)^T,  U^^T = R^T - (beta R)^T M^T,
//   O^T = (e^G Q S)^T + U^T P^T,   S^T = e^G_last S^T + (w U)^T K,
// and an accumulator of one product is, register for register, the left
// operand of the next.  Each warp solves and outputs one of the four 16-token
// blocks.  The team meets three times a chunk, over operands in shared memory:
// the quarters of the state, the blocks of beta R, those of U.  The first thread
// has the next chunk's tiles (K, Q, M, P and the row factors: 58 KB at K = 128)
// copied into the other stage.
//
// What bounds it: the chain of chunks, in which a warp issues about 800
// instructions one after the other, some six cycles apart with two warps a
// scheduler (issue 0.34 a cycle, shared memory 62 % of its rate); heads x V / 16
// column groups seldom fill the 608 sub-partitions, so a group is worth four
// warps.  32 heads x 4097 tokens, K = V = 128, bf16: 164 us, against 232 with two
// warps a group and 248 with one (162 without the branch for inputs that are no
// numbers).  With a copy of the code per block assignment, waiting for
// instructions was the largest stall; now the blocks' bounds are tested in
// unrolled loops (rolled ones: 10 us more).  Partial sums of S K^T
// shared instead of the state's operands took as long with one meeting more.
// Scaling the state's rows for each product and back took 175 us, scales per
// block of tokens 174.
#include <algorithm>

#include "delta_chunk_host.cuh"
#include "delta_chunk_walk.cuh"

namespace dwc {
namespace chunk {

namespace {

template <typename T, int KD> __host__ __device__ constexpr unsigned stage_bytes() {
    return 2 * kq16_elems<T, KD>() + mp16_bytes<T>() + 4 * kVec16Elems;
}

// Chunks that fit shared memory beside the team's buffers.
template <typename T, int KD> __host__ __device__ constexpr int stages() { return sizeof(T) == 4 && KD == 128 ? 1 : 2; }

// What a team exchanges: the state's quarters and the blocks of beta R and U as
// left operands, and the largest state and l beta R per column.
enum { OP_P = 0, OP_W = 2, kOps = 4 };
template <int KS> struct TeamBuf {
    uint4 s[kTeam][KS][2][32];  // [quarter][k-step][hi, lo][lane]
    uint4 br[4][2][32];         // [block][hi, lo][lane]
    uint4 op[4][kOps][32];      // [block][l U hi, lo, w U hi, lo][lane]
    float s_most[kTeam][16], most[kTeam][16];
};

// Largest magnitude of a row over its four lanes: rows lane / 4 (entries 0, 1)
// and lane / 4 + 8 (2, 3) of N tiles.  NAN_TOO: a NaN in a row is its largest.
template <bool NAN_TOO> __device__ __forceinline__ float largest(float a, float b, float c = 0.f) {
    return NAN_TOO ? max_or_nan(a, b, c) : fmaxf(fmaxf(a, b), c);
}
template <int N, bool NAN_TOO = false> __device__ __forceinline__ void row_max(const float (&x)[N][4], float (&m)[2]) {
    m[0] = m[1] = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) m[q] = largest<NAN_TOO>(m[q], fabsf(x[i][2 * q]), fabsf(x[i][2 * q + 1]));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        m[q] = largest<NAN_TOO>(m[q], __shfl_xor_sync(0xFFFFFFFFu, m[q], 1));
        m[q] = largest<NAN_TOO>(m[q], __shfl_xor_sync(0xFFFFFFFFu, m[q], 2));
    }
}
template <int N> __device__ __forceinline__ void scale_rows(float (&x)[N][4], const float (&f)[2]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] *= f[j >> 1];
}

// Rows' magnitudes, shared within the team: lanes 0, 4, .. write their two rows.
__device__ __forceinline__ void share_rows(float (&to)[16], const float (&m)[2], int lane) {
    if (lane % 4 == 0) {
        to[lane / 4] = m[0];
        to[lane / 4 + 8] = m[1];
    }
}
template <bool NAN_TOO = false>
__device__ __forceinline__ void most_rows(const float (&from)[kTeam][16], int lane, float (&m)[2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = lane / 4 + 8 * q;
        m[q] = largest<NAN_TOO>(largest<NAN_TOO>(from[0][r], from[1][r], from[2][r]), from[3][r]);
    }
}

// The state's columns, R, U and O are kept over a power of two per column, the
// same in all warps of the team, in which the largest l beta R, or 1/64 of the
// largest value of the decayed state, lies in [1/2, 32): 64 updates of a key of
// at most 2 then leave the state below 2^13, and a split value's error, 2^-25 at
// least, is below 2^-23 of the column.  Zeros fit everywhere.
constexpr float kUnderState = 1.f / 64;
struct Domain {
    float up[2] = {1.f, 1.f}, down[2] = {1.f, 1.f};
    static __device__ __forceinline__ bool off(float need) { return need != 0.f && !(need >= 0.5f && need < 32.f); }
    // What brings `need` to [4, 8), as far as the scale stays within 2^-100 and 2^100.
    __device__ __forceinline__ float fit(int q, float need) const {
        if (!(need > 0.f)) return 1.f;
        float by, back;
        pow2_scale(need, by, back);
        return fminf(fmaxf(by * 4.f, up[q] * 0x1p-100f), up[q] * 0x1p100f);
    }
    // Values are about to be multiplied by f.
    __device__ __forceinline__ void move(int q, float f) {
        down[q] *= f;
        unsigned e = __float_as_uint(down[q]) >> 23;
        up[q] = __uint_as_float((254 - e) << 23);
    }
};

// Where a row (a column of the state) meets a value, key or gate that is no finite
// number: the first token of a warp's block from which on it is lost (16: none).
// The zeros above the diagonals of M and P would spread it to tokens before, so
// entries from it on stay out of the products, the outputs from it on and the
// state are lost by themselves.  M and P hold numbers whatever the inputs.
struct Cut {
    int at[2] = {16, 16};
    // x: the block of l beta R; most: the largest in the blocks of all warps
    __device__ __forceinline__ void find(const float (&x)[2][4], const float (&most)[kTeam][16], int me, int lane) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int i = 1; i >= 0; --i)
#pragma unroll
                for (int j = 1; j >= 0; --j)
                    if (!is_finite(x[i][2 * q + j])) at[q] = 8 * i + 2 * (lane % 4) + j;
            at[q] = min(at[q], __shfl_xor_sync(0xFFFFFFFFu, at[q], 1));
            at[q] = min(at[q], __shfl_xor_sync(0xFFFFFFFFu, at[q], 2));
            for (int i = 0; i < me; ++i)
                if (!is_finite(most[i][lane / 4 + 8 * q])) at[q] = 0;
        }
    }
    __device__ __forceinline__ void fill(float (&x)[2][4], int lane, float from_there_on) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (8 * i + 2 * (lane % 4) + (j & 1) >= at[j >> 1]) x[i][j] = from_there_on;
    }
};

template <typename T, int KD, bool PAIRS, typename F>
__device__ __forceinline__ void walk(const DeltaArgs &a, const Saved &saved, Ring &ring, const unsigned char *smem,
                                     F &&copy, TeamBuf<KD / kTeam / 16> &buf, int team, int me, int nchunks, int live, int n, int h, int b,
                                     int col, unsigned *err) {
    constexpr int NT = terms16<T>(), TILE = kC * KD, KH = KD / kTeam, KS = KH / 16, NS = KH / 8, STAGES = stages<T, KD>();
    constexpr bool FINE = fine_out<T>(), FULL = !std::is_same<T, __nv_bfloat16>::value;
    const int lane = threadIdx.x % 32, c0 = 2 * (lane % 4), k0 = me * KH;
    const bool on = col < a.V;  // teams beyond the last column group only keep the barriers in step
    const T *v = static_cast<const T *>(a.v) + b * a.v_s[0] + h * a.v_s[2];
    T *out = static_cast<T *>(a.out) + (((long long)b * a.T) * a.Hv + h) * a.V;
    const long long o_row = (long long)a.Hv * a.V, s_at = ((long long)b * a.Hv + h) * a.K * a.V;
    const int v16 = (a.V + 15) / 16 * 16;
    auto mine = [&](int x) { return 2 * me + x; };  // 8-token tiles of this warp's block

    float S[NS][4];
    each_state<NS>(a, k0, col, lane, [&](int i, int j, bool in, long long at) {
        S[i][j] = a.state && in ? a.state[s_at + at] : 0.f;
    });
    Domain dom;
    {
        float m[2];
        row_max<NS>(S, m);
        share_rows(buf.most[me], m, lane);  // next written beyond the first meeting in a chunk
        team_sync(team);
        float need[2];
        most_rows(buf.most, lane, need);
#pragma unroll
        for (int q = 0; q < 2; ++q) dom.move(q, dom.fit(q, need[q] * kUnderState));
        scale_rows<NS>(S, dom.down);
    }
    VTile<T, 2, PAIRS> vt;
    if (on) vt.load(v, a.v_s[1], 0, n, col, a.V, lane, mine);
    // where this lane points ldmatrix in a tile, up to the block's row and column
    const int nk = nk_row(lane), nkc = nk_col(lane), kn = kn_row(lane), knc = kn_col(lane);

    // After a wait that gave up the walk goes on without waiting (the team's
    // barriers need all its warps); the result is reported as lost.
    bool ok = true;
    for (int c = 0; c < live; ++c) {
        const int st = c % STAGES;
        if (threadIdx.x == 0 && ok && c + STAGES - 1 < live && c + STAGES - 1 > 0) ok = copy(c + STAGES - 1);
        __syncwarp();
        if (ok && !mbar_wait(&ring.full[st], (c / STAGES) & 1)) {
            report_timeout(err);
            ok = false;
        }
        const __half *kt = reinterpret_cast<const __half *>(smem + st * stage_bytes<T, KD>());
        const __half *qt = kt + NT * TILE, *mt = kt + kq16_elems<T, KD>(), *pt = mt + 2 * kTile;
        const float *vec = reinterpret_cast<const float *>(mt + mp16_bytes<T>() / 2);
        auto factor = [&](int which, int tile) {
            return *reinterpret_cast<const float2 *>(vec + which * kC + 8 * tile + c0);
        };
        if (on) {
            const long long hc = ((long long)b * a.Hv + h) * nchunks + c;
            if (saved.s) {
                float t[NS][4];
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[i][j] = S[i][j] * dom.up[j >> 1];
                store_image<KD>(saved.s + (hc * terms(FULL) * v16 + col) * KD, t, lane,
                                FULL ? (long long)v16 * KD / 2 : 0, [&](int i) { return k0 / 8 + i; });
            }
            float X[2][4], Y[2][4], m[2];  // this warp's block: R, then U^; Q S, then O
            {
                // This warp's keys of the state as operands
                row_max<NS>(S, m);
                share_rows(buf.s_most[me], m, lane);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    Frag hi, lo;
                    to_frags16(S[2 * s], S[2 * s + 1], hi, lo);
                    buf.s[me][s][0][lane] = as_uint4(hi);
                    buf.s[me][s][1][lane] = as_uint4(lo);
                }
            }
            team_sync(team);
            // (K S)^T and (Q S)^T of its block, two sums of each side by side
            float R[2][2][4], O[2][2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j) R[k][x][j] = O[k][x][j] = 0.f;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int k = 0; k < kTeam; ++k) {
                    const Frag hi = as_frag(buf.s[k][s][0][lane]), lo = as_frag(buf.s[k][s][1][lane]);
                    const int at = swz<KD>(16 * me + nk, k * KH + 16 * s + nkc);
                    const Frag kb = ldsm(kt + at), qb = ldsm(qt + at);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma16(R[0][x], hi, kb.r[2 * x], kb.r[2 * x + 1]);
                        mma16(O[k & 1][x], hi, qb.r[2 * x], qb.r[2 * x + 1]);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma16(R[1][x], lo, kb.r[2 * x], kb.r[2 * x + 1]);
                        if (FINE) mma16(O[1 - (k & 1)][x], lo, qb.r[2 * x], qb.r[2 * x + 1]);
                    }
                    if (NT == 2) {
                        const Frag kl = ldsm(kt + TILE + at), ql = ldsm(qt + TILE + at);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            mma16(R[1][x], hi, kl.r[2 * x], kl.r[2 * x + 1]);
                            mma16(O[k & 1][x], hi, ql.r[2 * x], ql.r[2 * x + 1]);
                        }
                    }
                }
            float B[2][4];  // l beta R
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 ek = factor(F_EK, mine(x)), eq = factor(F_EQ, mine(x)), lb = factor(F_LB, mine(x));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    X[x][j] = fmaf(-(j & 1 ? ek.y : ek.x), R[0][x][j] + R[1][x][j], vt.get(x, j) * dom.down[j >> 1]);
                    Y[x][j] = (O[0][x][j] + O[1][x][j]) * (j & 1 ? eq.y : eq.x);
                    B[x][j] = X[x][j] * (j & 1 ? lb.y : lb.x);
                }
            }
            if (c + 1 < live) vt.load(v, a.v_s[1], (c + 1) * kC, n, col, a.V, lane, mine);
            row_max<2, true>(B, m);
            share_rows(buf.most[me], m, lane);
            auto share_blocks = [&] {
                float t[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[x][j] = -B[x][j];
                Frag hi, lo;
                to_frags16(t[0], t[1], hi, lo);
                buf.br[me][0][lane] = as_uint4(hi);
                buf.br[me][1][lane] = as_uint4(lo);
            };
            share_blocks();
            team_sync(team);
            // Where the scale of a column no longer suits both U and the state it moves,
            // or what they need is no number, the blocks are shared once more: all warps
            // see the same columns.
            const float last = vec[F_LAST * kC];
            float need[2], left[2], keep[2] = {last, last};
            most_rows<true>(buf.most, lane, need);
            most_rows(buf.s_most, lane, left);
            bool off = false, lost = false;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                left[q] *= last * kUnderState;
                need[q] = max_or_nan(need[q], left[q], 0.f);
                off |= Domain::off(need[q]);
            }
            if (__builtin_expect(__any_sync(0xFFFFFFFFu, off), 0)) {
                lost = __any_sync(0xFFFFFFFFu, !is_finite(need[0]) || !is_finite(need[1]));
                if (lost) {
                    Cut cut;
                    cut.find(B, buf.most, me, lane);
                    cut.fill(B, lane, 0.f);
                    cut.fill(X, lane, 0.f);
                    cut.fill(Y, lane, kNan);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (!is_finite(need[q])) keep[q] = kNan;
                    row_max<2>(B, m);
                    team_sync(team);  // `most` has been read
                    share_rows(buf.most[me], m, lane);
                    team_sync(team);
                    most_rows(buf.most, lane, need);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (is_finite(left[q])) need[q] = fmaxf(need[q], left[q]);
                }
                float f[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    f[q] = Domain::off(need[q]) ? dom.fit(q, need[q]) : 1.f;
                    dom.move(q, f[q]);
                    keep[q] *= f[q];
                }
                scale_rows<2>(B, f);
                scale_rows<2>(X, f);
                scale_rows<2>(Y, f);
                share_blocks();
                team_sync(team);
            }
            // U^^T = R^T - (l beta R)^T (l M)^T over the column blocks up to its own
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s > me) break;
                const Frag hi = as_frag(buf.br[s][0][lane]), lo = as_frag(buf.br[s][1][lane]);
                const int at = swz<kC>(16 * s + kn, 16 * me + knc);
                const Frag mh = ldsm_t(mt + at), ml = ldsm_t(mt + kTile + at);
#pragma unroll
                for (int x = 0; x < 2; ++x) mma16(X[x], hi, mh.r[2 * x], mh.r[2 * x + 1]);
#pragma unroll
                for (int x = 0; x < 2; ++x) mma16(X[x], lo, mh.r[2 * x], mh.r[2 * x + 1]);
#pragma unroll
                for (int x = 0; x < 2; ++x) mma16(X[x], hi, ml.r[2 * x], ml.r[2 * x + 1]);
            }
            if (saved.u) {
                float t[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[x][j] = X[x][j] * dom.up[j >> 1];
                if (lost)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[x][j] = fmaf(0.f, Y[x][j], t[x][j]);  // lost with its output
                store_image<kC>(saved.u + (hc * 2 * v16 + col) * kC, t, lane, (long long)v16 * kC / 2, mine);
            }
            // U as operands: l U for P, w U for the state
            {
                float t[2][4], w[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 lb = factor(F_LB, mine(x)), wb = factor(F_WB, mine(x));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        t[x][j] = X[x][j] * (j & 1 ? lb.y : lb.x);
                        w[x][j] = X[x][j] * (j & 1 ? wb.y : wb.x);
                    }
                }
                Frag hi, lo;
                to_frags16(t[0], t[1], hi, lo);
                buf.op[me][OP_P][lane] = as_uint4(hi);
                if (FINE) buf.op[me][OP_P + 1][lane] = as_uint4(lo);
                to_frags16(w[0], w[1], hi, lo);
                buf.op[me][OP_W][lane] = as_uint4(hi);
                buf.op[me][OP_W + 1][lane] = as_uint4(lo);
            }
            scale_rows<NS>(S, keep);
            team_sync(team);
            // S^T = e^G_last S^T + (w U)^T K for this warp's keys, and
            // O^T += (l U)^T P^T over the column blocks up to its own
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const Frag uh = as_frag(buf.op[s][OP_W][lane]), ul = as_frag(buf.op[s][OP_W + 1][lane]);
#pragma unroll
                for (int p = 0; p < KS; ++p) {
                    const int at = swz<KD>(16 * s + kn, k0 + 16 * p + knc);
                    const Frag kb = ldsm_t(kt + at);
#pragma unroll
                    for (int x = 0; x < 2; ++x) mma16(S[2 * p + x], uh, kb.r[2 * x], kb.r[2 * x + 1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) mma16(S[2 * p + x], ul, kb.r[2 * x], kb.r[2 * x + 1]);
                    if (NT == 2) {
                        const Frag kl = ldsm_t(kt + TILE + at);
#pragma unroll
                        for (int x = 0; x < 2; ++x) mma16(S[2 * p + x], uh, kl.r[2 * x], kl.r[2 * x + 1]);
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s > me) break;
                const Frag ph = as_frag(buf.op[s][OP_P][lane]);
                const int at = swz<kC>(16 * me + nk, 16 * s + nkc);
                const Frag bh = ldsm(pt + at);
#pragma unroll
                for (int x = 0; x < 2; ++x) mma16(Y[x], ph, bh.r[2 * x], bh.r[2 * x + 1]);
                if (FINE) {
                    const Frag pl = as_frag(buf.op[s][OP_P + 1][lane]), bl = ldsm(pt + kTile + at);
#pragma unroll
                    for (int x = 0; x < 2; ++x) mma16(Y[x], pl, bh.r[2 * x], bh.r[2 * x + 1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) mma16(Y[x], ph, bl.r[2 * x], bl.r[2 * x + 1]);
                }
            }
            if (a.out) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 fq = factor(F_FQ, mine(x));
#pragma unroll
                    for (int j = 0; j < 4; ++j) Y[x][j] *= (j & 1 ? fq.y : fq.x) * dom.up[j >> 1];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ring.empty[st]);  // the stage has been read
            if (a.out) store_tokens<T, PAIRS>(out, o_row, c * kC, a.T, col, a.V, lane, Y, mine);
        } else if (lane == 0) {
            mbar_arrive(&ring.empty[st]);
        }
    }
    if (!on) return;
    if (a.state_out)
        each_state<NS>(a, k0, col, lane, [&](int i, int j, bool in, long long at) {
            if (in) a.state_out[s_at + at] = S[i][j] * dom.up[j >> 1];
        });
    // padding beyond the last live chunk
    for (int t = a.out ? live * kC + 2 * me + lane / 16 : a.T; t < a.T; t += 2 * kTeam) {
        const int cc = col + lane % 16;
        if (cc < a.V) out[t * o_row + cc] = from_f32<T>(0.f);
    }
}

template <typename T, int KD, bool PAIRS>
__global__ void __launch_bounds__(32 * kTeam * kMostTeams, 1) delta_chunk_fwd_kernel(DeltaArgs a, Prepared w, Saved saved,
                                                                                 int nchunks, unsigned *err) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Ring ring;
    const int tid = threadIdx.x, warp = tid / 32, teams = blockDim.x / (32 * kTeam), team = warp / kTeam;
    const int h = blockIdx.y, b = blockIdx.z;
    after_previous();
    const int n = live_length(a.lengths, b, a.T), live = (n + kC - 1) / kC;
    const int col = (blockIdx.x * teams + team) * 16;
    auto copy = [&](int c) {
        constexpr unsigned KQ = 2 * kq16_elems<T, KD>();
        const long long hc = ((long long)b * a.Hv + h) * nchunks + c;
        const long long kc = ((long long)b * a.Hk + h / (a.Hv / a.Hk)) * nchunks + c;
        return copy_chunk<stages<T, KD>()>(ring, smem, stage_bytes<T, KD>(), c,
                                           Stage{{w.kq16 + kc * (KQ / 2), w.mp16 + hc * kMpElems, w.vec16 + hc * kVec16Elems},
                                                 {KQ, mp16_bytes<T>(), 4 * kVec16Elems}},
                                           err);
    };
    if (tid == 0) {
        ring.init(kTeam * teams);
        if (live > 0) copy(0);
    }
    __syncthreads();
    using Buf = TeamBuf<KD / kTeam / 16>;
    Buf &buf = reinterpret_cast<Buf *>(smem + stages<T, KD>() * stage_bytes<T, KD>())[team];
    walk<T, KD, PAIRS>(a, saved, ring, smem, copy, buf, team, warp % kTeam, nchunks, live, n, h, b, col, err);
}

template <typename T, int KD>
cudaError_t run(const DeltaArgs &a, const Prepared &w, const Saved &saved, cudaStream_t st) {
    constexpr int teams = kMostTeams;
    constexpr size_t smem = stages<T, KD>() * stage_bytes<T, KD>() + teams * sizeof(TeamBuf<KD / kTeam / 16>);
    static_assert(smem <= 227 * 1024 - 256, "shared memory of a CTA");
    const long long dense[3] = {0, (long long)a.Hv * a.V, a.V};
    const bool whole = column_pairs<T>(a.v, a.v_s, a.V) && column_pairs<T>(a.out, dense, a.V);
    auto kern = whole ? delta_chunk_fwd_kernel<T, KD, true> : delta_chunk_fwd_kernel<T, KD, false>;
    const int threads = 32 * kTeam * teams;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), threads, smem, nullptr);
    if (e != cudaSuccess) return e;
    const dim3 grid((a.V + 16 * teams - 1) / (16 * teams), a.Hv, a.B);
    note_launches(1);
    note_kernel("delta_chunk");
    return launch_after(kern, grid, threads, smem, st, a, w, saved, (a.T + kC - 1) / kC, device_error_word());
}

}  // namespace

cudaError_t launch_chunk_fwd(const DeltaArgs &a, dwconv_dtype dt, const Prepared &w, const Saved &saved,
                             cudaStream_t st) {
    auto width = [&](auto t) {
        using E = decltype(t);
        return a.K <= 64 ? run<E, 64>(a, w, saved, st) : run<E, 128>(a, w, saved, st);
    };
    switch (dt) {
        case DWCONV_FP32: return width(float{});
        case DWCONV_FP16: return width(__half{});
        default: return width(__nv_bfloat16{});
    }
}

}  // namespace chunk
}  // namespace dwc
