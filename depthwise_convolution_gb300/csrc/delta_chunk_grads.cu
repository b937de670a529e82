// Backward pass of the chunked gated delta rule, second part: the gradients of
// q, k, g and beta, chunk by chunk with no order between chunks.
//
// With S0 the state before the chunk, dS1 the gradient of the state after it,
// U^ and F of the two walks, per value head (rows are tokens):
//   dP   = dO U^T,  dL = -(beta F) U^T,               (the masked halves)
//   dQ   = scale e^G dO S0^T + (D dP) K,
//   dK_r = -e^G beta F S0^T + (D dL) K,                k as the reader of the state
//   dK_w = e^(G_last - G) U dS1^T + (D dP)^T Q + (D dL)^T K,      k as its writer
//   dbeta_i = F_i . U^_i,
//   dG_i = q_i.dQ_i + k_i.dK_r,i - k_i.dK_w,i,  dG_last += <S1, dS1>,
// the last because e^G_i stands with every read at i and e^-G_j with every
// write at j; dg is the running sum of dG from the end of the chunk.  The
// gradients of q and k before their norms follow from the same row sums.
//
// A CTA takes a chunk of one key head and goes through its value heads, whose
// contributions it adds in fp32 in their order (no atomics).  Sixteen warps: four
// blocks of 16 rows by four quarters of the columns.  The products over V run on
// 64 columns of the images at a time, staged by bulk copies.  Split operands
// (16 bits) where two roundings would meet in one bf16 gradient: U^, D dP, and
// the diagonal blocks that give dbeta; everything with FULL.
//
// What bounds it: latency in one CTA of 16 warps an SM (206 KB of tiles; issue
// 0.34 a cycle, shared memory 58 %), and waves: 32 chunks x 16 key heads, K = V =
// 128, two value heads each, bf16, are 512 CTAs or 3.4 waves in 97 us.  With eight
// warps of halves it took 113, with the totals of the heads before read one pair
// after the other 107, with the copies cut into smaller pieces 115.
#include <algorithm>

#include "delta_chunk_host.cuh"

namespace dwc {
namespace chunk {

namespace {

constexpr int kGradThreads = 512;
constexpr int kVT = 64;  // columns of V a tile holds

template <int KD, bool FULL> struct Plan {
    static constexpr int NT = terms(FULL);
    static constexpr int STAGES = FULL ? 1 : 2;
    // elements of a stage: S0, dS1, U^ (hi, lo), F (hi, lo), dO, then the row factors
    static constexpr int S0 = 0, DS = S0 + NT * kVT * KD, U = DS + NT * kVT * KD, F = U + 2 * kVT * kC,
                         DO = F + 2 * kVT * kC, VEC = DO + NT * kVT * kC, STAGE = VEC + 2 * kVecElems;
    static constexpr int KQ = kq_elems<KD, FULL>();
    static constexpr int D = KQ + STAGES * STAGE;                  // D dP hi, lo, D dL hi (FULL: lo)
    static constexpr int END = D + (FULL ? 4 : 3) * kTile;
    static constexpr size_t bytes = 2 * END;
};

template <typename T, int KD, bool FULL>
__global__ void __launch_bounds__(kGradThreads, 1)
    delta_chunk_grads_kernel(DeltaArgs a, DeltaGrads d, Prepared w, Saved saved, Walked walked, int nchunks,
                             unsigned *err) {
    using L = Plan<KD, FULL>;
    constexpr int NT = L::NT, TILE = kC * KD, NK = KD / 32;  // NK: 8-column tiles of a warp's quarter of K
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __nv_bfloat16 *sm = reinterpret_cast<__nv_bfloat16 *>(smem_raw);
    __shared__ uint64_t bar[2], bar_kq;
    __shared__ float red[4][3][kC], sum[kGradThreads / 32], diag[kC], tot[2][kC];
    __shared__ int gave_up;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, rb = warp % 4, quarter = warp / 4;
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, group = a.Hv / a.Hk;
    after_previous();
    const int n = live_length(a.lengths, b, a.T), t0 = c * kC;
    const int r0 = lane / 4, c0 = 2 * (lane % 4), k0 = quarter * (KD / 4);
    T *dq = static_cast<T *>(d.dq) + ((long long)b * a.T * a.Hk + hk) * a.K;
    T *dk = static_cast<T *>(d.dk) + ((long long)b * a.T * a.Hk + hk) * a.K;
    const long long k_row = (long long)a.Hk * a.K;
    const bool pairs = a.K % 2 == 0 && (reinterpret_cast<size_t>(d.dq) | reinterpret_cast<size_t>(d.dk)) % (2 * sizeof(T)) == 0;
    auto put_gate = [&](void *p, int t, int h, float v) {
        const long long at = ((long long)b * a.T + t) * a.Hv + h;
        if (a.gate_f32) static_cast<float *>(p)[at] = v;
        else static_cast<T *>(p)[at] = from_f32<T>(v);
    };
    const int end = min(a.T, t0 + kC);
    if (t0 >= n) {  // padding only
        for (int t = t0 + warp; t < end; t += kGradThreads / 32) {
            for (int k = lane; k < a.K; k += 32) dq[t * k_row + k] = dk[t * k_row + k] = from_f32<T>(0.f);
            for (int h = lane; h < group; h += 32) {
                put_gate(d.dg, t, hk * group + h, 0.f);
                put_gate(d.dbeta, t, hk * group + h, 0.f);
            }
        }
        return;
    }
    const int v16 = (a.V + 15) / 16 * 16, nvt = (v16 + kVT - 1) / kVT, iters = group * nvt;
    if (tid == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        mbar_init(&bar_kq, 1);
        mbar_fence_init();
        gave_up = 0;
    }
    if (tid < kC) tot[0][tid] = tot[1][tid] = 0.f;
    __syncthreads();
    auto fetch = [&](int it) {  // tile it: value head it / nvt, columns 64 (it % nvt) on
        const int s = it % L::STAGES, vt = it % nvt, rows = min(kVT, v16 - vt * kVT);
        const long long hc = ((long long)b * a.Hv + hk * group + it / nvt) * nchunks + c;
        __nv_bfloat16 *to = sm + L::KQ + s * L::STAGE;
        const unsigned wide = rows * KD * 2, narrow = rows * kC * 2;
        mbar_arrive_expect_tx(&bar[s], 2 * NT * wide + (4 + NT) * narrow + 4 * kVecElems);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const long long at = ((hc * NT + t) * v16 + vt * kVT) * KD;
            bulk_load(to + L::S0 + t * kVT * KD, saved.s + at, wide, &bar[s]);
            bulk_load(to + L::DS + t * kVT * KD, walked.ds + at, wide, &bar[s]);
            bulk_load(to + L::DO + t * kVT * kC, walked.d_o + ((hc * NT + t) * v16 + vt * kVT) * kC, narrow, &bar[s]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const long long at = ((hc * 2 + t) * v16 + vt * kVT) * kC;
            bulk_load(to + L::U + t * kVT * kC, saved.u + at, narrow, &bar[s]);
            bulk_load(to + L::F + t * kVT * kC, walked.f + at, narrow, &bar[s]);
        }
        bulk_load(to + L::VEC, w.vec + hc * kVecElems, 4 * kVecElems, &bar[s]);
    };
    if (tid == 0) {
        mbar_arrive_expect_tx(&bar_kq, 2 * L::KQ);
        bulk_load(sm, w.kq + (((long long)b * a.Hk + hk) * nchunks + c) * L::KQ, 2 * L::KQ, &bar_kq);
        for (int it = 0; it < min(L::STAGES, iters); ++it) fetch(it);
    }
    const __nv_bfloat16 *kt = sm, *qt = sm + NT * TILE;
    __nv_bfloat16 *dp = sm + L::D, *dl = dp + 2 * kTile;
    if (!mbar_wait(&bar_kq, 0)) gave_up = 1;

    float gq[NK][4], gr[NK][4], gw[NK][4];  // dQ, dK_r, dK_w of the value head
    float P[2][4], G[2][4];                 // dO U^^T and F U^^T
    float inner = 0.f;                      // this thread's part of <S0, dS1>
    // a row's value of a [64][KD] tile pair under an accumulator's columns
    auto pair = [&](const __nv_bfloat16 *t, int row, int col) {
        float2 v = unpack_bf16(*reinterpret_cast<const unsigned *>(t + swz<KD>(row, col)));
        if (FULL) {
            const float2 l = unpack_bf16(*reinterpret_cast<const unsigned *>(t + TILE + swz<KD>(row, col)));
            v.x += l.x;
            v.y += l.y;
        }
        return v;
    };
    for (int it = 0; it < iters; ++it) {
        const int s = it % L::STAGES, vt = it % nvt, g = it / nvt;
        if (vt == 0) {
#pragma unroll
            for (int i = 0; i < NK; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) gq[i][j] = gr[i][j] = gw[i][j] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) P[i][j] = G[i][j] = 0.f;
            inner = 0.f;
        }
        if (!mbar_wait(&bar[s], (it / L::STAGES) & 1)) gave_up = 1;
        __nv_bfloat16 *st = sm + L::KQ + s * L::STAGE;
        const __nv_bfloat16 *s0 = st + L::S0, *ds = st + L::DS, *ut = st + L::U, *ft = st + L::F, *ot = st + L::DO;
        const float *vec = reinterpret_cast<const float *>(st + L::VEC);
        const int rows = min(kVT, v16 - vt * kVT);
        for (int v = 0; v < rows; v += 16) {
            // left operands [16 tokens][16 columns] out of [column][token] images
            auto left = [&](const __nv_bfloat16 *t) {
                return ldsm_t(t + swz<kC>(v + nk_row(lane), 16 * rb + nk_col(lane)));
            };
            Frag o[NT], f[2], u[2];
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] = left(ot + t * kVT * kC);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f[t] = left(ft + t * kVT * kC);
                u[t] = left(ut + t * kVT * kC);
            }
#pragma unroll
            for (int p = 0; p < NK / 2; ++p) {
                const int at = swz<KD>(v + kn_row(lane), k0 + 16 * p + kn_col(lane));
                Frag sb[NT], db[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    sb[t] = ldsm_t(s0 + t * kVT * KD + at);
                    db[t] = ldsm_t(ds + t * kVT * KD + at);
                }
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int y = 0; y < NT - x; ++y)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            mma(gq[2 * p + j], o[x], sb[y].r[2 * j], sb[y].r[2 * j + 1]);
                            mma(gr[2 * p + j], f[x], sb[y].r[2 * j], sb[y].r[2 * j + 1]);
                        }
#pragma unroll
                for (int j = 0; j < 2; ++j) mma(gw[2 * p + j], u[0], db[0].r[2 * j], db[0].r[2 * j + 1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) mma(gw[2 * p + j], u[1], db[0].r[2 * j], db[0].r[2 * j + 1]);
                if (FULL) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) mma(gw[2 * p + j], u[0], db[NT - 1].r[2 * j], db[NT - 1].r[2 * j + 1]);
                }
            }
            if (quarter <= rb) {  // 16 columns of the token x token products
                const int at = swz<kC>(v + kn_row(lane), 16 * quarter + kn_col(lane));
                const Frag uh = ldsm_t(ut + at), ul = ldsm_t(ut + kVT * kC + at);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma(P[j], o[0], uh.r[2 * j], uh.r[2 * j + 1]);
                    mma(G[j], f[0], uh.r[2 * j], uh.r[2 * j + 1]);
                    mma(P[j], o[0], ul.r[2 * j], ul.r[2 * j + 1]);
                    if (FULL) mma(P[j], o[NT - 1], uh.r[2 * j], uh.r[2 * j + 1]);
                    if (FULL || quarter == rb) {
                        mma(G[j], f[0], ul.r[2 * j], ul.r[2 * j + 1]);
                        mma(G[j], f[1], uh.r[2 * j], uh.r[2 * j + 1]);
                    }
                }
            }
        }
        // <S0, dS1>: the two images have the same layout
        for (int i = tid; i < rows * KD / 8; i += kGradThreads) {
            auto word = [](const uint4 &v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
            const uint4 xh = reinterpret_cast<const uint4 *>(s0)[i], yh = reinterpret_cast<const uint4 *>(ds)[i];
            uint4 xl, yl;
            if (FULL) {
                xl = reinterpret_cast<const uint4 *>(s0 + kVT * KD)[i];
                yl = reinterpret_cast<const uint4 *>(ds + kVT * KD)[i];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 x = unpack_bf16(word(xh, j)), y = unpack_bf16(word(yh, j));
                if (FULL) {
                    const float2 u = unpack_bf16(word(xl, j)), v = unpack_bf16(word(yl, j));
                    x.x += u.x; x.y += u.y; y.x += v.x; y.y += v.y;
                }
                inner = fmaf(x.x, y.x, fmaf(x.y, y.y, inner));
            }
        }
        if (vt + 1 < nvt) {
            __syncthreads();  // everyone is done with the stage
            if (tid == 0 && it + L::STAGES < iters) fetch(it + L::STAGES);
            continue;
        }

        // The head's sums over V are complete: row factors, masked products.
        const int h = hk * group + g;
        inner *= vec[V_LAST * kC];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = 16 * rb + r0 + 8 * q;
            const float be = vec[V_BETA * kC + r], eq = vec[V_EQ * kC + r], er = -vec[V_EK * kC + r] * be;
            const float ew = vec[V_W * kC + r] * be, nq = vec[V_NQ * kC + r], nk = vec[V_NK * kC + r];
            const float gh = vec[V_GH * kC + r], gl = vec[V_GL * kC + r];
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const float2 kv = pair(kt, r, k0 + 8 * i + c0);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    gq[i][2 * q + j] *= eq;
                    gr[i][2 * q + j] *= er;
                    gw[i][2 * q + j] *= ew;
                }
                inner = fmaf(kv.x, gw[i][2 * q], fmaf(kv.y, gw[i][2 * q + 1], inner));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = 16 * quarter + 8 * i + c0;
                auto two = [&](int which) { return *reinterpret_cast<const float2 *>(vec + which * kC + col); };
                const float2 b2 = two(V_BETA), n2 = two(V_NK), h2 = two(V_GH), l2 = two(V_GL);
                float p[2], l[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int cj = col + j;
                    const float bj = j ? b2.y : b2.x, nj = j ? n2.y : n2.x;
                    const float e = cj <= r ? __expf((gh - (j ? h2.y : h2.x)) + (gl - (j ? l2.y : l2.x))) : 0.f;
                    p[j] = cj <= r ? P[i][2 * q + j] * bj * nq * nj * e : 0.f;
                    l[j] = cj < r ? -G[i][2 * q + j] * be * bj * nk * nj * e : 0.f;
                    if (cj == r) diag[r] = G[i][2 * q + j];
                }
                unsigned hi, lo;
                const int at = swz<kC>(r, col);
                split_bf16(p[0], p[1], hi, lo);
                *reinterpret_cast<unsigned *>(dp + at) = hi;
                *reinterpret_cast<unsigned *>(dp + kTile + at) = lo;
                split_bf16(l[0], l[1], hi, lo);
                *reinterpret_cast<unsigned *>(dl + at) = hi;
                if (FULL) *reinterpret_cast<unsigned *>(dl + kTile + at) = lo;
            }
        }
        __syncthreads();
        // gq += (D dP) K, gr += (D dL) K: columns j up to the row block
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x > rb) continue;
            const int at = swz<kC>(16 * rb + kn_row(lane), 16 * x + kn_col(lane));
            const Frag ph = ldsm(dp + at), pl = ldsm(dp + kTile + at), lh = ldsm(dl + at);
            Frag ll;
            if (FULL) ll = ldsm(dl + kTile + at);
#pragma unroll
            for (int p = 0; p < NK / 2; ++p) {
                const int kat = swz<KD>(16 * x + kn_row(lane), k0 + 16 * p + kn_col(lane));
                const Frag kb = ldsm_t(kt + kat);
                Frag kl;
                if (FULL) kl = ldsm_t(kt + TILE + kat);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma(gq[2 * p + j], ph, kb.r[2 * j], kb.r[2 * j + 1]);
                    mma(gr[2 * p + j], lh, kb.r[2 * j], kb.r[2 * j + 1]);
                    mma(gq[2 * p + j], pl, kb.r[2 * j], kb.r[2 * j + 1]);
                    if (FULL) {
                        mma(gr[2 * p + j], ll, kb.r[2 * j], kb.r[2 * j + 1]);
                        mma(gq[2 * p + j], ph, kl.r[2 * j], kl.r[2 * j + 1]);
                        mma(gr[2 * p + j], lh, kl.r[2 * j], kl.r[2 * j + 1]);
                    }
                }
            }
        }
        // gw += (D dP)^T Q + (D dL)^T K: rows i from the row block on
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x < rb) continue;
            const int at = swz<kC>(16 * x + nk_row(lane), 16 * rb + nk_col(lane));
            const Frag ph = ldsm_t(dp + at), pl = ldsm_t(dp + kTile + at), lh = ldsm_t(dl + at);
            Frag ll;
            if (FULL) ll = ldsm_t(dl + kTile + at);
#pragma unroll
            for (int p = 0; p < NK / 2; ++p) {
                const int kat = swz<KD>(16 * x + kn_row(lane), k0 + 16 * p + kn_col(lane));
                const Frag qb = ldsm_t(qt + kat), kb = ldsm_t(kt + kat);
                Frag ql, kl;
                if (FULL) {
                    ql = ldsm_t(qt + TILE + kat);
                    kl = ldsm_t(kt + TILE + kat);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma(gw[2 * p + j], ph, qb.r[2 * j], qb.r[2 * j + 1]);
                    mma(gw[2 * p + j], pl, qb.r[2 * j], qb.r[2 * j + 1]);
                    mma(gw[2 * p + j], lh, kb.r[2 * j], kb.r[2 * j + 1]);
                    if (FULL) {
                        mma(gw[2 * p + j], ph, ql.r[2 * j], ql.r[2 * j + 1]);
                        mma(gw[2 * p + j], ll, kb.r[2 * j], kb.r[2 * j + 1]);
                        mma(gw[2 * p + j], lh, kl.r[2 * j], kl.r[2 * j + 1]);
                    }
                }
            }
        }
        // Row sums with q and k; dQ and dK go to the running totals.
        float *total = d.totals ? d.totals + (((long long)b * a.Hk + hk) * nchunks + c) * 2 * TILE : nullptr;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = 16 * rb + r0 + 8 * q;
            float z[3] = {0.f, 0.f, 0.f};
            float2 was[NK][2];  // totals of the heads before, all reads on their way at once
            if (g > 0)
#pragma unroll
                for (int i = 0; i < NK; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        was[i][j] = *reinterpret_cast<const float2 *>(total + j * TILE + r * KD + k0 + 8 * i + c0);
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int col = k0 + 8 * i + c0;
                const float2 qv = pair(qt, r, col), kv = pair(kt, r, col);
                z[0] = fmaf(qv.x, gq[i][2 * q], fmaf(qv.y, gq[i][2 * q + 1], z[0]));
                z[1] = fmaf(kv.x, gr[i][2 * q], fmaf(kv.y, gr[i][2 * q + 1], z[1]));
                z[2] = fmaf(kv.x, gw[i][2 * q], fmaf(kv.y, gw[i][2 * q + 1], z[2]));
                float2 tq = make_float2(gq[i][2 * q], gq[i][2 * q + 1]);
                float2 tk = make_float2(gr[i][2 * q] + gw[i][2 * q], gr[i][2 * q + 1] + gw[i][2 * q + 1]);
                if (g > 0) {
                    tq.x += was[i][0].x; tq.y += was[i][0].y; tk.x += was[i][1].x; tk.y += was[i][1].y;
                }
                if (g + 1 < group) {
                    *reinterpret_cast<float2 *>(total + r * KD + col) = tq;
                    *reinterpret_cast<float2 *>(total + TILE + r * KD + col) = tk;
                }
                gq[i][2 * q] = tq.x; gq[i][2 * q + 1] = tq.y;
                gr[i][2 * q] = tk.x; gr[i][2 * q + 1] = tk.y;
            }
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                z[j] += __shfl_xor_sync(0xFFFFFFFFu, z[j], 1);
                z[j] += __shfl_xor_sync(0xFFFFFFFFu, z[j], 2);
                if (lane % 4 == 0) red[quarter][j][r] = z[j];
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) inner += __shfl_xor_sync(0xFFFFFFFFu, inner, o);
        if (lane == 0) sum[warp] = inner;
        __syncthreads();
        if (warp == 0) {
            float dg[2], last = 0.f;
#pragma unroll
            for (int i = 0; i < kGradThreads / 32; ++i) last += sum[i];
            const int r = 2 * lane;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float z[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    z[i] = (red[0][i][r + j] + red[1][i][r + j]) + (red[2][i][r + j] + red[3][i][r + j]);
                tot[0][r + j] += z[0];
                tot[1][r + j] += z[1] + z[2];
                dg[j] = z[0] + z[1] - z[2];
            }
            // dG of a token counts for its own g and every earlier one of the chunk
            float run = dg[0] + dg[1];
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const float dn = __shfl_down_sync(0xFFFFFFFFu, run, o);
                if (lane + o < 32) run += dn;
            }
            const float next = __shfl_down_sync(0xFFFFFFFFu, run, 1);
            dg[0] = run + last;
            dg[1] += (lane < 31 ? next : 0.f) + last;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = t0 + r + j;
                // nothing comes through a decay of zero or out of an empty past; the sum above has the roundings
                // of terms that cancel
                const float *gh = vec + V_GH * kC + r + j, *gl = vec + V_GL * kC + r + j;
                const float g = r + j ? (gh[0] - gh[-1]) + (gl[0] - gl[-1]) : gh[0] + gl[0];
                if (__expf(g) == 0.f || (t == 0 && !a.state)) dg[j] *= 0.f;  // a NaN stays one
                if (t < end) {
                    put_gate(d.dg, t, h, t < n ? dg[j] : 0.f);
                    put_gate(d.dbeta, t, h, t < n ? diag[r + j] : 0.f);
                }
            }
        }
        if (g + 1 == group) {
            __syncthreads();  // tot is complete
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = 16 * rb + r0 + 8 * q, t = t0 + r;
                if (t >= end) continue;
                const float iq = vec[V_IQ * kC + r], ik = vec[V_NK * kC + r];
                const float cq = a.qk_norm ? tot[0][r] * iq * iq : 0.f, ck = a.qk_norm ? tot[1][r] * ik * ik : 0.f;
#pragma unroll
                for (int i = 0; i < NK; ++i) {
                    const int col = k0 + 8 * i + c0;
                    const float2 qv = pair(qt, r, col), kv = pair(kt, r, col);
                    const float x[2] = {gq[i][2 * q] - cq * qv.x, gq[i][2 * q + 1] - cq * qv.y};
                    const float y[2] = {gr[i][2 * q] - ck * kv.x, gr[i][2 * q + 1] - ck * kv.y};
                    if (pairs) {
                        if (col < a.K) {
                            store_pack<T, 2>(dq + t * k_row + col, Pack<T, 2>::of(x));
                            store_pack<T, 2>(dk + t * k_row + col, Pack<T, 2>::of(y));
                        }
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (col + j < a.K) {
                            dq[t * k_row + col + j] = from_f32<T>(x[j]);
                            dk[t * k_row + col + j] = from_f32<T>(y[j]);
                        }
                }
            }
        }
        __syncthreads();  // the stage, the masked products and the sums are free
        if (tid == 0 && it + L::STAGES < iters) fetch(it + L::STAGES);
    }
    if (tid == 0 && gave_up) report_timeout(err);
}

template <typename T, int KD>
cudaError_t run(const DeltaArgs &a, const DeltaGrads &d, const Prepared &w, const Saved &saved, const Walked &walked,
                cudaStream_t st) {
    constexpr bool FULL = !std::is_same<T, __nv_bfloat16>::value;
    constexpr size_t smem = Plan<KD, FULL>::bytes;
    auto kern = delta_chunk_grads_kernel<T, KD, FULL>;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void *>(kern), kGradThreads, smem, nullptr);
    if (e != cudaSuccess) return e;
    const int n = (a.T + kC - 1) / kC;
    note_launches(1);
    note_kernel("delta_chunk_bwd");
    return launch_after(kern, dim3(n, a.Hk, a.B), kGradThreads, smem, st, a, d, w, saved, walked, n, device_error_word());
}

}  // namespace

cudaError_t launch_chunk_grads(const DeltaArgs &a, const DeltaGrads &d, dwconv_dtype dt, const Prepared &w,
                               const Saved &saved, const Walked &walked, cudaStream_t st) {
    auto width = [&](auto t) {
        using E = decltype(t);
        return a.K <= 64 ? run<E, 64>(a, d, w, saved, walked, st) : run<E, 128>(a, d, w, saved, walked, st);
    };
    switch (dt) {
        case DWCONV_FP32: return width(float{});
        case DWCONV_FP16: return width(__half{});
        default: return width(__nv_bfloat16{});
    }
}

}  // namespace chunk
}  // namespace dwc
