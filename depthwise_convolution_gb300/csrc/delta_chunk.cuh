// Pieces shared by the chunked kernels of the gated delta rule.
//
// A chunk is 64 tokens.  With G the running sum of g in the chunk (first token
// included), D_ij = e^(G_i - G_j) and L_ij = D_ij k_i.k_j for j < i, the rows
// u_t = beta_t (v_t - e^g_t S_(t-1)^T k_t) of a chunk solve a triangular system:
//   R  = V - e^G K S0,   U^ = R - M (beta R),   U = beta U^,
//   M  = (I + L beta)^-1 L   (strictly lower triangular, no division by beta),
//   O  = scale e^G Q S0 + P U,   P_ij = scale D_ij q_i.k_j  for j <= i,
//   S1 = e^G_last S0 + (e^(G_last - G) K)^T U.
// Every exponent is a sum of log decays over a stretch of tokens, never the
// difference of two exponentials, so nothing overflows when g <= 0.
//
// Operands of matrix instructions have 16 bits and split values enter as
// hi + lo with lo = round(x - hi); a product of two split values drops lo lo.
//
// The forward pass computes with fp16 operands (11 bits, split 22): k and q per
// token are brought to magnitudes in [1, 2), the state and its updates per
// column to a range around 1 by powers of two, and the factors are undone in
// fp32, where the norms, decays and beta are applied as row factors too.  bf16
// and fp16 inputs are exact in such a row (to 2^-25 of its largest value), so
// states carry the error of fp32 arithmetic; fp32 inputs are split.  Rows of P and M
// are stored over the tokens' key and query lengths, where they are at most
// about 1.  Where only a bf16 output depends on it, an operand is hi only.
//
// The backward pass computes with bf16 operands (8 bits, split 16): gradients
// have no such scale, and its products run over the columns, whose factors
// could not be taken out.  bf16 inputs are exact; with fp16 and fp32 inputs
// (FULL) every operand is split.
#pragma once

#include "delta.cuh"
#include "mma_common.cuh"
#include "tma.cuh"

namespace dwc {
namespace chunk {

constexpr int kC = kDeltaChunk;
constexpr int kTile = kC * kC;  // elements of an M^T or P tile

// Tiles are images of shared memory: rows of W bf16, the 16-byte units of row
// r permuted by r % 8 so that ldmatrix reads 8 rows without bank conflicts.
// They are written and read by bulk copies as they are.
template <int W> __device__ __forceinline__ int swz(int r, int c) {
    static_assert(W % 64 == 0, "rows of whole 128-byte lines");
    return r * W + ((((c >> 3) ^ (r & 7)) << 3) | (c & 7));
}

// Row factors per chunk and value head, floats.  l_k = |k| as the rule uses it
// (1 with the norms), r_q = 1 / |q|, 2^a and 2^b the scales of the rows of k and q:
//   forward: [0] l_k beta, [1] e^G of the key a row of the tile stands for, [2] e^G r_q 2^-b,
//   [3] beta e^(G_last - G) of the key, [4] scale l_q, [5] e^G_last everywhere;
constexpr int kVecs16 = 6;
enum { F_LB = 0, F_EK = 1, F_EQ = 2, F_WB = 3, F_FQ = 4, F_LAST = 5 };
//   backward: [0] beta, [1] e^G |k|^-1, [2] e^G scale |q|^-1,
// [3] e^(G_last - G) |k|^-1, [4] |k|^-1, [5] scale |q|^-1, [6] e^G_last everywhere,
// [7] |q|^-1, [8] and [9] G as hi + lo.
constexpr int kVecs = 10;
enum { V_BETA = 0, V_EK = 1, V_EQ = 2, V_W = 3, V_NK = 4, V_NQ = 5, V_LAST = 6, V_IQ = 7, V_GH = 8, V_GL = 9 };

// What the preparing kernel leaves per chunk; NT = terms of an input operand.
// kq, mp, vec serve the backward pass (null: not wanted).
struct Prepared {
    __half *kq16;        // [B][Hk][n][K: NT16 tiles of 64 x KD, then Q: NT16 tiles]
    __half *mp16;        // [B][Hv][n][l_k M^T hi, lo (rows over l_k), P hi, lo (over l_q l_k)]
    float *vec16;        // [B][Hv][n][kVecs16][64]
    __nv_bfloat16 *kq;   // [B][Hk][n][K: NT tiles of 64 x KD, then Q: NT tiles]
    __nv_bfloat16 *mp;   // [B][Hv][n][M^T hi, lo, P hi, lo]; blocks (of 16) above P's diagonal hold nothing
    float *vec;          // [B][Hv][n][kVecs][64]
};

struct Frag {
    unsigned r[4];
};

constexpr float kNan = __builtin_nanf("");
__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) < __int_as_float(0x7F800000); }
__device__ __forceinline__ float finite_or_zero(float v) { return is_finite(v) ? v : 0.f; }
// The largest of three (NaN if one is NaN): one instruction.
__device__ __forceinline__ float max_or_nan(float a, float b, float c) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// 2^-e and 2^e for m in [2^e, 2^(e+1)); 1 for zero and subnormals.
__device__ __forceinline__ void pow2_scale(float m, float &down, float &up) {
    unsigned e = __float_as_uint(m) >> 23;
    e = e == 0 ? 127 : e > 253 ? 253 : e;
    down = __uint_as_float((254 - e) << 23);
    up = __uint_as_float(e << 23);
}
__device__ __forceinline__ unsigned pack_half(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&v);
}
__device__ __forceinline__ void split_half(float a, float b, unsigned &hi, unsigned &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const unsigned *>(&h);
    lo = pack_half(a - f.x, b - f.y);
}
// Two accumulator tiles (columns 2s, 2s + 1 of a row of tiles) as the left
// operand of k-step s, hi and lo.
__device__ __forceinline__ void to_frags16(const float (&t0)[4], const float (&t1)[4], Frag &hi, Frag &lo) {
    split_half(t0[0], t0[1], hi.r[0], lo.r[0]);
    split_half(t0[2], t0[3], hi.r[1], lo.r[1]);
    split_half(t1[0], t1[1], hi.r[2], lo.r[2]);
    split_half(t1[2], t1[3], hi.r[3], lo.r[3]);
}
// d (16 x 8) += a (16 x 16) b (16 x 8), fp16 operands.
__device__ __forceinline__ void mma16(float (&d)[4], const Frag &a, unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.r[0]), "r"(a.r[1]), "r"(a.r[2]), "r"(a.r[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ Frag ldsm(const void *p) {
    Frag f;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(f.r[0]), "=r"(f.r[1]), "=r"(f.r[2]), "=r"(f.r[3])
                 : "r"(smem_addr(p)));
    return f;
}
__device__ __forceinline__ Frag ldsm_t(const void *p) {
    Frag f;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(f.r[0]), "=r"(f.r[1]), "=r"(f.r[2]), "=r"(f.r[3])
                 : "r"(smem_addr(p)));
    return f;
}

// d (16 x 8) += a (16 x 16) b (16 x 8).  Not volatile: the compiler may move it
// between the loads of later operands.
__device__ __forceinline__ void mma(float (&d)[4], const Frag &a, unsigned b0, unsigned b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.r[0]), "r"(a.r[1]), "r"(a.r[2]), "r"(a.r[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&v);
}
__device__ __forceinline__ float2 unpack_bf16(unsigned v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
// hi and lo words of a pair.
__device__ __forceinline__ void split_bf16(float a, float b, unsigned &hi, unsigned &lo) {
    hi = pack_bf16(a, b);
    const float2 h = unpack_bf16(hi);
    lo = pack_bf16(a - h.x, b - h.y);
}

// Accumulator tiles (16 x 8 each) -> operand fragment of 16 x 16: tiles 2s and
// 2s + 1 of a row of tiles are the columns of k-step s.
__device__ __forceinline__ void to_frags(const float (&t0)[4], const float (&t1)[4], Frag &hi, Frag &lo) {
    split_bf16(t0[0], t0[1], hi.r[0], lo.r[0]);
    split_bf16(t0[2], t0[3], hi.r[1], lo.r[1]);
    split_bf16(t1[0], t1[1], hi.r[2], lo.r[2]);
    split_bf16(t1[2], t1[3], hi.r[3], lo.r[3]);
}
// Where a lane points ldmatrix for the 16 x 16 block at (r0, c0) of a tile:
//   nk: the block is [n][k] (rows are n), registers = b0, b1 of n-tile r0 and
//       b0, b1 of n-tile r0 + 8 (plain), or the A operand's a0, a2, a1, a3;
//   kn: the block is [k][n] (rows are k), read with .trans: b0, b1 of n-tile
//       c0 and of n-tile c0 + 8.
__device__ __forceinline__ int nk_row(int lane) { return (lane & 7) + ((lane >> 4) << 3); }
__device__ __forceinline__ int nk_col(int lane) { return ((lane >> 3) & 1) << 3; }
__device__ __forceinline__ int kn_row(int lane) { return (lane & 7) + (((lane >> 3) & 1) << 3); }
__device__ __forceinline__ int kn_col(int lane) { return (lane >> 4) << 3; }

// Untiled bulk copies: 16-byte aligned addresses and sizes.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, const void *src, unsigned bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(smem_addr(src)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

__host__ __device__ constexpr int terms(bool full) { return full ? 2 : 1; }
template <int KD, bool FULL> __host__ __device__ constexpr int kq_elems() { return 2 * terms(FULL) * kC * KD; }
constexpr int kMpElems = 4 * kTile;
constexpr int kVec16Elems = kVecs16 * kC;
// fp16 terms of an input operand of the forward pass, and elements of its K and Q tiles
template <typename T> __host__ __device__ constexpr int terms16() { return sizeof(T) == 4 ? 2 : 1; }
template <typename T, int KD> __host__ __device__ constexpr int kq16_elems() { return 2 * terms16<T>() * kC * KD; }
constexpr int kVecElems = kVecs * kC;

// Operands that only a bf16 output depends on are hi only: the last tile (P lo)
// is then neither written nor read.
template <typename T> __host__ __device__ constexpr bool fine_out() { return !std::is_same<T, __nv_bfloat16>::value; }
template <typename T> __host__ __device__ constexpr unsigned mp16_bytes() { return 2 * (fine_out<T>() ? 4 : 3) * kTile; }

}  // namespace chunk
}  // namespace dwc
