// delta_util.cuh -- what the chunked kernels of the gated delta rule share:
// the chunk's formulas, the number format, the workspace, warp-level products.
//
// Within a chunk of C = 64 tokens, with G_i the sum of g up to token i,
// D_ij = exp(G_i - G_j) for i >= j, M_ij = D_ij (k_i . k_j) for i > j:
//     T = (I + diag(beta) M)^-1                       (unit lower triangular)
//     R = V - exp(G) (K S0)                            (rows scaled)
//     U = T diag(beta) R                               (the corrections u_t)
//     O = exp(G) (Q S0) + P U,  P_ij = D_ij (q_i . k_j), i >= j
//     S1 = exp(G_C) S0 + K^T diag(exp(G_C - G)) U.
// Every exponent is a sum of g over tokens of the chunk, so never positive.
//
// Numbers.  The tensor cores multiply fp16.  What is computed (S, R, U, T, P and
// the gradients) is held in fp32 and enters a product as two fp16 terms, hi + lo,
// 22 bits: x y = hi hi + hi lo + lo hi (two bf16 terms carry 16 bits, which the
// gradients of the gates, differences of sums, do not survive).  Each addition
// in the tensor cores rounds towards zero, a bias of up to 2^-23 of the sum that
// adds up over them.  So where the gradients come from, products of low terms go
// first, onto a small sum, and sums over groups are taken in fp32 outside (dbeta
// off by 4e-7 instead of 6e-7, dg by 4e-7 instead of 7e-7).  fp16 has a
// narrow range, so everything is brought near one by powers of two, which are
// exact:
//   * a key k_i = s_i k'_i with its largest element in [1, 2) (a query likewise);
//     the rule for k' has beta' = beta s^2, v' = v / s, u' = s u, and the same S
//     and G;
//   * S (and its gradient) is scaled by the largest value of a half of its rows,
//     R and U (dU and Y) by a bound on theirs: the largest of beta' V' and of S,
//     times that of beta'.  beta' |S k'| <= 2 sqrt(dk) max |S| for beta |k|^2 <= 2,
//     and |K' dS| <= 2 dk max |dS|: the scale leaves R below 2^10 and dU below
//     2^14, and a value 2^-6 of the bound still has its 22 bits.
//   * what passes a gate on its way to the state (exp(G_C - G) U, exp(G) dO',
//     exp(G) beta' Y) by the largest value after the gate.
// What this leaves is relative to the largest value of a tile: a contribution that
// decays within its chunk below 2^-24 of another one beside it is lost.
// A bf16 output is the fp32 one rounded.  (With one term of S, U and P, 2^-12 each,
// it differed from that by 1.0e-3 of its norm; 4 x 2047, 16 heads of 128 / 128: 187 us
// instead of 203.)
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_util.cuh"
#include "tmap.h"

namespace ret {
namespace delta {

constexpr int C = 64;              // tokens of a chunk
constexpr int kTile = C * C * 2;   // bytes of a 64 x 64 fp16 tile (128-byte rows, swizzled)
// Gates of a chunk, 64 values each: in fp32 exp(G), exp(G_C - G), beta', 1 / s
// of the keys, s of the queries, the largest |beta'| of each half; then G in 64
// bits.
constexpr int gEG = 0, gEC = C, gBeta = 2 * C, gIk = 3 * C, gSq = 4 * C, gMax = 5 * C;
constexpr int kGates = 5 * C * 4 + 16;
constexpr int kGateRow = kGates + C * 8;
// Below this a decay is zero in fp32; keeps -inf out of the sums.
constexpr float kMinG = -128.f;

inline int chunks_of(int N) { return (N + C - 1) / C; }

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
    return lengths ? max(0, min(lengths[b], N)) : N;
}

// The workspace.  Per (sequence, key head, chunk): K', Q' [dk/64][64][128 B].
// Per (sequence, head, chunk): T hi, T lo, P hi, P lo; the gates.
struct Tables {
    uint8_t *keys, *tiles, *gates;
};
inline size_t table_bytes(const DeltaArgs& a) {
    const size_t nc = chunks_of(a.N);
    return a.B * nc * ((size_t)a.H * (4 * kTile + kGateRow) + (size_t)a.Hk * 4 * C * a.dk);
}
inline Tables tables_at(const DeltaArgs& a, void* ws) {
    const size_t nc = chunks_of(a.N);
    Tables t;
    t.keys = reinterpret_cast<uint8_t*>(ws);
    t.tiles = t.keys + a.B * nc * a.Hk * 4 * C * a.dk;
    t.gates = t.tiles + a.B * nc * a.H * 4 * kTile;
    return t;
}

// ------------------------------------------------------- warp-level products

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 in, fp32 accumulate.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with D[16 x 8] = A B.
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
        "%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// A block row of products: D[2 p], D[2 p + 1] += A B[p] for p0 <= p < p1.  One
// accumulator comes up again after all the others: a product takes about four
// issue slots of the tensor pipe until its sum can be added to (measured, clocks
// per product on a sub-partition: 23 back to back, 12.4, 9.3, 8.7 and 8.4 with
// 2, 4, 8 and 16 accumulators in turn).
template <int P0, int P1>
__device__ __forceinline__ void mma_row(float (&d)[8][4], const uint32_t (&a)[4], const uint32_t (&b)[4][4]) {
#pragma unroll
    for (int p = P0; p < P1; p++) {
        mma(d[2 * p], a, b[p][0], b[p][1]);
        mma(d[2 * p + 1], a, b[p][2], b[p][3]);
    }
}
__device__ __forceinline__ void add_scaled(float (&d)[4], const float (&x)[4], float s) {
#pragma unroll
    for (int e = 0; e < 4; e++) d[e] = fmaf(s, x[e], d[e]);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
// Transpose of an 8 x 8 matrix of 16-bit values held across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Offset of 16-byte piece `c` (8 values) of row `r` in slabs of ROWS rows of
// 128 swizzled bytes.
template <int ROWS = C>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    return (uint32_t)(c >> 3) * (ROWS * 128u) + (uint32_t)r * 128u + (uint32_t)(((c ^ r) & 7) << 4);
}
// The four 8 x 8 blocks of a 16-row, 16-column part at (row, piece):
// rows first (blocks 0, 1 side by side): a B operand whose rows are n, or,
// transposed, an A operand whose rows are k.
template <int ROWS = C>
__device__ __forceinline__ uint32_t at_n(uint32_t base, int row, int piece, int lane) {
    const int m = lane >> 3;
    return base + tile_at<ROWS>(row + ((m >> 1) << 3) + (lane & 7), piece + (m & 1));
}
// columns first (blocks 0, 1 on top of each other): an A operand whose rows
// are m, or, transposed, a B operand whose rows are k.
template <int ROWS = C>
__device__ __forceinline__ uint32_t at_k(uint32_t base, int row, int piece, int lane) {
    const int m = lane >> 3;
    return base + tile_at<ROWS>(row + ((m & 1) << 3) + (lane & 7), piece + (m >> 1));
}

__device__ __forceinline__ uint32_t pack_h2(float x0, float x1) {
    const __half2 h = __floats2half2_rn(x0, x1);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// x = hi + lo, pairs of fp16.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    hi = pack_h2(x0, x1);
    const float2 h = unpack_h2(hi);
    lo = pack_h2(x0 - h.x, x1 - h.y);
}
// The A operand (16 x 16) from two neighbouring accumulator tiles, scaled by s.
__device__ __forceinline__ void split_a(const float (&x)[4], const float (&y)[4], float s, uint32_t (&hi)[4],
                                        uint32_t (&lo)[4]) {
    split2(x[0] * s, x[1] * s, hi[0], lo[0]);
    split2(x[2] * s, x[3] * s, hi[1], lo[1]);
    split2(y[0] * s, y[1] * s, hi[2], lo[2]);
    split2(y[2] * s, y[3] * s, hi[3], lo[3]);
}

// The power of two that brings a largest value m >= 0 into [4, 8), and its
// inverse.  (Headroom to fp16's 65,504: sums of 64 terms and the solve.)
__device__ __forceinline__ float scale_for(float m, float& inverse) {
    const int e = (__float_as_int(m) >> 23) & 255;
    const int s = e == 0 || e == 255 ? 127 : min(max(256 - e, 27), 227);
    inverse = __int_as_float((254 - s) << 23);
    return __int_as_float(s << 23);
}
// The same for a bound: into [8, 16).
__device__ __forceinline__ float bound_scale(float m, float& inverse) {
    const float s = scale_for(m, inverse);
    inverse *= 0.5f;
    return 2.f * s;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// The scale of a warp's values (a pair of accumulator tiles).
__device__ __forceinline__ float scale_of(const float (&x)[4], const float (&y)[4], float& inverse) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; e++) m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));
    return scale_for(warp_max(m), inverse);
}

// Untiled asynchronous copy of `bytes` (a multiple of 16) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

// The chunk tables (k_delta_prep.cu).
ret_status launch_prep(const DeltaArgs& a, const Tables& t, cudaStream_t s);

// What the backward's two chains (k_delta_chunk.cu) keep, one record per
// (chunk, group of 16 value columns); the values transposed (a row per value
// column), hi then lo:
//   s   [hi, lo][dk/64][16][64]  the state before the chunk
//   ds  the same                 the gradient of the state after it
//   u   [hi, lo][16][64]         the corrections U'
//   y   the same                 dY = T^T dU
//   o   [16][64]                 dO' = s_q dO, one term
//   f   7 fp32: the inverse scales of s and ds (a half of dk each), u, y, o
template <int DK>
struct Record {
    static constexpr int s = 0, ds = 64 * DK, u = 128 * DK, y = u + 4096, o = y + 4096, f = o + 2048, bytes = f + 128;
};
inline size_t record_bytes(int dk) { return 128 * (size_t)dk + 4096 * 2 + 2048 + 128; }
enum : int { fS = 0, fDs = 2, fU = 4, fY = 5, fO = 6 };
__host__ __device__ __forceinline__ int groups_of(int dv) { return (dv + 15) / 16; }
ret_status launch_chains(const DeltaArgs& a, const Tables& t, uint8_t* records, cudaStream_t s);

}  // namespace delta
}  // namespace ret
