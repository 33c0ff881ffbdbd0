// delta_util.cuh -- what the chunked kernels of the gated delta rule share:
// the chunk's formulas, the workspace tiles, warp-level matrix products and
// the split of an fp32 value into two bf16 terms.
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
// Precision.  q, k, v are bf16, everything computed from them is held in fp32
// and enters a matrix product as hi + lo, two bf16 terms whose sum is within
// 2^-17 of the value: x y is hi hi + hi lo + lo hi (one product less where a
// factor is an input, exact in bf16).  One bf16 term would leave the carried
// state 2^-9 off after every chunk.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "tc_util.cuh"
#include "tmap.h"

namespace ret {
namespace delta {

constexpr int C = 64;              // tokens of a chunk
constexpr int kTile = C * C * 2;   // bytes of a 64 x 64 bf16 tile (128-byte rows, swizzled)
constexpr int kSlice = 64;         // value columns of a tile
constexpr int kGates = 3 * C * 4;       // bytes: exp(G), exp(G_C - G), beta in fp32
constexpr int kGateRow = kGates + C * 8;  // and G in 64 bits
// Below this a decay is zero in fp32; keeps -inf out of the sums.
constexpr float kMinG = -128.f;

inline int chunks_of(int N) { return (N + C - 1) / C; }
inline int slices_of(int dv) { return (dv + kSlice - 1) / kSlice; }

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
    return lengths ? max(0, min(lengths[b], N)) : N;
}

// ------------------------------------------------------- warp-level products

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 in, fp32 accumulate.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Address of 16-byte piece `c` (8 bf16) of row `r` of a tile of 64-row slabs
// with 128-byte swizzled rows.
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int r, int c) {
    return base + (uint32_t)(c >> 3) * 8192u + (uint32_t)r * 128u + (uint32_t)(((c ^ r) & 7) << 4);
}

// The four 8 x 8 blocks of a 16-row, 16-column part at (row, piece):
// rows first (blocks 0, 1 side by side): a B operand whose rows are n.
__device__ __forceinline__ uint32_t at_n(uint32_t base, int row, int piece, int lane) {
    const int m = lane >> 3;
    return tile_at(base, row + ((m >> 1) << 3) + (lane & 7), piece + (m & 1));
}
// columns first (blocks 0, 1 on top of each other): an A operand, or
// (transposed) a B operand whose rows are k.
__device__ __forceinline__ uint32_t at_k(uint32_t base, int row, int piece, int lane) {
    const int m = lane >> 3;
    return tile_at(base, row + ((m & 1) << 3) + (lane & 7), piece + (m >> 1));
}

// x = hi + lo in bf16 pairs.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    hi = tc::pack_bf16x2(x0, x1);
    lo = tc::pack_bf16x2(x0 - tc::bf16lo(hi), x1 - tc::bf16hi(hi));
}
// The A operand (16 x 16) from two neighbouring accumulator tiles.
__device__ __forceinline__ void split_a(const float (&x)[4], const float (&y)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(x[0], x[1], hi[0], lo[0]);
    split2(x[2], x[3], hi[1], lo[1]);
    split2(y[0], y[1], hi[2], lo[2]);
    split2(y[2], y[3], hi[3], lo[3]);
}
__device__ __forceinline__ void round_a(const float (&x)[4], const float (&y)[4], uint32_t (&hi)[4]) {
    hi[0] = tc::pack_bf16x2(x[0], x[1]);
    hi[1] = tc::pack_bf16x2(x[2], x[3]);
    hi[2] = tc::pack_bf16x2(y[0], y[1]);
    hi[3] = tc::pack_bf16x2(y[2], y[3]);
}

// Untiled asynchronous copy of `bytes` (a multiple of 16) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

// Clears rows L .. 63 of a tile of `pieces` 16-byte pieces a row (a warp's work).
__device__ __forceinline__ void clear_rows(uint8_t* tile, int L, int pieces, int lane) {
    for (int i = lane; i < (C - L) * pieces; i += 32)
        *reinterpret_cast<uint4*>(tile + tile_at(0, L + i / pieces, i % pieces)) = make_uint4(0, 0, 0, 0);
}

// [B, N, heads, d] bf16 as a {d, heads, N, B} tensor, boxes of one head's
// chunk, 64 columns wide.
inline bool chunk_map(CUtensorMap* m, const void* p, int B, int N, int heads, int d) {
    const uint64_t dims[4] = {(uint64_t)d, (uint64_t)heads, (uint64_t)N, (uint64_t)B};
    const uint64_t strides[3] = {(uint64_t)d * 2, (uint64_t)heads * d * 2, (uint64_t)N * heads * d * 2};
    const uint32_t box[4] = {64, 1, (uint32_t)C, 1};
    return make_tmap_bf16(m, p, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The chunk tables (k_delta_chunk.cu): T, P and the gates of every chunk.
ret_status launch_prep(const DeltaArgs& a, uint8_t* tiles, uint8_t* gates, cudaStream_t s);

// The backward's two chains (k_delta_chunk.cu).  Per (chunk, slice of 64 value
// columns), transposed (a row per value column), hi then lo:
//   s   [dk/64][64][128 B]  the state before the chunk
//   u   [64][128 B]         the corrections
//   ds  [dk/64][64][128 B]  the gradient of the state after the chunk
//   y   [64][128 B]         dY = T^T dU
struct Kept {
    uint8_t *s, *u, *ds, *y;
};
ret_status launch_chains(const DeltaArgs& a, const uint8_t* tiles, const uint8_t* gates, const Kept& kept, cudaStream_t s);

}  // namespace delta
}  // namespace ret
