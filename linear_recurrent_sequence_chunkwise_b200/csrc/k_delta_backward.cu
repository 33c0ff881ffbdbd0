// k_delta_backward.cu -- gradients of the gated delta rule's chunked forward
// (notation: delta_util.cuh).  Three launches: the chunk tables, the two chains
// of k_delta_chunk.cu side by side (states before each chunk, corrections U;
// gradients of the states after each chunk, dY), and this pass, chunk by chunk
// in parallel.  With W = dY U^T, E = dO U^T, row i of a chunk:
//     dq_i = exp(G_i) dO_i S0^T + sum_{j<=i} E_ij D_ij k_j
//     r_i  = -(exp(G_i) dY_i S0^T + sum_{j<i} W_ij D_ij k_j)
//     w_j  = sum_{i>=j} E_ij D_ij q_i - sum_{i>j} beta_i W_ij D_ij k_i + exp(G_C - G_j) U_j dS1^T
//     dk   = beta r + w,  dv = beta dY,  dbeta_i = dY_i . v_i + k_i . r_i
//     dG_i = q_i . dq_i + beta_i k_i . r_i - k_i . w_i   (a row's decay multiplies
//            what it reads and divides what it writes), the last row also <dS1, S1>,
//     dg   = sums of dG to the end of the chunk,
//     <dS1, S1> = exp(G_C) <dS1, S0> + sum_j k_j . (exp(G_C - G_j) U_j dS1^T).
// A key head's gradient is the sum over its value heads: one block takes them
// all, one after the other, so the order is fixed.
//
// A warp takes 16 rows and a share of the dk columns; the five products over
// dv accumulate in registers while slices of 64 value columns pass through
// shared memory, then the two 64 x 64 score tiles take the place of dY and U,
// and K and Q that of S0.
#include <algorithm>

#include "delta_util.cuh"

namespace ret {

static __device__ int g_grad_err = 0;

cudaError_t read_clear_error_delta_grads(int* flag) {
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_grad_err, sizeof(int));
    if (e == cudaSuccess && *flag) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_grad_err, &zero, sizeof(int));
    }
    return e;
}

namespace delta {

namespace {

struct GradArgs {
    const uint8_t* gates;
    const int* lengths;
    const __nv_bfloat16* v;
    Kept kept;
    void *dq, *dk, *dv;
    float *dg, *dbeta;
    int N, nc, Hk, H, dv_dim;
};

template <int DK>
struct Grad {
    static constexpr int NH = DK == 256 ? 4 : 2;       // column shares
    static constexpr int threads = 4 * NH * 32;
    static constexpr int DW = DK / NH;                 // dk columns of a warp
    static constexpr int JW = C / NH;                  // score columns of a warp
    static constexpr int oO = 0, O = C * kSlice * 2;   // dO
    static constexpr int oY = O, Y = 2 * kTile;        // dY hi, lo; later E D hi, lo
    static constexpr int oU = oY + Y, U = 2 * kTile;   // U hi, lo; later W D hi, lo
    static constexpr int oS = oU + U, S = 4 * C * DK;  // S0 hi, lo; later K and Q
    static constexpr int oD = oS + S, D = 4 * C * DK;  // dS1 hi, lo
    static constexpr int oG = oD + D;                  // the chunk's gates
    static constexpr int smem = oG + 2048 + 1024;
};

template <typename T>
__device__ __forceinline__ void st_pair(T* p, float x, float y) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(p) = make_float2(x, y);
    else *reinterpret_cast<uint32_t*>(p) = tc::pack_bf16x2(x, y);
}

template <int DK, typename T>
__global__ void __launch_bounds__(Grad<DK>::threads, 1)
    k_delta_grads(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mo, const __grid_constant__ GradArgs a) {
    using Gr = Grad<DK>;
    constexpr int NH = Gr::NH, DW = Gr::DW, JW = Gr::JW;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t bar;
    __shared__ float row_g[NH][C], row_b[NH][C], red[32];
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rg = w & 3, cg = w >> 2;  // row group, column share
    const int g = lane >> 2, t = lane & 3;
    const int rep = a.H / a.Hk;
    const int ns = (a.dv_dim + kSlice - 1) / kSlice;
    const int L = min(C, length_of(a.lengths, b, a.N) - c * C);
    const int rows = min(C, a.N - c * C);  // rows of the tensors in this chunk
    const size_t row0 = (size_t)b * a.N + (size_t)c * C;
    T* dq = reinterpret_cast<T*>(a.dq);
    T* dk = reinterpret_cast<T*>(a.dk);
    T* dv = reinterpret_cast<T*>(a.dv);

    if (L <= 0) {  // behind the end: no gradient
        for (int i = tid; i < rows * DK; i += Gr::threads) {
            const size_t e = ((row0 + i / DK) * a.Hk + hk) * DK + i % DK;
            st_from_float(dq, e, 0.f);
            st_from_float(dk, e, 0.f);
        }
        for (int i = tid; i < rows * rep * a.dv_dim; i += Gr::threads) {
            const int r = i / (rep * a.dv_dim), x = i % (rep * a.dv_dim);
            st_from_float(dv, ((row0 + r) * a.H + hk * rep) * a.dv_dim + x, 0.f);
        }
        for (int i = tid; i < rows * rep; i += Gr::threads) {
            const size_t e = (row0 + i / rep) * a.H + hk * rep + i % rep;
            a.dg[e] = 0.f;
            a.dbeta[e] = 0.f;
        }
        return;
    }
    if (tid == 0) {
        tc::mbar_init(&bar, 1);
        tc::fence_barrier_init();
    }
    __syncthreads();
    uint32_t phase = 0;

    const uint32_t base = tc::smem_u32(sm);
    const uint32_t sO = base + Gr::oO, sY = base + Gr::oY, sU = base + Gr::oU, sS = base + Gr::oS, sD = base + Gr::oD;
    const float* gt = reinterpret_cast<const float*>(sm + Gr::oG);
    const double* G = reinterpret_cast<const double*>(sm + Gr::oG + kGates);

    float dqa[DW / 8][4], dka[DW / 8][4];  // sums over the value heads
#pragma unroll
    for (int n = 0; n < DW / 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) dqa[n][e] = dka[n][e] = 0.f;

    for (int r = 0; r < rep; r++) {
        const int h = hk * rep + r;
        const size_t ch = ((size_t)b * a.H + h) * a.nc + c;
        float E[JW / 8][4], W[JW / 8][4], Zq[DW / 8][4], Z[DW / 8][4], Zw[DW / 8][4];
#pragma unroll
        for (int n = 0; n < JW / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) E[n][e] = W[n][e] = 0.f;
#pragma unroll
        for (int n = 0; n < DW / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) Zq[n][e] = Z[n][e] = Zw[n][e] = 0.f;
        float db0 = 0.f, db1 = 0.f;  // dY . v of rows g and g + 8
        float inner = 0.f;           // <dS1, S0>

        for (int sl = 0; sl < ns; sl++) {
            __syncthreads();  // the tiles are free
            if (tid == 0) {
                tc::fence_proxy_async_smem();
                const size_t cs = ch * ns + sl;
                tc::mbar_arrive_expect_tx(&bar, Gr::O + Gr::Y + Gr::U + Gr::S + Gr::D + (sl == 0 ? kGateRow : 0));
                tc::tma_load_4d(sm + Gr::oO, &mo, &bar, sl * kSlice, h, c * C, b);
                bulk_load(sm + Gr::oY, a.kept.y + cs * Gr::Y, Gr::Y, &bar);
                bulk_load(sm + Gr::oU, a.kept.u + cs * Gr::U, Gr::U, &bar);
                bulk_load(sm + Gr::oS, a.kept.s + cs * Gr::S, Gr::S, &bar);
                bulk_load(sm + Gr::oD, a.kept.ds + cs * Gr::D, Gr::D, &bar);
                if (sl == 0) bulk_load(sm + Gr::oG, a.gates + ch * kGateRow, kGateRow, &bar);
            }
            if (!tc::mbar_wait(&bar, phase)) atomicExch(&g_grad_err, kErrTimeout);  // goes on: nothing here waits for a peer
            phase ^= 1;
            if (L < C) {
                clear_rows(sm + Gr::oO, L, kSlice / 8, lane);  // every warp for itself, the same zeros
                __syncwarp();
            }
#pragma unroll
            for (int ks = 0; ks < 4; ks++) {
                uint32_t ao[4], yh[4], yl[4], uh[4], ul[4];
                ldsm4(ao, at_k(sO, 16 * rg, 2 * ks, lane));
                ldsm4_t(yh, at_n(sY, 16 * ks, 2 * rg, lane));
                ldsm4_t(yl, at_n(sY + kTile, 16 * ks, 2 * rg, lane));
                ldsm4_t(uh, at_n(sU, 16 * ks, 2 * rg, lane));
                ldsm4_t(ul, at_n(sU + kTile, 16 * ks, 2 * rg, lane));
                // scores, up to the diagonal
#pragma unroll
                for (int p = 0; p < JW / 16; p++) {
                    const int jp = cg * (JW / 16) + p;
                    if (jp > rg) continue;
                    uint32_t bh[4], bl[4];
                    ldsm4_t(bh, at_k(sU, 16 * ks, 2 * jp, lane));
                    ldsm4_t(bl, at_k(sU + kTile, 16 * ks, 2 * jp, lane));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        mma(E[2 * p + i], ao, bh[2 * i], bh[2 * i + 1]);
                        mma(W[2 * p + i], yh, bh[2 * i], bh[2 * i + 1]);
                        mma(E[2 * p + i], ao, bl[2 * i], bl[2 * i + 1]);
                        mma(W[2 * p + i], yl, bh[2 * i], bh[2 * i + 1]);
                        mma(W[2 * p + i], yh, bl[2 * i], bl[2 * i + 1]);
                    }
                }
#pragma unroll
                for (int p = 0; p < DW / 16; p++) {
                    const int piece = cg * (DW / 8) + 2 * p;
                    uint32_t bh[4], bl[4];
                    ldsm4_t(bh, at_k(sS, 16 * ks, piece, lane));
                    ldsm4_t(bl, at_k(sS + 2 * C * DK, 16 * ks, piece, lane));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        mma(Zq[2 * p + i], ao, bh[2 * i], bh[2 * i + 1]);
                        mma(Z[2 * p + i], yh, bh[2 * i], bh[2 * i + 1]);
                        mma(Zq[2 * p + i], ao, bl[2 * i], bl[2 * i + 1]);
                        mma(Z[2 * p + i], yl, bh[2 * i], bh[2 * i + 1]);
                        mma(Z[2 * p + i], yh, bl[2 * i], bl[2 * i + 1]);
                    }
                    ldsm4_t(bh, at_k(sD, 16 * ks, piece, lane));
                    ldsm4_t(bl, at_k(sD + 2 * C * DK, 16 * ks, piece, lane));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        mma(Zw[2 * p + i], uh, bh[2 * i], bh[2 * i + 1]);
                        mma(Zw[2 * p + i], ul, bh[2 * i], bh[2 * i + 1]);
                        mma(Zw[2 * p + i], uh, bl[2 * i], bl[2 * i + 1]);
                    }
                }
                // dv and dY . v from the A operand: rows g, g + 8; columns 2t, 2t + 1 and eight on
                if (ks % NH == cg) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int row = 16 * rg + g + 8 * (e & 1), col = sl * kSlice + 16 * ks + 2 * t + 8 * (e >> 1);
                        if (row < rows && col < a.dv_dim) {
                            const float y0 = tc::bf16lo(yh[e]) + tc::bf16lo(yl[e]), y1 = tc::bf16hi(yh[e]) + tc::bf16hi(yl[e]);
                            const size_t at = ((row0 + row) * a.H + h) * a.dv_dim + col;
                            const float bt = gt[2 * C + row];
                            st_pair(dv + at, bt * y0, bt * y1);
                            if (row < L) {
                                const uint32_t v2 = *reinterpret_cast<const uint32_t*>(a.v + at);
                                const float d = fmaf(y0, tc::bf16lo(v2), y1 * tc::bf16hi(v2));
                                if (e & 1) db1 += d;
                                else db0 += d;
                            }
                        }
                    }
                }
            }
            // <dS1, S0> of the slice
            for (int i = tid; i < C * DK / 8; i += Gr::threads) {
                uint4 q[4];
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    q[j] = *reinterpret_cast<const uint4*>(sm + Gr::oS + j * 2 * C * DK + 16 * i);
                    q[2 + j] = *reinterpret_cast<const uint4*>(sm + Gr::oD + j * 2 * C * DK + 16 * i);
                }
                const uint32_t* x = reinterpret_cast<const uint32_t*>(q);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    inner = fmaf(tc::bf16lo(x[j]) + tc::bf16lo(x[4 + j]), tc::bf16lo(x[8 + j]) + tc::bf16lo(x[12 + j]), inner);
                    inner = fmaf(tc::bf16hi(x[j]) + tc::bf16hi(x[4 + j]), tc::bf16hi(x[8 + j]) + tc::bf16hi(x[12 + j]), inner);
                }
            }
        }

        // K and Q take S0's place, the scores that of dY and U
        __syncthreads();
        if (tid == 0) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive_expect_tx(&bar, 4 * C * DK);
#pragma unroll
            for (int i = 0; i < DK / 64; i++) {
                tc::tma_load_4d(sm + Gr::oS + i * 8192, &mk, &bar, 64 * i, hk, c * C, b);
                tc::tma_load_4d(sm + Gr::oS + 2 * C * DK + i * 8192, &mq, &bar, 64 * i, hk, c * C, b);
            }
        }
#pragma unroll
        for (int n = 0; n < JW / 8; n++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const int i = 16 * rg + g + 8 * half, j = cg * JW + 8 * n + 2 * t;
                float ev[2], wv[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const bool in = i >= j + e && i < L;
                    const float D = in ? expf((float)(G[i] - G[j + e])) : 0.f;
                    ev[e] = in ? E[n][2 * half + e] * D : 0.f;
                    wv[e] = in && i > j + e ? W[n][2 * half + e] * D : 0.f;
                }
                uint32_t hi, lo;
                const uint32_t off = tile_at(0, i, j >> 3) + 4 * t;
                split2(ev[0], ev[1], hi, lo);
                *reinterpret_cast<uint32_t*>(sm + Gr::oY + off) = hi;
                *reinterpret_cast<uint32_t*>(sm + Gr::oY + kTile + off) = lo;
                split2(wv[0], wv[1], hi, lo);
                *reinterpret_cast<uint32_t*>(sm + Gr::oU + off) = hi;
                *reinterpret_cast<uint32_t*>(sm + Gr::oU + kTile + off) = lo;
            }
        if (!tc::mbar_wait(&bar, phase)) atomicExch(&g_grad_err, kErrTimeout);
        phase ^= 1;
        const uint32_t sK = sS, sQ = sS + 2 * C * DK;
        if (L < C) {
            clear_rows(sm + Gr::oS, L, DK / 8, lane);
            clear_rows(sm + Gr::oS + 2 * C * DK, L, DK / 8, lane);
        }
        __syncthreads();

        const int i0 = 16 * rg + g, i1 = i0 + 8;
        const float eg0 = gt[i0], eg1 = gt[i1], ec0 = gt[C + i0], ec1 = gt[C + i1], bt0 = gt[2 * C + i0], bt1 = gt[2 * C + i1];
        float end = 0.f;  // sum of k . (exp(G_C - G) U dS1^T)
        auto pair_at = [&](uint32_t off, int row, int n) {
            return *reinterpret_cast<const uint32_t*>(sm + Gr::oS + off + tile_at(0, row, cg * (DW / 8) + n) + 4 * t);
        };
        float dg0 = 0.f, dg1 = 0.f;
#pragma unroll
        for (int n = 0; n < DW / 8; n++) {
            const uint32_t k0 = pair_at(0, i0, n), k1 = pair_at(0, i1, n);
            Zq[n][0] *= eg0; Zq[n][1] *= eg0; Zq[n][2] *= eg1; Zq[n][3] *= eg1;
            Z[n][0] *= eg0; Z[n][1] *= eg0; Z[n][2] *= eg1; Z[n][3] *= eg1;
            Zw[n][0] *= ec0; Zw[n][1] *= ec0; Zw[n][2] *= ec1; Zw[n][3] *= ec1;
            end += tc::bf16lo(k0) * Zw[n][0] + tc::bf16hi(k0) * Zw[n][1] + tc::bf16lo(k1) * Zw[n][2] + tc::bf16hi(k1) * Zw[n][3];
        }
#pragma unroll
        for (int ks = 0; ks < 4; ks++) {
            if (ks <= rg) {  // rows i take j <= i
                uint32_t eh[4], el[4], wh[4], wl[4];
                ldsm4(eh, at_k(sY, 16 * rg, 2 * ks, lane));
                ldsm4(el, at_k(sY + kTile, 16 * rg, 2 * ks, lane));
                ldsm4(wh, at_k(sU, 16 * rg, 2 * ks, lane));
                ldsm4(wl, at_k(sU + kTile, 16 * rg, 2 * ks, lane));
#pragma unroll
                for (int p = 0; p < DW / 16; p++) {
                    uint32_t bk[4];
                    ldsm4_t(bk, at_k(sK, 16 * ks, cg * (DW / 8) + 2 * p, lane));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        mma(Zq[2 * p + i], eh, bk[2 * i], bk[2 * i + 1]);
                        mma(Z[2 * p + i], wh, bk[2 * i], bk[2 * i + 1]);
                        mma(Zq[2 * p + i], el, bk[2 * i], bk[2 * i + 1]);
                        mma(Z[2 * p + i], wl, bk[2 * i], bk[2 * i + 1]);
                    }
                }
            }
            if (ks >= rg) {  // rows j take i >= j
                uint32_t eh[4], el[4], wh[4], wl[4];
                ldsm4_t(eh, at_n(sY, 16 * ks, 2 * rg, lane));
                ldsm4_t(el, at_n(sY + kTile, 16 * ks, 2 * rg, lane));
                ldsm4_t(wh, at_n(sU, 16 * ks, 2 * rg, lane));
                ldsm4_t(wl, at_n(sU + kTile, 16 * ks, 2 * rg, lane));
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float2 bt = *reinterpret_cast<const float2*>(gt + 2 * C + 16 * ks + 2 * t + 8 * (e >> 1));
                    split2(-bt.x * (tc::bf16lo(wh[e]) + tc::bf16lo(wl[e])), -bt.y * (tc::bf16hi(wh[e]) + tc::bf16hi(wl[e])),
                           wh[e], wl[e]);
                }
#pragma unroll
                for (int p = 0; p < DW / 16; p++) {
                    uint32_t bq[4], bk[4];
                    ldsm4_t(bq, at_k(sQ, 16 * ks, cg * (DW / 8) + 2 * p, lane));
                    ldsm4_t(bk, at_k(sK, 16 * ks, cg * (DW / 8) + 2 * p, lane));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        mma(Zw[2 * p + i], eh, bq[2 * i], bq[2 * i + 1]);
                        mma(Zw[2 * p + i], el, bq[2 * i], bq[2 * i + 1]);
                        mma(Zw[2 * p + i], wh, bk[2 * i], bk[2 * i + 1]);
                        mma(Zw[2 * p + i], wl, bk[2 * i], bk[2 * i + 1]);
                    }
                }
            }
        }
        // now Zq = dq, -Z = r, Zw = w
#pragma unroll
        for (int n = 0; n < DW / 8; n++) {
            const uint32_t k0 = pair_at(0, i0, n), k1 = pair_at(0, i1, n);
            const uint32_t q0 = pair_at(2 * C * DK, i0, n), q1 = pair_at(2 * C * DK, i1, n);
            const float kr0 = -(tc::bf16lo(k0) * Z[n][0] + tc::bf16hi(k0) * Z[n][1]);
            const float kr1 = -(tc::bf16lo(k1) * Z[n][2] + tc::bf16hi(k1) * Z[n][3]);
            db0 += kr0;
            db1 += kr1;
            dg0 += tc::bf16lo(q0) * Zq[n][0] + tc::bf16hi(q0) * Zq[n][1] + bt0 * kr0 -
                   (tc::bf16lo(k0) * Zw[n][0] + tc::bf16hi(k0) * Zw[n][1]);
            dg1 += tc::bf16lo(q1) * Zq[n][2] + tc::bf16hi(q1) * Zq[n][3] + bt1 * kr1 -
                   (tc::bf16lo(k1) * Zw[n][2] + tc::bf16hi(k1) * Zw[n][3]);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                dqa[n][e] += Zq[n][e];
                dka[n][e] += Zw[n][e] - (e < 2 ? bt0 : bt1) * Z[n][e];
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            dg0 += __shfl_xor_sync(0xffffffffu, dg0, o);
            dg1 += __shfl_xor_sync(0xffffffffu, dg1, o);
            db0 += __shfl_xor_sync(0xffffffffu, db0, o);
            db1 += __shfl_xor_sync(0xffffffffu, db1, o);
        }
        if (t == 0) {
            row_g[cg][i0] = dg0;
            row_g[cg][i1] = dg1;
            row_b[cg][i0] = db0;
            row_b[cg][i1] = db1;
        }
        end = fmaf(gt[C - 1], inner, end);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) end += __shfl_xor_sync(0xffffffffu, end, o);
        if (lane == 0) red[w] = end;
        __syncthreads();
        if (w == 0) {
            // dg: sums from a row to the last one, in 64 bits (they cancel)
            double e = 0.0;
            for (int i = 0; i < 4 * NH; i++) e += red[i];
            double x[2];
            float y[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int row = C - 1 - (2 * lane + i);  // backwards
                x[i] = 0.0;
                y[i] = 0.f;
#pragma unroll
                for (int j = 0; j < NH; j++) {
                    x[i] += row_g[j][row];
                    y[i] += row_b[j][row];
                }
            }
            double s = x[0] + x[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            s += e;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int row = C - 1 - (2 * lane + i);
                if (row < rows) {
                    const size_t at = (row0 + row) * a.H + h;
                    a.dg[at] = row < L ? (float)(i ? s : s - x[1]) : 0.f;
                    a.dbeta[at] = row < L ? y[i] : 0.f;
                }
            }
        }
    }

#pragma unroll
    for (int n = 0; n < DW / 8; n++)
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int row = 16 * rg + g + 8 * half;
            if (row < rows) {
                const size_t at = ((row0 + row) * a.Hk + hk) * DK + cg * DW + 8 * n + 2 * t;
                st_pair(dq + at, dqa[n][2 * half], dqa[n][2 * half + 1]);
                st_pair(dk + at, dka[n][2 * half], dka[n][2 * half + 1]);
            }
        }
}

template <int DK, typename T>
ret_status grads(const DeltaArgs& a, const GradArgs& g, cudaStream_t s) {
    CUtensorMap mq, mk, mo;
    if (!chunk_map(&mq, a.q, a.B, a.N, a.Hk, DK) || !chunk_map(&mk, a.k, a.B, a.N, a.Hk, DK) ||
        !chunk_map(&mo, a.dout, a.B, a.N, a.H, a.dv))
        return RET_ERR_CUDA;
    cudaError_t e = cudaFuncSetAttribute(k_delta_grads<DK, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Grad<DK>::smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule gradients: %s", cudaGetErrorString(e));
    k_delta_grads<DK, T><<<dim3(g.nc, a.Hk, a.B), Grad<DK>::threads, Grad<DK>::smem, s>>>(mq, mk, mo, g);
    return check_launch("delta rule: gradients");
}

template <typename T>
ret_status grads_dk(const DeltaArgs& a, const GradArgs& g, cudaStream_t s) {
    return a.dk == 64 ? grads<64, T>(a, g, s) : a.dk == 128 ? grads<128, T>(a, g, s) : grads<256, T>(a, g, s);
}

}  // namespace
}  // namespace delta

using namespace delta;

// The workspace's parts, per (sequence, head, chunk): tables and gates; per
// slice of 64 value columns the kept states, their gradients, U and dY.
size_t delta_backward_ws_bytes(const DeltaArgs& a) {
    const size_t n = (size_t)a.B * a.H * chunks_of(a.N);
    return n * (4 * kTile + kGateRow) + n * slices_of(a.dv) * (size_t)(8 * C * a.dk + 4 * kTile);
}

ret_status launch_delta_backward(const DeltaArgs& a, void* ws, cudaStream_t s) {
    const size_t n = (size_t)a.B * a.H * chunks_of(a.N), m = n * slices_of(a.dv);
    uint8_t* tiles = reinterpret_cast<uint8_t*>(ws);
    Kept kept;
    kept.s = tiles + n * 4 * kTile;
    kept.ds = kept.s + m * 4 * C * a.dk;
    kept.u = kept.ds + m * 4 * C * a.dk;
    kept.y = kept.u + m * 2 * kTile;
    uint8_t* gates = kept.y + m * 2 * kTile;
    ret_status st = launch_prep(a, tiles, gates, s);
    if (st != RET_OK) return st;
    if ((st = launch_chains(a, tiles, gates, kept, s)) != RET_OK) return st;
    GradArgs g{};
    g.gates = gates;
    g.lengths = a.lengths;
    g.v = (const __nv_bfloat16*)a.v;
    g.kept = kept;
    g.dq = a.dq; g.dk = a.dkk; g.dv = a.dvv;
    g.dg = a.dg; g.dbeta = a.dbeta;
    g.N = a.N; g.nc = chunks_of(a.N); g.Hk = a.Hk; g.H = a.H; g.dv_dim = a.dv;
    return a.grad_dt == RET_F32 ? grads_dk<float>(a, g, s) : grads_dk<__nv_bfloat16>(a, g, s);
}

}  // namespace ret
