// k_delta_backward.cu -- gradients of the gated delta rule's chunked forward
// (notation and number format: delta_util.cuh).  Three launches: the chunk
// tables, the two chains of k_delta_chunk.cu side by side (states before each
// chunk, corrections U'; gradients of the states after each chunk, Y), and this
// pass, chunk by chunk in parallel.  All in the scaled keys and queries, primes
// left out; with W = Y U^T, E = dO U^T, row i of a chunk:
//     dq_i = exp(G_i) dO_i S0^T + sum_{j<=i} E_ij D_ij k_j
//     r_i  = -(exp(G_i) Y_i S0^T + sum_{j<i} W_ij D_ij k_j)
//     z_j  = exp(G_C - G_j) U_j dS1^T
//     w_j  = sum_{i>=j} E_ij D_ij q_i - sum_{i>j} beta_i W_ij D_ij k_i
//     dk   = beta r + w + z,  dv = beta Y,  dbeta_i = Y_i . v_i + k_i . r_i.
// A row's decay multiplies what it reads and divides what it writes, and the
// last row's also scales the state:
//     dg_i = sum_{j>=i} (q_j . dq_j + beta_j k_j . r_j - k_j . w_j)
//            + sum_{j<i} k_j . z_j + exp(G_C) <dS1, S0>
// (the sums over z cancel up to the rows before i).  Then
// dq' = dq / s_q and so on undo the scaling.
//
// A key head's gradient is the sum over its value heads: one block takes them
// all, one after the other, so the order is fixed.  Sixteen warps: a row group
// of 16 tokens and a quarter of dk each.  The records of 16 value columns come
// through a ring of bulk copies that runs on across value heads,
// and the five products over dv accumulate in registers; then the 64 x 64
// scores go through shared memory once, in two terms, to meet K and Q.
//
// %FIG%
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
    Tables tb;
    const int* lengths;
    const __nv_bfloat16* v;
    const uint8_t* records;
    void *dq, *dk, *dv;
    float *dg, *dbeta;
    int N, nc, Hk, H, dv_dim;
};

template <int DK>
struct Grad {
    static constexpr int NH = 4, warps = 4 * NH;       // column shares
    static constexpr int threads = warps * 32;
    static constexpr int DW = DK / NH;                 // dk columns of a warp
    static constexpr int oK = 0, oQ = 2 * C * DK;      // K, Q
    static constexpr int oE = 4 * C * DK;              // E D, W D, beta W D: hi, lo each
    static constexpr int oR = oE + 6 * kTile;          // the ring
    static constexpr int most = 222 * 1024;
    static constexpr int fit = (most - oR - 2 * 2048) / Record<DK>::bytes;
    static constexpr int stages = fit > 6 ? 6 : fit;
    static constexpr int oG = oR + stages * Record<DK>::bytes;  // the gates of this value head and the next one
    static constexpr int smem = oG + 2 * 2048 + 1024;
};

template <typename T>
__device__ __forceinline__ void st_pair(T* p, float x, float y) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(p) = make_float2(x, y);
    else *reinterpret_cast<uint32_t*>(p) = tc::pack_bf16x2(x, y);
}
__device__ __forceinline__ float2 sum_h2(uint32_t hi, uint32_t lo) {
    const float2 h = unpack_h2(hi), l = unpack_h2(lo);
    return make_float2(h.x + l.x, h.y + l.y);
}

template <int DK, typename T>
__global__ void __launch_bounds__(Grad<DK>::threads, 1) k_delta_grads(const __grid_constant__ GradArgs a) {
    using Gr = Grad<DK>;
    using Rec = Record<DK>;
    constexpr int NH = Gr::NH, DW = Gr::DW, NS = Gr::stages;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[NS], empty[NS], keys, gfull[2], gempty[2];
    __shared__ float inv_e[4][4], inv_w[4][4], inv_b[4][4];
    __shared__ float row_a[NH][C], row_c[NH][C], row_b[NH][C], red[Gr::warps];
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rep = a.H / a.Hk, ng = groups_of(a.dv_dim);
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
        for (int i = 0; i < NS; i++) tc::mbar_init(full + i, 1), tc::mbar_init(empty + i, Gr::warps);
        for (int i = 0; i < 2; i++) tc::mbar_init(gfull + i, 1), tc::mbar_init(gempty + i, Gr::warps);
        tc::mbar_init(&keys, 1);
        tc::fence_barrier_init();
    }
    __syncthreads();
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {  // after one gave up the others are skipped: the barriers stay complete
        if (ok && !tc::mbar_wait(bar, phase & 1)) {
            ok = false;
            atomicExch(&g_grad_err, kErrTimeout);
        }
    };

    // one lane: records and gates into the ring, ahead of the warps
    const size_t ch0 = ((size_t)b * a.H + hk * rep) * a.nc + c;
    const int steps = rep * ng;
    auto load = [&](int s) {
        if (s >= NS) wait(empty + s % NS, s / NS - 1);
        if (!ok) return;
        const int r = s / ng;
        tc::mbar_arrive_expect_tx(full + s % NS, Rec::bytes);
        bulk_load(sm + Gr::oR + (s % NS) * Rec::bytes, a.records + ((ch0 + (size_t)r * a.nc) * ng + s % ng) * Rec::bytes,
                  Rec::bytes, full + s % NS);
    };
    auto load_gates = [&](int r) {
        if (r >= 2) wait(gempty + (r & 1), (r >> 1) - 1);
        if (!ok) return;
        tc::mbar_arrive_expect_tx(gfull + (r & 1), kGateRow);
        bulk_load(sm + Gr::oG + (r & 1) * 2048, a.tb.gates + (ch0 + (size_t)r * a.nc) * kGateRow, kGateRow, gfull + (r & 1));
    };
    if (tid == 0) {
        load_gates(0);
        for (int s = 0; s < NS - 1 && s < steps; s++) load(s);
        tc::mbar_arrive_expect_tx(&keys, 4 * C * DK);
        bulk_load(sm, a.tb.keys + (((size_t)b * a.Hk + hk) * a.nc + c) * (4 * C * DK), 4 * C * DK, &keys);
    }
    __syncwarp();

    const int rg = w & 3, cg = w >> 2;  // row group, column share
    const int g = lane >> 2, t = lane & 3;
    const uint32_t base = tc::smem_u32(sm), sK = base + Gr::oK, sQ = base + Gr::oQ, sE = base + Gr::oE;
    const int i0 = 16 * rg + g, i1 = i0 + 8;

    float dqa[DW / 8][4], dka[DW / 8][4];  // sums over the value heads
#pragma unroll
    for (int n = 0; n < DW / 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) dqa[n][e] = dka[n][e] = 0.f;

    for (int r = 0, it = 0; r < rep; r++) {
        const int h = hk * rep + r;
        const float* gt = reinterpret_cast<const float*>(sm + Gr::oG + (r & 1) * 2048);
        const double* G = reinterpret_cast<const double*>(sm + Gr::oG + (r & 1) * 2048 + kGates);
        if (tid == 0 && r + 1 < rep) load_gates(r + 1);
        __syncwarp();
        wait(gfull + (r & 1), r >> 1);
        float E[2][4], W[2][4], Zq[DW / 8][4], Z[DW / 8][4], Zw[DW / 8][4];
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) E[n][e] = W[n][e] = 0.f;
#pragma unroll
        for (int n = 0; n < DW / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) Zq[n][e] = Z[n][e] = Zw[n][e] = 0.f;
        float db0 = 0.f, db1 = 0.f;  // Y . v of rows g and g + 8
        float inner = 0.f;           // <dS1, S0>
        const float b0 = gt[gBeta + i0], b1 = gt[gBeta + i1], k0 = gt[gIk + i0], k1 = gt[gIk + i1];

        for (int gr = 0; gr < ng; gr++, it++) {
            const int st = it % NS;
            if (tid == 0 && it + NS - 1 < steps) load(it + NS - 1);
            __syncwarp();
            const uint8_t* rec = sm + Gr::oR + st * Rec::bytes;
            const uint32_t sr = tc::smem_u32(rec);
            const float* f = reinterpret_cast<const float*>(rec + Rec::f);
            // dv and Y . v: of the rows' 16 columns a share takes every fourth group
            const bool mine = (gr & 3) == cg;
            uint32_t v2[4] = {0, 0, 0, 0};
            if (mine) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int row = 16 * rg + g + 8 * (e & 1), col = 16 * gr + 2 * t + 8 * (e >> 1);
                    if (row < L && col < a.dv_dim)
                        v2[e] = *reinterpret_cast<const uint32_t*>(a.v + ((row0 + row) * a.H + h) * a.dv_dim + col);
                }
            }
            wait(full + st, it / NS);
            uint32_t ao[4], yh[4], yl[4], uh[4], ul[4];
            ldsm4_t(ao, at_n<16>(sr + Rec::o, 0, 2 * rg, lane));
            ldsm4_t(yh, at_n<16>(sr + Rec::y, 0, 2 * rg, lane));
            ldsm4_t(yl, at_n<16>(sr + Rec::y + 2048, 0, 2 * rg, lane));
            ldsm4_t(uh, at_n<16>(sr + Rec::u, 0, 2 * rg, lane));
            ldsm4_t(ul, at_n<16>(sr + Rec::u + 2048, 0, 2 * rg, lane));
            const float io = f[fO], iy = f[fY], iu = f[fU];
            if (cg <= rg) {  // scores, up to the diagonal
                uint32_t bh[4], bl[4];
                ldsm4_t(bh, at_k<16>(sr + Rec::u, 0, 2 * cg, lane));
                ldsm4_t(bl, at_k<16>(sr + Rec::u + 2048, 0, 2 * cg, lane));
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float x[4], y[4];
                    mma0(x, ao, bh[2 * i], bh[2 * i + 1]);
                    mma0(y, yh, bh[2 * i], bh[2 * i + 1]);
                    mma(x, ao, bl[2 * i], bl[2 * i + 1]);
                    mma(y, yl, bh[2 * i], bh[2 * i + 1]);
                    mma(y, yh, bl[2 * i], bl[2 * i + 1]);
                    add_scaled(E[i], x, io * iu);
                    add_scaled(W[i], y, iy * iu);
                }
            }
            const float is = f[fS + cg / 2], id = f[fDs + cg / 2];
#pragma unroll
            for (int p = 0; p < DW / 16; p++) {
                uint32_t bh[4], bl[4], dh[4], dl[4];
                const uint32_t off = at_k<16>(0, 0, cg * (DW / 8) + 2 * p, lane);
                ldsm4_t(bh, sr + Rec::s + off);
                ldsm4_t(bl, sr + Rec::s + 32 * DK + off);
                ldsm4_t(dh, sr + Rec::ds + off);
                ldsm4_t(dl, sr + Rec::ds + 32 * DK + off);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float x[4], y[4], z[4];
                    mma0(x, ao, bh[2 * i], bh[2 * i + 1]);
                    mma0(y, yh, bh[2 * i], bh[2 * i + 1]);
                    mma0(z, uh, dh[2 * i], dh[2 * i + 1]);
                    mma(x, ao, bl[2 * i], bl[2 * i + 1]);
                    mma(y, yl, bh[2 * i], bh[2 * i + 1]);
                    mma(z, ul, dh[2 * i], dh[2 * i + 1]);
                    mma(y, yh, bl[2 * i], bl[2 * i + 1]);
                    mma(z, uh, dl[2 * i], dl[2 * i + 1]);
                    add_scaled(Zq[2 * p + i], x, io * is);
                    add_scaled(Z[2 * p + i], y, iy * is);
                    add_scaled(Zw[2 * p + i], z, iu * id);
                }
            }
            // <dS1, S0> of the share's columns, four of the 16 rows each
            {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < DW / 16; i++) {
                    const int q = i * 32 + lane;  // of the DW / 2 pairs of four rows
                    const uint32_t off = tile_at<16>(4 * rg + q / (DW / 2), (cg * DW + 2 * (q % (DW / 2))) / 8) + 4 * (q & 3);
                    const uint8_t *ps = rec + Rec::s + off, *pd = rec + Rec::ds + off;
                    const float2 s2 = sum_h2(*reinterpret_cast<const uint32_t*>(ps), *reinterpret_cast<const uint32_t*>(ps + 32 * DK));
                    const float2 d2 = sum_h2(*reinterpret_cast<const uint32_t*>(pd), *reinterpret_cast<const uint32_t*>(pd + 32 * DK));
                    x = fmaf(s2.x, d2.x, x);
                    x = fmaf(s2.y, d2.y, x);
                }
                inner = fmaf(x, is * id, inner);
            }
            if (mine) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int row = 16 * rg + g + 8 * (e & 1), col = 16 * gr + 2 * t + 8 * (e >> 1);
                    float2 y = sum_h2(yh[e], yl[e]);
                    y.x *= iy;
                    y.y *= iy;
                    const float s = (e & 1 ? b1 * k1 : b0 * k0);  // dv = beta' Y / s_k
                    if (row < rows && col < a.dv_dim)
                        st_pair(dv + ((row0 + row) * a.H + h) * a.dv_dim + col, s * y.x, s * y.y);
                    const float d = fmaf(y.x, tc::bf16lo(v2[e]), y.y * tc::bf16hi(v2[e]));
                    if (e & 1) db1 = fmaf(d, k1, db1);
                    else db0 = fmaf(d, k0, db0);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty + st);
        }

        // the scores, with the decays, in two terms
        if (cg <= rg) {
            float bw[2][4];
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int i = e < 2 ? i0 : i1, j = 16 * cg + 8 * n + 2 * t + (e & 1);
                    const bool in = i >= j && i < L;
                    const float D = in ? expf((float)(G[i] - G[j])) : 0.f;
                    E[n][e] = in ? E[n][e] * D : 0.f;
                    W[n][e] = in && i > j ? W[n][e] * D : 0.f;
                    bw[n][e] = W[n][e] * (e < 2 ? b0 : b1);
                }
            auto put = [&](float (&x)[2][4], int tile, float* inv) {
                float v;
                const float s = scale_of(x[0], x[1], v);
                uint32_t hi[4], lo[4];
                split_a(x[0], x[1], s, hi, lo);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const uint32_t off = Gr::oE + tile * 2 * kTile + tile_at(16 * rg + g + 8 * (e & 1), 2 * cg + (e >> 1)) + 4 * t;
                    *reinterpret_cast<uint32_t*>(sm + off) = hi[e];
                    *reinterpret_cast<uint32_t*>(sm + off + kTile) = lo[e];
                }
                if (lane == 0) *inv = v;
            };
            put(E, 0, &inv_e[rg][cg]);
            put(W, 1, &inv_w[rg][cg]);
            put(bw, 2, &inv_b[rg][cg]);
        }
        if (r == 0) wait(&keys, 0);
        tc::barrier(1, Gr::threads);

        const float eg0 = gt[gEG + i0], eg1 = gt[gEG + i1], ec0 = gt[gEC + i0], ec1 = gt[gEC + i1];
        auto pair_at = [&](int off, int row, int n) {
            return unpack_h2(*reinterpret_cast<const uint32_t*>(sm + off + tile_at(row, cg * (DW / 8) + n) + 4 * t));
        };
        float ca0 = 0.f, ca1 = 0.f, cc0 = 0.f, cc1 = 0.f;  // row sums of dg
#pragma unroll
        for (int n = 0; n < DW / 8; n++) {
            const float2 x0 = pair_at(Gr::oK, i0, n), x1 = pair_at(Gr::oK, i1, n);
            Zq[n][0] *= eg0; Zq[n][1] *= eg0; Zq[n][2] *= eg1; Zq[n][3] *= eg1;
            Z[n][0] *= eg0; Z[n][1] *= eg0; Z[n][2] *= eg1; Z[n][3] *= eg1;
            Zw[n][0] *= ec0; Zw[n][1] *= ec0; Zw[n][2] *= ec1; Zw[n][3] *= ec1;
            cc0 = fmaf(x0.x, Zw[n][0], fmaf(x0.y, Zw[n][1], cc0));
            cc1 = fmaf(x1.x, Zw[n][2], fmaf(x1.y, Zw[n][3], cc1));
            // z into the sum over the value heads; Zw goes on with w
#pragma unroll
            for (int e = 0; e < 4; e++) {
                dka[n][e] += Zw[n][e];
                Zw[n][e] = 0.f;
            }
        }
#pragma unroll
        for (int ks = 0; ks < 4; ks++) {
            if (ks <= rg) {  // rows i take j <= i
                uint32_t eh[4], el[4], wh[4], wl[4];
                ldsm4(eh, at_k(sE, 16 * rg, 2 * ks, lane));
                ldsm4(el, at_k(sE + kTile, 16 * rg, 2 * ks, lane));
                ldsm4(wh, at_k(sE + 2 * kTile, 16 * rg, 2 * ks, lane));
                ldsm4(wl, at_k(sE + 3 * kTile, 16 * rg, 2 * ks, lane));
                const float ie = inv_e[rg][ks], iw = inv_w[rg][ks];
#pragma unroll
                for (int p = 0; p < DW / 16; p++) {
                    uint32_t bk[4];
                    ldsm4_t(bk, at_k(sK, 16 * ks, cg * (DW / 8) + 2 * p, lane));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float x[4], y[4];
                        mma0(x, eh, bk[2 * i], bk[2 * i + 1]);
                        mma0(y, wh, bk[2 * i], bk[2 * i + 1]);
                        mma(x, el, bk[2 * i], bk[2 * i + 1]);
                        mma(y, wl, bk[2 * i], bk[2 * i + 1]);
                        add_scaled(Zq[2 * p + i], x, ie);
                        add_scaled(Z[2 * p + i], y, iw);
                    }
                }
            }
            if (ks >= rg) {  // rows j take i >= j
                uint32_t eh[4], el[4], wh[4], wl[4];
                ldsm4_t(eh, at_n(sE, 16 * ks, 2 * rg, lane));
                ldsm4_t(el, at_n(sE + kTile, 16 * ks, 2 * rg, lane));
                ldsm4_t(wh, at_n(sE + 4 * kTile, 16 * ks, 2 * rg, lane));
                ldsm4_t(wl, at_n(sE + 5 * kTile, 16 * ks, 2 * rg, lane));
                const float ie = inv_e[ks][rg], ib = -inv_b[ks][rg];
#pragma unroll
                for (int p = 0; p < DW / 16; p++) {
                    uint32_t bq[4], bk[4];
                    ldsm4_t(bq, at_k(sQ, 16 * ks, cg * (DW / 8) + 2 * p, lane));
                    ldsm4_t(bk, at_k(sK, 16 * ks, cg * (DW / 8) + 2 * p, lane));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float x[4], y[4];
                        mma0(x, eh, bq[2 * i], bq[2 * i + 1]);
                        mma0(y, wh, bk[2 * i], bk[2 * i + 1]);
                        mma(x, el, bq[2 * i], bq[2 * i + 1]);
                        mma(y, wl, bk[2 * i], bk[2 * i + 1]);
                        add_scaled(Zw[2 * p + i], x, ie);
                        add_scaled(Zw[2 * p + i], y, ib);
                    }
                }
            }
        }
        // now Zq = dq, -Z = r, Zw = w
#pragma unroll
        for (int n = 0; n < DW / 8; n++) {
            const float2 x0 = pair_at(Gr::oK, i0, n), x1 = pair_at(Gr::oK, i1, n);
            const float2 q0 = pair_at(Gr::oQ, i0, n), q1 = pair_at(Gr::oQ, i1, n);
            const float kr0 = -(x0.x * Z[n][0] + x0.y * Z[n][1]), kr1 = -(x1.x * Z[n][2] + x1.y * Z[n][3]);
            db0 += kr0;
            db1 += kr1;
            ca0 += q0.x * Zq[n][0] + q0.y * Zq[n][1] + b0 * kr0 - (x0.x * Zw[n][0] + x0.y * Zw[n][1]);
            ca1 += q1.x * Zq[n][2] + q1.y * Zq[n][3] + b1 * kr1 - (x1.x * Zw[n][2] + x1.y * Zw[n][3]);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                dqa[n][e] += Zq[n][e];
                dka[n][e] += Zw[n][e] - (e < 2 ? b0 : b1) * Z[n][e];
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            ca0 += __shfl_xor_sync(0xffffffffu, ca0, o);
            ca1 += __shfl_xor_sync(0xffffffffu, ca1, o);
            cc0 += __shfl_xor_sync(0xffffffffu, cc0, o);
            cc1 += __shfl_xor_sync(0xffffffffu, cc1, o);
            db0 += __shfl_xor_sync(0xffffffffu, db0, o);
            db1 += __shfl_xor_sync(0xffffffffu, db1, o);
        }
        if (t == 0) {
            row_a[cg][i0] = ca0;
            row_a[cg][i1] = ca1;
            row_c[cg][i0] = cc0;
            row_c[cg][i1] = cc1;
            row_b[cg][i0] = db0;
            row_b[cg][i1] = db1;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
        if (lane == 0) red[w] = inner;
        tc::barrier(1, Gr::threads);
        if (w == 0) {
            // in 64 bits (the sums cancel): a from a row to the last one, c of the rows before
            double e = 0.0;
            for (int i = 0; i < Gr::warps; i++) e += red[i];
            e *= gt[gEG + C - 1];
            double x[2], z[2];
            float y[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int row = C - 1 - (2 * lane + i);  // backwards
                x[i] = z[i] = 0.0;
                y[i] = 0.f;
#pragma unroll
                for (int j = 0; j < NH; j++) {
                    x[i] += row_a[j][row];
                    z[i] += row_c[j][row];
                    y[i] += row_b[j][row];
                }
            }
            // sum_{j>=i} a_j + sum_{j<i} c_j = (sum of all c) + sum_{j>=i} (a_j - c_j),
            // kept apart: c's sum over the rows before i is its own scan
            double s = x[0] + x[1], before = z[0] + z[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, s, o), d = __shfl_down_sync(0xffffffffu, before, o);
                if (lane >= o) s += u;
                if (lane + o < 32) before += d;
            }
            // before: c of this lane's two rows and all earlier ones
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int row = C - 1 - (2 * lane + i);
                if (row < rows) {
                    const size_t at = (row0 + row) * a.H + h;
                    const double d = (i ? s : s - x[1]) + (i ? before - z[0] - z[1] : before - z[0]) + e;
                    const float sk = 1.f / gt[gIk + row];
                    a.dg[at] = row < L ? (float)d : 0.f;
                    a.dbeta[at] = row < L ? y[i] * sk * sk : 0.f;
                }
            }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(gempty + (r & 1));
    }

    // undo the scaling: any value head's gates hold the keys' and queries' scales
    const float* gt = reinterpret_cast<const float*>(sm + Gr::oG + ((rep - 1) & 1) * 2048);
#pragma unroll
    for (int half = 0; half < 2; half++) {
        const int row = half ? i1 : i0;
        if (row >= rows) continue;
        const float ik = gt[gIk + row], iq = 1.f / gt[gSq + row];
#pragma unroll
        for (int n = 0; n < DW / 8; n++) {
            const size_t at = ((row0 + row) * a.Hk + hk) * DK + cg * DW + 8 * n + 2 * t;
            st_pair(dq + at, dqa[n][2 * half] * iq, dqa[n][2 * half + 1] * iq);
            st_pair(dk + at, dka[n][2 * half] * ik, dka[n][2 * half + 1] * ik);
        }
    }
}

template <int DK, typename T>
ret_status grads(const DeltaArgs& a, const GradArgs& g, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_delta_grads<DK, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Grad<DK>::smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule gradients: %s", cudaGetErrorString(e));
    k_delta_grads<DK, T><<<dim3(g.nc, a.Hk, a.B), Grad<DK>::threads, Grad<DK>::smem, s>>>(g);
    return check_launch("delta rule: gradients");
}

template <typename T>
ret_status grads_dk(const DeltaArgs& a, const GradArgs& g, cudaStream_t s) {
    return a.dk == 64 ? grads<64, T>(a, g, s) : a.dk == 128 ? grads<128, T>(a, g, s) : grads<256, T>(a, g, s);
}

}  // namespace
}  // namespace delta

using namespace delta;

// The workspace: the tables, then the records of every (sequence, head, chunk).
size_t delta_backward_ws_bytes(const DeltaArgs& a) {
    const size_t n = (size_t)a.B * a.H * chunks_of(a.N) * groups_of(a.dv);
    return (table_bytes(a) + 255) / 256 * 256 + n * record_bytes(a.dk);
}

ret_status launch_delta_backward(const DeltaArgs& a, void* ws, cudaStream_t s) {
    const Tables t = tables_at(a, ws);
    uint8_t* records = reinterpret_cast<uint8_t*>(ws) + (table_bytes(a) + 255) / 256 * 256;
    ret_status st = launch_prep(a, t, s);
    if (st != RET_OK) return st;
    if ((st = launch_chains(a, t, records, s)) != RET_OK) return st;
    GradArgs g{};
    g.tb = t;
    g.lengths = a.lengths;
    g.v = (const __nv_bfloat16*)a.v;
    g.records = records;
    g.dq = a.dq; g.dk = a.dkk; g.dv = a.dvv;
    g.dg = a.dg; g.dbeta = a.dbeta;
    g.N = a.N; g.nc = chunks_of(a.N); g.Hk = a.Hk; g.H = a.H; g.dv_dim = a.dv;
    return a.grad_dt == RET_F32 ? grads_dk<float>(a, g, s) : grads_dk<__nv_bfloat16>(a, g, s);
}

}  // namespace ret
