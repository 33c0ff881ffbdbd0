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
// dg_i is the sum of what passes row i: from the state before to rows from i
// on, from rows before i to the state after, from state to state, from rows to
// rows (dq0 and r0 are dq and r without their sums over j):
//     dg_i = sum_{j>=i} (q_j . dq0_j + beta_j k_j . r0_j) + sum_{j<i} k_j . z_j
//            + exp(G_C) <dS1, S0> + sum_{a>=i>b} X_ab,
//     X_ab = E_ab D_ab q_a . k_b - beta_a W_ab D_ab k_a . k_b,
// the last as sums of rows less sums of columns from i on, in 64 bits, where the
// pairs on one side of i cancel to the bit.  (As row sums of q . dq + beta k . r -
// k . w, each rounded by itself, they left 2^-22 of |q . dq|: 1% of dg behind a
// decay of 1e-11.)  Then dq' = dq / s_q and so on undo the scaling.
//
// A key head's gradient is the sum over its value heads: one block takes them
// all, one after the other, so the order is fixed.  Sixteen warps: a row group
// of 16 tokens and a quarter of dk each.  The records of 16 value columns come
// through a ring of bulk copies that runs on across value heads and chunks (one
// block an SM, each walking its share of the chunks),
// and the five products over dv accumulate in registers; then the 64 x 64
// scores go through shared memory once, in two terms, to meet K and Q.
//
// Each group's products are added in fp32 (in one accumulator over all groups 18
// us less, but dg off by half as much again: the tensor cores round towards zero).
//
// 1 x 4096, 16 heads of 128 / 128: 232 us, 31 us for a chunk and head (221 us before
// the fences and votes).  Bound by the latency of 16 warps at 128 registers (IPC 1.5;
// 264 bytes of spills a thread at dk 128, 24 at 64, 1,700 at 256), of which the five
// products need 8 us; 272 MB of records are read at 1.2 TB/s.
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
    const uint8_t* records;
    float4* sums;  // more than one value head to a key head: its gradients so far
    void *dq, *dk, *dv;
    float *dg, *dbeta;
    int N, nc, Hk, H, dv_dim, B;
};

template <int DK>
struct Grad {
    static constexpr int NH = 4, warps = 4 * NH;       // column shares
    static constexpr int threads = warps * 32;
    static constexpr int DW = DK / NH;                 // dk columns of a warp
    static constexpr int oK = 0, oQ = 2 * C * DK;      // K, Q
    static constexpr int oE = 4 * C * DK;              // E D, W D, beta W D: hi, lo each
    static constexpr int oR = oE + 6 * kTile;          // the ring
    // a stage: a record, 16 columns of V, the head's gates
    static constexpr int oV = Record<DK>::bytes, oGate = oV + C * 32, stage = (oGate + kGateRow + 127) / 128 * 128;
    static constexpr int most = 218 * 1024, fit = (most - oR) / stage, stages = fit > 6 ? 6 : fit;
    static constexpr int smem = oR + stages * stage + 1024;
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

template <int N>
__device__ __forceinline__ void times(float (&acc)[N][4], float f0, float f1) {
#pragma unroll
    for (int n = 0; n < N; n++) acc[n][0] *= f0, acc[n][1] *= f0, acc[n][2] *= f1, acc[n][3] *= f1;
}

template <int DK, typename T>
__global__ void __launch_bounds__(Grad<DK>::threads, 1) k_delta_grads(const __grid_constant__ CUtensorMap mv,
                                                                          const __grid_constant__ GradArgs a) {
    using Gr = Grad<DK>;
    using Rec = Record<DK>;
    constexpr int NH = Gr::NH, DW = Gr::DW, NS = Gr::stages;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[NS], empty[NS], keys;
    __shared__ int filled, asked;  // thread 0's: stages, and K and Q, that it asked for
    __shared__ float inv_e[4][4], inv_w[4][4], inv_b[4][4];
    __shared__ float row_a[NH][C], row_c[NH][C], row_b[NH][C], red[Gr::warps];
    __shared__ double row_x[NH][C], col_x[4][C];  // of X
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rep = a.H / a.Hk, ng = groups_of(a.dv_dim);
    T* dq = reinterpret_cast<T*>(a.dq);
    T* dk = reinterpret_cast<T*>(a.dk);
    T* dv = reinterpret_cast<T*>(a.dv);
    // Items: (chunk, key head, sequence).  A block takes every gridDim.x-th, and
    // its ring runs on from one to the next.
    const int items = a.nc * a.Hk * a.B;
    auto tokens_of = [&](int item) {
        return min(C, length_of(a.lengths, item / (a.nc * a.Hk), a.N) - item % a.nc * C);
    };
    if (tid == 0) {
        for (int i = 0; i < NS; i++) tc::mbar_init(full + i, 1), tc::mbar_init(empty + i, Gr::warps);
        tc::mbar_init(&keys, 1);
        filled = asked = 0;
        tc::fence_barrier_init();
    }
    __syncthreads();
    // After a wait that gave up the others are skipped: the barriers stay complete.
    bool ok = true;
    auto wait_lane = [&](uint64_t* bar, int phase) {
        if (ok && !tc::mbar_wait(bar, phase & 1)) {
            ok = false;
            atomicExch(&g_grad_err, kErrTimeout);
        }
    };
    // A warp's wait ends in a vote: polling ends lane by lane, and ldmatrix and
    // mma.sync are defined only for a warp whose lanes execute them together.
    auto wait = [&](uint64_t* bar, int phase) {
        wait_lane(bar, phase);
        ok = __all_sync(0xffffffffu, ok);
    };
    // A warp hands a stage back.  It has read it through the generic proxy and the
    // copies write through the async proxy: the mbarrier alone does not order them.
    auto release = [&](uint64_t* bar) {
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    };
    // One lane: the next record, its columns of V and its head's gates into the
    // ring, ahead of the warps.
    int ahead = blockIdx.x, stage = 0, round = 0, group = 0, head = 0, row = 0, seq = 0;
    size_t chunk = 0;
    auto find = [&]() {  // the next item with tokens
        while (ahead < items && tokens_of(ahead) <= 0) ahead += gridDim.x;
        if (ahead >= items) return;
        const int c = ahead % a.nc, x = ahead / a.nc;
        seq = x / a.Hk, head = x % a.Hk * rep, row = c * C;
        chunk = ((size_t)seq * a.H + head) * a.nc + c;
    };
    auto load = [&]() {
        if (ahead >= items) return;
        uint64_t* bar = full + stage;
        if (round > 0) wait_lane(empty + stage, round - 1);
        if (ok) {
            filled++;
            uint8_t* st = sm + Gr::oR + stage * Gr::stage;
            tc::mbar_arrive_expect_tx(bar, Rec::bytes + C * 32 + kGateRow);
            bulk_load(st, a.records + (chunk * ng + group) * Rec::bytes, Rec::bytes, bar);
            bulk_load(st + Gr::oGate, a.tb.gates + chunk * kGateRow, kGateRow, bar);
            tc::tma_load_4d(st + Gr::oV, &mv, bar, 16 * group, head, row, seq);
        }
        if (++stage == NS) stage = 0, round++;
        if (++group < ng) return;
        group = 0, head++, chunk += a.nc;
        if (head % rep == 0) {
            ahead += gridDim.x;
            find();
        }
    };
    if (tid == 0) find();
    if (tid == 0)
        for (int i = 0; i < NS - 1; i++) load();
    __syncwarp();

    const int rg = w & 3, cg = w >> 2;  // row group, column share
    const int g = lane >> 2, t = lane & 3;
    const uint32_t base = tc::smem_u32(sm), sK = base + Gr::oK, sQ = base + Gr::oQ, sE = base + Gr::oE;
    const int i0 = 16 * rg + g, i1 = i0 + 8;
    int it = 0, done = 0;  // steps and items so far

    for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int c = item % a.nc, hk = item / a.nc % a.Hk, b = item / (a.nc * a.Hk);
    const int L = tokens_of(item);
    const int rows = min(C, a.N - c * C);  // rows of the tensors in this chunk
    const size_t row0 = (size_t)b * a.N + (size_t)c * C;
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
        continue;
    }
    if (tid == 0 && ok) {  // K and Q: the last item's readers have passed its last barrier
        asked++;
        tc::mbar_arrive_expect_tx(&keys, 4 * C * DK);
        bulk_load(sm, a.tb.keys + (((size_t)b * a.Hk + hk) * a.nc + c) * (4 * C * DK), 4 * C * DK, &keys);
    }
    __syncwarp();
    float ik0 = 0.f, ik1 = 0.f, sq0 = 0.f, sq1 = 0.f;  // 1 / s_k and s_q of rows i0 and i1

    for (int r = 0; r < rep; r++) {
        const int h = hk * rep + r;
        const float* gt = nullptr;
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
        float b0 = 0.f, b1 = 0.f;

        for (int gr = 0; gr < ng; gr++, it++) {
            const int st = it % NS;
            if (tid == 0) load();
            ok = __all_sync(0xffffffffu, ok);
            const uint8_t* rec = sm + Gr::oR + st * Gr::stage;
            const uint32_t sr = tc::smem_u32(rec);
            const float* f = reinterpret_cast<const float*>(rec + Rec::f);
            wait(full + st, it / NS);
            gt = reinterpret_cast<const float*>(rec + Gr::oGate);
            if (gr == 0) {
                b0 = gt[gBeta + i0], b1 = gt[gBeta + i1], ik0 = gt[gIk + i0], ik1 = gt[gIk + i1];
                sq0 = gt[gSq + i0], sq1 = gt[gSq + i1];
            }
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
                const float ie = io * iu, iw = iy * iu;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float x[4], y[4];
                    mma0(x, ao, bl[2 * i], bl[2 * i + 1]);
                    mma0(y, yl, bh[2 * i], bh[2 * i + 1]);
                    mma(x, ao, bh[2 * i], bh[2 * i + 1]);
                    mma(y, yh, bl[2 * i], bl[2 * i + 1]);
                    mma(y, yh, bh[2 * i], bh[2 * i + 1]);
                    add_scaled(E[i], x, ie);
                    add_scaled(W[i], y, iw);
                }
            }
            const float is = f[fS + cg / 2], id = f[fDs + cg / 2];
            const float iq = io * is, iz = iy * is, iw = iu * id;
#pragma unroll
            for (int p = 0; p < DW / 16; p++) {
                uint32_t bh[4], bl[4];
                const uint32_t off = at_k<16>(0, 0, cg * (DW / 8) + 2 * p, lane);
                ldsm4_t(bh, sr + Rec::s + off);
                ldsm4_t(bl, sr + Rec::s + 32 * DK + off);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float x[4], y[4];
                    mma0(x, ao, bl[2 * i], bl[2 * i + 1]);
                    mma0(y, yl, bh[2 * i], bh[2 * i + 1]);
                    mma(x, ao, bh[2 * i], bh[2 * i + 1]);
                    mma(y, yh, bl[2 * i], bl[2 * i + 1]);
                    mma(y, yh, bh[2 * i], bh[2 * i + 1]);
                    add_scaled(Zq[2 * p + i], x, iq);
                    add_scaled(Z[2 * p + i], y, iz);
                }
                ldsm4_t(bh, sr + Rec::ds + off);
                ldsm4_t(bl, sr + Rec::ds + 32 * DK + off);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float x[4];
                    mma0(x, ul, bh[2 * i], bh[2 * i + 1]);
                    mma(x, uh, bl[2 * i], bl[2 * i + 1]);
                    mma(x, uh, bh[2 * i], bh[2 * i + 1]);
                    add_scaled(Zw[2 * p + i], x, iw);
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
            // dv and Y . v: a share takes every fourth group
            if ((gr & 3) == cg) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int row = 16 * rg + g + 8 * (e & 1), col = 16 * gr + 2 * t + 8 * (e >> 1);
                    const uint32_t v2 = *reinterpret_cast<const uint32_t*>(rec + Gr::oV + row * 32 + 4 * t + 16 * (e >> 1));
                    float2 y = sum_h2(yh[e], yl[e]);
                    y.x *= iy;
                    y.y *= iy;
                    const float s = (e & 1 ? b1 * ik1 : b0 * ik0);  // dv = beta' Y / s_k
                    if (row < rows && col < a.dv_dim)
                        st_pair(dv + ((row0 + row) * a.H + h) * a.dv_dim + col, s * y.x, s * y.y);
                    const float d = row < L ? fmaf(y.x, tc::bf16lo(v2), y.y * tc::bf16hi(v2)) : 0.f;
                    if (e & 1) db1 = fmaf(d, ik1, db1);
                    else db0 = fmaf(d, ik0, db0);
                }
            }
            // the last stage of a head holds the gates until its end
            if (gr < ng - 1) release(empty + st);
        }
        const double* G = reinterpret_cast<const double*>(reinterpret_cast<const uint8_t*>(gt) + kGates);

        if (r == 0) wait(&keys, done);
        // the scores, with the decays, in two terms; the sums of X
        double xr[2] = {0.0, 0.0}, xc[4] = {0.0, 0.0, 0.0, 0.0};
        if (cg <= rg) {
            float bw[2][4], qk[2][4], kk[2][4];
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) qk[n][e] = kk[n][e] = 0.f;
#pragma unroll 2
            for (int s = 0; s < DK / 16; s++) {
                uint32_t aq[4], ak[4], bk[4];
                ldsm4(aq, at_k(sQ, 16 * rg, 2 * s, lane));
                ldsm4(ak, at_k(sK, 16 * rg, 2 * s, lane));
                ldsm4(bk, at_n(sK, 16 * cg, 2 * s, lane));
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    mma(qk[i], aq, bk[2 * i], bk[2 * i + 1]);
                    mma(kk[i], ak, bk[2 * i], bk[2 * i + 1]);
                }
            }
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
                    const double x = fmaf(E[n][e], qk[n][e], -(bw[n][e] * kk[n][e]));
                    xr[e >> 1] += x;
                    xc[2 * n + (e & 1)] += x;
                }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1)
#pragma unroll
                for (int i = 0; i < 2; i++) xr[i] += __shfl_xor_sync(0xffffffffu, xr[i], o);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 4; i++) xc[i] += __shfl_xor_sync(0xffffffffu, xc[i], o);
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
        tc::barrier(1, Gr::threads);
        if (t == 0) row_x[cg][i0] = xr[0], row_x[cg][i1] = xr[1];
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < 4; i++) col_x[rg][16 * cg + 8 * (i >> 1) + 2 * t + (i & 1)] = xc[i];
        }

        const float eg0 = gt[gEG + i0], eg1 = gt[gEG + i1], ec0 = gt[gEC + i0], ec1 = gt[gEC + i1];
        auto pair_at = [&](int off, int row, int n) {
            return unpack_h2(*reinterpret_cast<const uint32_t*>(sm + off + tile_at(row, cg * (DW / 8) + n) + 4 * t));
        };
        times(Zq, eg0, eg1);
        times(Z, eg0, eg1);
        times(Zw, ec0, ec1);
        float ca0 = 0.f, ca1 = 0.f, cc0 = 0.f, cc1 = 0.f;  // row sums of dg
#pragma unroll
        for (int n = 0; n < DW / 8; n++) {
            const float2 x0 = pair_at(Gr::oK, i0, n), x1 = pair_at(Gr::oK, i1, n);
            cc0 = fmaf(x0.x, Zw[n][0], fmaf(x0.y, Zw[n][1], cc0));
            cc1 = fmaf(x1.x, Zw[n][2], fmaf(x1.y, Zw[n][3], cc1));
            const float2 q0 = pair_at(Gr::oQ, i0, n), q1 = pair_at(Gr::oQ, i1, n);
            ca0 += q0.x * Zq[n][0] + q0.y * Zq[n][1] - b0 * (x0.x * Z[n][0] + x0.y * Z[n][1]);
            ca1 += q1.x * Zq[n][2] + q1.y * Zq[n][3] - b1 * (x1.x * Z[n][2] + x1.y * Z[n][3]);
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
                        mma0(x, el, bk[2 * i], bk[2 * i + 1]);
                        mma0(y, wl, bk[2 * i], bk[2 * i + 1]);
                        mma(x, eh, bk[2 * i], bk[2 * i + 1]);
                        mma(y, wh, bk[2 * i], bk[2 * i + 1]);
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
                        mma0(x, el, bq[2 * i], bq[2 * i + 1]);
                        mma0(y, wl, bk[2 * i], bk[2 * i + 1]);
                        mma(x, eh, bq[2 * i], bq[2 * i + 1]);
                        mma(y, wh, bk[2 * i], bk[2 * i + 1]);
                        add_scaled(Zw[2 * p + i], x, ie);
                        add_scaled(Zw[2 * p + i], y, ib);
                    }
                }
            }
        }
        // now Zq = dq, -Z = r, Zw = z + w
#pragma unroll
        for (int n = 0; n < DW / 8; n++) {
            const float2 x0 = pair_at(Gr::oK, i0, n), x1 = pair_at(Gr::oK, i1, n);
            db0 -= x0.x * Z[n][0] + x0.y * Z[n][1];
            db1 -= x1.x * Z[n][2] + x1.y * Z[n][3];
            // dk
#pragma unroll
            for (int e = 0; e < 4; e++) Zw[n][e] -= (e < 2 ? b0 : b1) * Z[n][e];
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
        tc::fence_proxy_async_smem();  // behind this barrier the next K and Q come
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
                    // tiles of X lie on and below the diagonal
                    x[i] += row_a[j][row] + (16 * j <= row ? row_x[j][row] : 0.0) - (16 * j + 15 >= row ? col_x[j][row] : 0.0);
                    z[i] += row_c[j][row];
                    y[i] += row_b[j][row];
                }
            }
            // sums over the rows from one on, and over those before one
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
        release(empty + (it - 1) % NS);
        // the sum over the value heads, in their order, through memory that this
        // thread alone touches (kept in registers over a head they would spill)
        if (rep > 1) {
            float4* sum = a.sums + (size_t)item * (C * DK / 2) + tid;
#pragma unroll
            for (int n = 0; n < DW / 8; n++) {
                float(&x)[4] = Zq[n], (&y)[4] = Zw[n];
                if (r > 0) {
                    const float4 u = sum[2 * n * Gr::threads], v = sum[(2 * n + 1) * Gr::threads];
                    x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
                    y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
                }
                if (r < rep - 1) {
                    sum[2 * n * Gr::threads] = make_float4(x[0], x[1], x[2], x[3]);
                    sum[(2 * n + 1) * Gr::threads] = make_float4(y[0], y[1], y[2], y[3]);
                }
            }
        }
        if (r < rep - 1) continue;
        // undo the scaling
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int row = half ? i1 : i0;
            if (row >= rows) continue;
            const float ik = half ? ik1 : ik0, iq = 1.f / (half ? sq1 : sq0);
#pragma unroll
            for (int n = 0; n < DW / 8; n++) {
                const size_t at = ((row0 + row) * a.Hk + hk) * DK + cg * DW + 8 * n + 2 * t;
                st_pair(dq + at, Zq[n][2 * half] * iq, Zq[n][2 * half + 1] * iq);
                st_pair(dk + at, Zw[n][2 * half] * ik, Zw[n][2 * half + 1] * ik);
            }
        }
    }
    done++;
    }
    // No copy of the block's is in flight when it ends: warp 0 has seen all that it
    // asked for, unless it gave up a wait.
    if (tid == 0 && !ok) {
        for (int i = max(filled - NS, 0); i < filled; i++) tc::mbar_wait(full + i % NS, (i / NS) & 1);
        if (asked) tc::mbar_wait(&keys, (asked - 1) & 1);
    }
}

template <int DK, typename T>
ret_status grads(const DeltaArgs& a, const GradArgs& g, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_delta_grads<DK, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Grad<DK>::smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule gradients: %s", cudaGetErrorString(e));
    // [B, N, heads, dv] as boxes of 16 columns of a head's chunk; zeros behind N and dv
    CUtensorMap mv;
    const uint64_t dims[4] = {(uint64_t)a.dv, (uint64_t)a.H, (uint64_t)a.N, (uint64_t)a.B};
    const uint64_t strides[3] = {(uint64_t)a.dv * 2, (uint64_t)a.H * a.dv * 2, (uint64_t)a.N * a.H * a.dv * 2};
    const uint32_t box[4] = {16, 1, (uint32_t)C, 1};
    if (!make_tmap_bf16(&mv, a.v, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE)) return RET_ERR_CUDA;
    const long long items = (long long)g.nc * a.Hk * a.B;
    k_delta_grads<DK, T><<<(unsigned)std::min<long long>(148, items), Grad<DK>::threads, Grad<DK>::smem, s>>>(mv, g);
    return check_launch("delta rule: gradients");
}

template <typename T>
ret_status grads_dk(const DeltaArgs& a, const GradArgs& g, cudaStream_t s) {
    return a.dk == 64 ? grads<64, T>(a, g, s) : a.dk == 128 ? grads<128, T>(a, g, s) : grads<256, T>(a, g, s);
}

}  // namespace
}  // namespace delta

using namespace delta;

// The workspace: the tables, the records of every (sequence, head, chunk), and
// the sums over the value heads of a key head if it has more than one.
static size_t records_at(const DeltaArgs& a) { return (table_bytes(a) + 255) / 256 * 256; }
static size_t sums_at(const DeltaArgs& a) {
    const size_t n = (size_t)a.B * a.H * chunks_of(a.N) * groups_of(a.dv);
    return (records_at(a) + n * record_bytes(a.dk) + 255) / 256 * 256;
}
size_t delta_backward_ws_bytes(const DeltaArgs& a) {
    return sums_at(a) + (a.H > a.Hk ? (size_t)a.B * a.Hk * chunks_of(a.N) * C * a.dk * 8 : 0);
}

ret_status launch_delta_backward(const DeltaArgs& a, void* ws, cudaStream_t s) {
    const Tables t = tables_at(a, ws);
    uint8_t* records = reinterpret_cast<uint8_t*>(ws) + records_at(a);
    ret_status st = launch_prep(a, t, s);
    if (st != RET_OK) return st;
    if ((st = launch_chains(a, t, records, s)) != RET_OK) return st;
    GradArgs g{};
    g.tb = t;
    g.lengths = a.lengths;
    g.records = records;
    g.sums = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(ws) + sums_at(a));
    g.dq = a.dq; g.dk = a.dkk; g.dv = a.dvv;
    g.dg = a.dg; g.dbeta = a.dbeta;
    g.N = a.N; g.nc = chunks_of(a.N); g.Hk = a.Hk; g.H = a.H; g.dv_dim = a.dv; g.B = a.B;
    return a.grad_dt == RET_F32 ? grads_dk<float>(a, g, s) : grads_dk<__nv_bfloat16>(a, g, s);
}

}  // namespace ret
