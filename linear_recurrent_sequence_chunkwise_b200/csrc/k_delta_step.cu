// k_delta_step.cu -- the gated delta rule token by token: one decode step, and
// a whole sequence on the CUDA cores.  Per value head, S [dk, dv] fp32:
//     S' = exp(g) S,  u = beta (v - S'^T k),  S <- S' + k u^T,  o = S^T q.
// Both dot products run on the old state, so a step needs one reduction:
//     u = beta (v - a S^T k),  o = a S^T q + (q . k) u,  a = exp(g).
#include <algorithm>

#include "kernels.h"
#include "tc_util.cuh"
#include "tmap.h"

namespace ret {

static __device__ int g_step_err = 0;

cudaError_t read_clear_error_delta_step(int* flag) {
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_step_err, sizeof(int));
    if (e == cudaSuccess && *flag) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_step_err, &zero, sizeof(int));
    }
    return e;
}

namespace {

// ---------------------------------------------------------------- one step
//
// Bound by memory: the state is read and written once.  A block holds 4 CL
// columns of one (sequence, head) in registers, all of dk: CL lanes of four
// consecutive columns, the other lanes and warps over the rows.  The
// reduction over the rows goes through shared memory once, then the block
// updates its registers and writes them back.
template <typename Tin, typename Tout, int CL, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) k_delta_step(const Tin* __restrict__ q, const Tin* __restrict__ k,
                                                          const Tin* __restrict__ v, const float* __restrict__ g,
                                                          const float* __restrict__ beta, float* __restrict__ state,
                                                          Tout* __restrict__ out, int Hk, int H, int dk, int dv, int ncol) {
    constexpr int RL = WARPS * (32 / CL);      // threads over the rows
    constexpr int R = kDeltaMaxDk / RL;        // rows of a thread
    __shared__ float ks[kDeltaMaxDk], qs[kDeltaMaxDk];
    __shared__ float4 part[2][WARPS][CL];
    __shared__ float4 us[CL];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int cl = lane % CL, rl = w * (32 / CL) + lane / CL;
    const size_t bh = blockIdx.x / ncol;  // the blocks of a head follow one another: they share its rows
    const int b = (int)(bh / H), h = (int)(bh % H);
    const size_t kb = ((size_t)b * Hk + h / (H / Hk)) * dk;
    const int c = ((int)(blockIdx.x % ncol) * CL + cl) * 4;
    const bool live = c < dv;
    float4* S = reinterpret_cast<float4*>(state + bh * dk * dv + min(c, dv - 4));
    const size_t ld = dv / 4;

    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; i++) {
        // rows behind the last one meet k = q = 0 (no branch around the load)
        s[i] = __ldcs(S + (size_t)min(rl + i * RL, dk - 1) * ld);
    }
    for (int i = tid; i < kDeltaMaxDk; i += WARPS * 32) {
        const float kx = ld_as_float(k, kb + min(i, dk - 1)), qx = ld_as_float(q, kb + min(i, dk - 1));
        ks[i] = i < dk ? kx : 0.f;
        qs[i] = i < dk ? qx : 0.f;
    }
    const float a = expf(g[bh]), bt = beta[bh];
    __syncthreads();

    float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
#pragma unroll
    for (int i = 0; i < R; i++) {
        const float kr = ks[rl + i * RL], qr = qs[rl + i * RL];
        sk.x = fmaf(kr, s[i].x, sk.x); sk.y = fmaf(kr, s[i].y, sk.y);
        sk.z = fmaf(kr, s[i].z, sk.z); sk.w = fmaf(kr, s[i].w, sk.w);
        sq.x = fmaf(qr, s[i].x, sq.x); sq.y = fmaf(qr, s[i].y, sq.y);
        sq.z = fmaf(qr, s[i].z, sq.z); sq.w = fmaf(qr, s[i].w, sq.w);
    }
#pragma unroll
    for (int o = CL; o < 32; o <<= 1) {
        sk.x += __shfl_xor_sync(0xffffffffu, sk.x, o); sk.y += __shfl_xor_sync(0xffffffffu, sk.y, o);
        sk.z += __shfl_xor_sync(0xffffffffu, sk.z, o); sk.w += __shfl_xor_sync(0xffffffffu, sk.w, o);
        sq.x += __shfl_xor_sync(0xffffffffu, sq.x, o); sq.y += __shfl_xor_sync(0xffffffffu, sq.y, o);
        sq.z += __shfl_xor_sync(0xffffffffu, sq.z, o); sq.w += __shfl_xor_sync(0xffffffffu, sq.w, o);
    }
    if (lane < CL) {
        part[0][w][cl] = sk;
        part[1][w][cl] = sq;
    }
    __syncthreads();
    if (w == 0) {
        float kq = 0.f;
        for (int i = lane; i < kDeltaMaxDk; i += 32) kq = fmaf(ks[i], qs[i], kq);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
        if (lane < CL) {
            sk = part[0][0][cl];
            sq = part[1][0][cl];
#pragma unroll
            for (int i = 1; i < WARPS; i++) {
                const float4 x = part[0][i][cl], y = part[1][i][cl];
                sk.x += x.x; sk.y += x.y; sk.z += x.z; sk.w += x.w;
                sq.x += y.x; sq.y += y.y; sq.z += y.z; sq.w += y.w;
            }
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live) {
                const size_t e = bh * dv + c;
                u.x = bt * (ld_as_float(v, e) - a * sk.x);
                u.y = bt * (ld_as_float(v, e + 1) - a * sk.y);
                u.z = bt * (ld_as_float(v, e + 2) - a * sk.z);
                u.w = bt * (ld_as_float(v, e + 3) - a * sk.w);
                st_from_float(out, e, fmaf(kq, u.x, a * sq.x));
                st_from_float(out, e + 1, fmaf(kq, u.y, a * sq.y));
                st_from_float(out, e + 2, fmaf(kq, u.z, a * sq.z));
                st_from_float(out, e + 3, fmaf(kq, u.w, a * sq.w));
            }
            us[cl] = u;
        }
    }
    __syncthreads();
    const float4 u = us[cl];
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int r = rl + i * RL;
        if (live && r < dk) {
            const float kr = ks[r];
            float4 x = s[i];
            x.x = fmaf(kr, u.x, a * x.x);
            x.y = fmaf(kr, u.y, a * x.y);
            x.z = fmaf(kr, u.z, a * x.z);
            x.w = fmaf(kr, u.w, a * x.w);
            __stcs(S + (size_t)r * ld, x);
        }
    }
}

// The same for a large batch: one block per SM walks tiles of 32 columns (all
// of dk, up to 32 KB) that TMA brings into a ring of stages and takes back
// from them, so the loads of the next tiles and the stores of the last ones
// run beside the arithmetic.  A lane has four columns of every 32nd row.  Two
// groups of warps take turns at the tiles: one's reductions and barriers hide
// behind the other's.  64 sequences of 16 heads of 256 x 512, 1.07 GB: 169 us,
// 6.4 TB/s (one group alone 240 us; the kernel above 285 us).
constexpr int kRingGroups = 2, kRingWarps = 8, kRingCols = 32;  // warps of a group
constexpr int kRingBytes = 192 * 1024;
constexpr double kRingMin = 64e6;  // bytes of state

template <typename Tin, typename Tout, int R>
__global__ void __launch_bounds__(kRingGroups * kRingWarps * 32, 1)
    k_delta_step_ring(const __grid_constant__ CUtensorMap map, const Tin* __restrict__ q, const Tin* __restrict__ k,
                      const Tin* __restrict__ v, const float* __restrict__ g, const float* __restrict__ beta,
                      Tout* __restrict__ out, int Hk, int H, int dk, int dv, int ncol, int tiles) {
    constexpr int kRows = kRingWarps * 4;  // rows of the block at a time; a thread has R of them
    constexpr int kStage = R * kRows * kRingCols * 4, NS = kRingBytes / kStage;
    constexpr int kAhead = NS - kRingGroups;  // loads ahead of a tile
    extern __shared__ __align__(128) uint8_t raw[];
    uint8_t* sm = raw + ((128 - (tc::smem_u32(raw) & 127)) & 127);
    __shared__ uint64_t full[NS];
    __shared__ float2 kq_[kRingGroups][2][kDeltaMaxDk];
    __shared__ __align__(16) float part_[kRingGroups][2][2][kRingWarps][kRingCols];
    __shared__ float dots_[kRingGroups][2][kRingWarps];
    constexpr int kThreads = kRingWarps * 32;
    const int gi = threadIdx.x / kThreads, tid = threadIdx.x % kThreads, lane = tid & 31, w = tid >> 5;
    auto& kq = kq_[gi];
    auto& part = part_[gi];
    auto& dots = dots_[gi];
    const int first = blockIdx.x, step = gridDim.x;
    const int n = (tiles - first + step - 1) / step;
    const uint32_t bytes = (uint32_t)dk * kRingCols * 4;  // a box, zeros outside the tensor included
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; i++) tc::mbar_init(full + i, 1);
        tc::fence_barrier_init();
        tc::fence_proxy_async_smem();
    }
    __syncthreads();
    auto load = [&](int i) {  // one thread
        const int t = first + i * step;
        uint64_t* bar = full + i % NS;
        tc::mbar_arrive_expect_tx(bar, bytes);
        tc::tma_load_2d(sm + (i % NS) * kStage, &map, bar, t % ncol * kRingCols, t / ncol * dk);
    };
    const int cq = (lane & 7) * 4, row0 = w * 4 + (lane >> 3);
    float kn = 0.f, qn = 0.f, vn[4] = {0.f, 0.f, 0.f, 0.f}, gn = 0.f, bn = 0.f;
    // A tile's small inputs, a tile ahead; lanes without a share read another's
    // (a branch around a load would wait for the load).
    auto fetch = [&](int i) {
        const int t = min(first + i * step, tiles - 1), bh = t / ncol;
        const int c = min((t - bh * ncol) * kRingCols + cq, dv - 4), bb = bh / H;
        const size_t kb = ((size_t)bb * Hk + (bh - bb * H) / (H / Hk)) * dk + min(tid, dk - 1);
        kn = ld_as_float(k, kb);
        qn = ld_as_float(q, kb);
#pragma unroll
        for (int j = 0; j < 4; j++) vn[j] = ld_as_float(v, (size_t)bh * dv + c + j);
        gn = g[bh];
        bn = beta[bh];
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < kAhead && i < n; i++) load(i);
    fetch(gi);
    for (int i = gi; i < n; i += kRingGroups) {
        const int t = first + i * step, bh = t / ncol;
        const int c = (t - bh * ncol) * kRingCols + cq, hb = (i / kRingGroups) & 1;
        kq[hb][tid] = make_float2(kn, qn);
        const float4 vc = make_float4(vn[0], vn[1], vn[2], vn[3]);
        const float a = expf(gn), bt = bn;
        fetch(i + kRingGroups);
        const bool ok = tc::mbar_wait(full + i % NS, (i / NS) & 1);
        if (!tc::barrier_and(1 + gi, kThreads, ok)) {  // the group leaves, behind its loads; its stores are waited for below
            if (tid == 0) {
                atomicExch(&g_step_err, kErrTimeout);
                for (int j = i; j < i + kAhead && j < n; j += kRingGroups) tc::mbar_wait(full + j % NS, (j / NS) & 1);
            }
            break;
        }
        float4* S = reinterpret_cast<float4*>(sm + (i % NS) * kStage) + row0 * (kRingCols / 4) + (lane & 7);
        float4 s[R];
        float d[8], dot = 0.f;  // S^T k, S^T q of the four columns
#pragma unroll
        for (int j = 0; j < 8; j++) d[j] = 0.f;
#pragma unroll
        for (int r = 0; r < R; r++) {
            s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row0 + r * kRows < dk) {
                const float2 x = kq[hb][row0 + r * kRows];
                s[r] = S[r * kRows * (kRingCols / 4)];
                d[0] = fmaf(x.x, s[r].x, d[0]);
                d[1] = fmaf(x.x, s[r].y, d[1]);
                d[2] = fmaf(x.x, s[r].z, d[2]);
                d[3] = fmaf(x.x, s[r].w, d[3]);
                d[4] = fmaf(x.y, s[r].x, d[4]);
                d[5] = fmaf(x.y, s[r].y, d[5]);
                d[6] = fmaf(x.y, s[r].z, d[6]);
                d[7] = fmaf(x.y, s[r].w, d[7]);
                dot = fmaf(x.x, x.y, dot);
            }
        }
        // over the four rows of a warp: each exchange halves what a lane goes on with
#pragma unroll
        for (int o = 16, m = 4; o >= 8; o >>= 1, m >>= 1)
#pragma unroll
            for (int j = 0; j < m; j++) {
                const bool up = lane & o;
                const float give = up ? d[j] : d[j + m];
                d[j] = (up ? d[j + m] : d[j]) + __shfl_xor_sync(0xffffffffu, give, o);
            }
        dot += __shfl_xor_sync(0xffffffffu, dot, 16);
        dot += __shfl_xor_sync(0xffffffffu, dot, 8);
        *reinterpret_cast<float2*>(&part[hb][lane >> 4][w][cq + ((lane >> 3) & 1) * 2]) = make_float2(d[0], d[1]);
        if (lane == 0) dots[hb][w] = dot;
        tc::barrier(1 + gi, kThreads);
        auto total = [&](int which) {
            float4 x = *reinterpret_cast<const float4*>(&part[hb][which][0][cq]);
#pragma unroll
            for (int j = 1; j < kRingWarps; j++) {
                const float4 y = *reinterpret_cast<const float4*>(&part[hb][which][j][cq]);
                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
            }
            return x;
        };
        const float4 sk = total(0);
        const float4 u = make_float4(bt * (vc.x - a * sk.x), bt * (vc.y - a * sk.y), bt * (vc.z - a * sk.z), bt * (vc.w - a * sk.w));
        if (w == kRingWarps - 1 && lane < 8 && c < dv) {
            const float4 sq = total(1);
            dot = dots[hb][0];
#pragma unroll
            for (int j = 1; j < kRingWarps; j++) dot += dots[hb][j];
            const size_t e = (size_t)bh * dv + c;
            st_from_float(out, e, fmaf(dot, u.x, a * sq.x));
            st_from_float(out, e + 1, fmaf(dot, u.y, a * sq.y));
            st_from_float(out, e + 2, fmaf(dot, u.z, a * sq.z));
            st_from_float(out, e + 3, fmaf(dot, u.w, a * sq.w));
        }
#pragma unroll
        for (int r = 0; r < R; r++)
            if (row0 + r * kRows < dk) {
                const float kr = kq[hb][row0 + r * kRows].x;
                S[r * kRows * (kRingCols / 4)] = make_float4(fmaf(kr, u.x, a * s[r].x), fmaf(kr, u.y, a * s[r].y),
                                                             fmaf(kr, u.z, a * s[r].z), fmaf(kr, u.w, a * s[r].w));
            }
        tc::fence_proxy_async_smem();
        tc::barrier(1 + gi, kThreads);
        if (tid == 0) {
            tc::tma_store_2d(&map, sm + (i % NS) * kStage, c - cq, bh * dk);
            tc::bulk_commit_group();
            // tile i - 2 was this group's too, and its store has read its stage: load into it
            static_assert(kAhead == NS - kRingGroups, "");
            if (i + kAhead < n) {
                tc::bulk_wait_group_read<1>();
                load(i + kAhead);
            }
        }
    }
    if (tid == 0) tc::bulk_wait_group<0>();
}

// -------------------------------------------------------- a whole sequence
//
// Bound by the latency of a token: a warp keeps four columns of the state in
// registers (lane l the rows l, l + 32, ...) and reduces the eight dot
// products of a token together: each exchange halves the values a lane
// holds, so the eight cost nine exchanges instead of forty.  The next
// token's q, k, v and gates are loaded before the current one is computed.
template <typename Tin, typename Tout, int R>
__global__ void __launch_bounds__(128) k_delta_recurrent(DeltaArgs a) {
    const Tin* q = (const Tin*)a.q;
    const Tin* k = (const Tin*)a.k;
    const Tin* v = (const Tin*)a.v;
    Tout* out = (Tout*)a.out;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c0 = (blockIdx.x * 4 + w) * 4;
    if (c0 >= a.dv) return;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.H / a.Hk);
    const int len = a.lengths ? max(0, min(a.lengths[b], a.N)) : a.N;
    const size_t sb = ((size_t)b * a.H + h) * a.dk * a.dv;
    float S[R][4];
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int r = lane + 32 * i;
            S[i][j] = a.initial_state && r < a.dk && c0 + j < a.dv ? a.initial_state[sb + (size_t)r * a.dv + c0 + j] : 0.f;
        }
    float kn[R], qn[R], vn[4], gn = 0.f, bn = 0.f;
    auto load = [&](int t) {
        const size_t tk = (((size_t)b * a.N + t) * a.Hk + hk) * a.dk, th = ((size_t)b * a.N + t) * a.H + h;
#pragma unroll
        for (int i = 0; i < R; i++) {
            const int r = lane + 32 * i;
            kn[i] = r < a.dk ? ld_as_float(k, tk + r) : 0.f;
            qn[i] = r < a.dk ? ld_as_float(q, tk + r) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; j++) vn[j] = c0 + j < a.dv ? ld_as_float(v, th * a.dv + c0 + j) : 0.f;
        gn = a.g[th];
        bn = a.beta[th];
    };
    if (len > 0) load(0);
    for (int t = 0; t < len; t++) {
        float kk[R], qq[R], vv[4];
#pragma unroll
        for (int i = 0; i < R; i++) kk[i] = kn[i], qq[i] = qn[i];
#pragma unroll
        for (int j = 0; j < 4; j++) vv[j] = vn[j];
        const float al = expf(gn), bt = bn;
        if (t + 1 < len) load(t + 1);
        float d[8], kq = 0.f;  // S^T k of the four columns, then S^T q
#pragma unroll
        for (int j = 0; j < 8; j++) d[j] = 0.f;
#pragma unroll
        for (int i = 0; i < R; i++) {
            kq = fmaf(kk[i], qq[i], kq);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                d[j] = fmaf(kk[i], S[i][j], d[j]);
                d[4 + j] = fmaf(qq[i], S[i][j], d[4 + j]);
            }
        }
#pragma unroll
        for (int o = 16, n = 4; o >= 4; o >>= 1, n >>= 1)
#pragma unroll
            for (int j = 0; j < n; j++) {
                const bool up = lane & o;
                const float give = up ? d[j] : d[j + n];
                const float keep = up ? d[j + n] : d[j];
                d[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        d[0] += __shfl_xor_sync(0xffffffffu, d[0], 2);
        d[0] += __shfl_xor_sync(0xffffffffu, d[0], 1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
        const float mine = d[0];  // lanes 4 m .. 4 m + 3 hold dot product m
        float u[4], o4[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float sk = __shfl_sync(0xffffffffu, mine, 4 * j), sq = __shfl_sync(0xffffffffu, mine, 16 + 4 * j);
            u[j] = bt * (vv[j] - al * sk);
            o4[j] = fmaf(kq, u[j], al * sq);
        }
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) S[i][j] = fmaf(kk[i], u[j], al * S[i][j]);
        if (lane < 4 && c0 + lane < a.dv) {
            const float o = lane == 0 ? o4[0] : lane == 1 ? o4[1] : lane == 2 ? o4[2] : o4[3];
            st_from_float(out, (((size_t)b * a.N + t) * a.H + h) * a.dv + c0 + lane, o);
        }
    }
    if (a.final_state) {
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int r = lane + 32 * i;
                if (r < a.dk && c0 + j < a.dv) a.final_state[sb + (size_t)r * a.dv + c0 + j] = S[i][j];
            }
    }
}

template <typename Tin, typename Tout, int R>
ret_status step_ring(const DeltaArgs& a, float* state, cudaStream_t s) {
    const uint64_t dims[2] = {(uint64_t)a.dv, (uint64_t)a.B * a.H * a.dk};
    const uint64_t strides[1] = {(uint64_t)a.dv * 4};
    const uint32_t box[2] = {kRingCols, (uint32_t)a.dk};
    CUtensorMap map;
    if (!make_tmap_f32(&map, state, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE)) return RET_ERR_CUDA;
    auto kern = k_delta_step_ring<Tin, Tout, R>;
    constexpr int smem = kRingBytes + 128;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "ret_delta_decode_step: %s", cudaGetErrorString(e));
    const int ncol = (a.dv + kRingCols - 1) / kRingCols;
    const long long tiles = (long long)a.B * a.H * ncol;
    kern<<<(unsigned)std::min<long long>(148, tiles), kRingGroups * kRingWarps * 32, smem, s>>>(
        map, (const Tin*)a.q, (const Tin*)a.k, (const Tin*)a.v, a.g, a.beta, (Tout*)a.out, a.Hk, a.H, a.dk, a.dv, ncol,
        (int)tiles);
    return check_launch("ret_delta_decode_step");
}

template <typename Tin, typename Tout>
ret_status step(const DeltaArgs& a, float* state, cudaStream_t s) {
    const unsigned bh = (unsigned)(a.B * a.H), wide = (a.dv + 63) / 64, narrow = (a.dv + 15) / 16;
    // The ring when every SM has work for a while (kRingMin bytes of state in
    // all) and rows and tiles fit 31 bits.
    if ((double)bh * a.dk * a.dv * 4 >= kRingMin && (long long)bh * a.dk < (1ll << 31) &&
        (long long)bh * ((a.dv + kRingCols - 1) / kRingCols) < (1ll << 30))
        return a.dk <= 64    ? step_ring<Tin, Tout, 2>(a, state, s)
               : a.dk <= 128 ? step_ring<Tin, Tout, 4>(a, state, s)
                             : step_ring<Tin, Tout, 8>(a, state, s);
    // 64 columns a block (256-byte rows of the state) when that gives two
    // blocks for each of the 148 SMs, else 16 columns for more blocks.
    if ((long long)wide * bh >= 296)
        k_delta_step<Tin, Tout, 16, 16><<<wide * bh, 512, 0, s>>>(
            (const Tin*)a.q, (const Tin*)a.k, (const Tin*)a.v, a.g, a.beta, state, (Tout*)a.out, a.Hk, a.H, a.dk, a.dv,
            wide);
    else
        k_delta_step<Tin, Tout, 4, 8><<<narrow * bh, 256, 0, s>>>(
            (const Tin*)a.q, (const Tin*)a.k, (const Tin*)a.v, a.g, a.beta, state, (Tout*)a.out, a.Hk, a.H, a.dk, a.dv,
            narrow);
    return check_launch("ret_delta_decode_step");
}

template <typename Tin, typename Tout>
void recurrent(const DeltaArgs& a, cudaStream_t s) {
    const dim3 grid((a.dv + 15) / 16, a.H, a.B);
    if (a.dk <= 32) k_delta_recurrent<Tin, Tout, 1><<<grid, 128, 0, s>>>(a);
    else if (a.dk <= 64) k_delta_recurrent<Tin, Tout, 2><<<grid, 128, 0, s>>>(a);
    else if (a.dk <= 128) k_delta_recurrent<Tin, Tout, 4><<<grid, 128, 0, s>>>(a);
    else k_delta_recurrent<Tin, Tout, 8><<<grid, 128, 0, s>>>(a);
}

}  // namespace

ret_status launch_delta_step(const DeltaArgs& a, float* state, cudaStream_t s) {
    if (a.in_dt == RET_F32)
        return a.out_dt == RET_F32 ? step<float, float>(a, state, s) : step<float, __nv_bfloat16>(a, state, s);
    return a.out_dt == RET_F32 ? step<__nv_bfloat16, float>(a, state, s) : step<__nv_bfloat16, __nv_bfloat16>(a, state, s);
}

ret_status launch_delta_recurrent(const DeltaArgs& a, cudaStream_t s) {
    if (a.in_dt == RET_F32) a.out_dt == RET_F32 ? recurrent<float, float>(a, s) : recurrent<float, __nv_bfloat16>(a, s);
    else a.out_dt == RET_F32 ? recurrent<__nv_bfloat16, float>(a, s) : recurrent<__nv_bfloat16, __nv_bfloat16>(a, s);
    return check_launch("ret_delta_forward_chunkwise: token by token");
}

}  // namespace ret
