// k_delta_chunk.cu -- the gated delta rule over sequences, in chunks of 64
// tokens (formulas and precision: delta_util.cuh).  Two launches:
//
// k_delta_prep, one block per (chunk, value head): the scores K K^T and Q K^T
// on the tensor cores, the decays, T by forward substitution (a thread per
// column, the column in registers) and P, written as swizzled bf16 tiles.
//
// k_delta_chain, one block per (64 value columns, head, sequence): walks the
// chunks with the state in registers.  The columns of the state are
// independent of each other, so a warp carries 16 of them through the whole
// recurrence without a barrier: it holds the transposed state [16 x dk] as
// fp32 accumulator tiles, whose layout is that of the A operand of the next
// product (X^T = S^T K^T, U^T = (beta R)^T T^T, O^T = S^T Q^T + U^T P^T,
// S^T += U^T K), so nothing but the shared K, Q, T, P tiles leaves the
// registers.  One warp feeds the tiles by TMA through a ring of stages.
#include <algorithm>

#include "delta_util.cuh"

namespace ret {

static __device__ int g_delta_err = 0;

cudaError_t read_clear_error_delta(int* flag) {
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_delta_err, sizeof(int));
    if (e == cudaSuccess && *flag) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_delta_err, &zero, sizeof(int));
    }
    return e;
}

namespace delta {

namespace {

// ------------------------------------------------------------ chunk tables

constexpr int kPrepThreads = 128;
template <int DK>
constexpr int prep_smem() {
    const int operands = 2 * C * DK * 2, tiles = 4 * kTile;
    return (operands > tiles ? operands : tiles) + C * C * 4;
}

template <int DK>
__global__ void __launch_bounds__(kPrepThreads) k_delta_prep(DeltaArgs a, uint8_t* __restrict__ tiles,
                                                            uint8_t* __restrict__ gates, int nc) {
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ double sG[C];
    __shared__ float sb[C];
    // K and Q, later the four tiles; then A = diag(beta) M in fp32
    constexpr int kOperands = prep_smem<DK>() - C * C * 4;
    float* sA = reinterpret_cast<float*>(sm + kOperands);
    const int c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int L = min(C, length_of(a.lengths, b, a.N) - c * C);
    if (L <= 0) return;
    const int hk = h / (a.H / a.Hk);
    const size_t ch = ((size_t)b * a.H + h) * nc + c;
    const size_t t0 = (size_t)b * a.N + (size_t)c * C;

    // K and Q rows into shared memory, zeros behind the end
    const uint32_t sK = tc::smem_u32(sm), sQ = sK + C * DK * 2;
    constexpr int kPieces = DK / 8;
    for (int i = tid; i < C * kPieces; i += kPrepThreads) {
        const int r = i / kPieces, p = i % kPieces;
        uint4 k4 = make_uint4(0, 0, 0, 0), q4 = k4;
        if (r < L) {
            const size_t e = ((t0 + r) * a.Hk + hk) * DK + 8 * p;
            k4 = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.k + e);
            q4 = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q + e);
        }
        const uint32_t off = tile_at(0, r, p);
        *reinterpret_cast<uint4*>(sm + off) = k4;
        *reinterpret_cast<uint4*>(sm + C * DK * 2 + off) = q4;
    }
    // running sum of g in 64 bits: differences of far larger sums stay exact
    if (w == 0) {
        double x[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int r = 2 * lane + i;
            x[i] = r < L ? (double)fmaxf(a.g[(t0 + r) * a.H + h], kMinG) : 0.0;
            sb[r] = r < L ? a.beta[(t0 + r) * a.H + h] : 0.f;
        }
        double s = x[0] + x[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        sG[2 * lane] = s - x[1];
        sG[2 * lane + 1] = s;
    }
    __syncthreads();
    if (tid < C) {
        float* gt = reinterpret_cast<float*>(gates + ch * kGateRow);
        gt[tid] = expf((float)sG[tid]);
        gt[C + tid] = expf((float)(sG[C - 1] - sG[tid]));
        gt[2 * C + tid] = sb[tid];
        reinterpret_cast<double*>(gt + 3 * C)[tid] = sG[tid];
    }

    // a warp takes 16 rows of both score matrices, columns up to the diagonal
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) kk[n][e] = qk[n][e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < DK / 16; s++) {
        uint32_t ak[4], aq[4];
        ldsm4(ak, at_k(sK, 16 * w, 2 * s, lane));
        ldsm4(aq, at_k(sQ, 16 * w, 2 * s, lane));
#pragma unroll
        for (int p = 0; p < 4; p++)
            if (p <= w) {
                uint32_t bk[4];
                ldsm4(bk, at_n(sK, 16 * p, 2 * s, lane));
                mma(kk[2 * p], ak, bk[0], bk[1]);
                mma(kk[2 * p + 1], ak, bk[2], bk[3]);
                mma(qk[2 * p], aq, bk[0], bk[1]);
                mma(qk[2 * p + 1], aq, bk[2], bk[3]);
            }
    }
    __syncthreads();  // the operands are done with
    uint8_t* sT = sm;  // T hi, T lo, P hi, P lo
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < 8; n++)
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int i = 16 * w + g + 8 * half, j = 8 * n + 2 * t;
            float av[2], pv[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const bool in = i >= j + e && i < L;  // columns behind the end lie above the diagonal of rows before it
                const float D = in ? expf((float)(sG[i] - sG[j + e])) : 0.f;
                pv[e] = in ? qk[n][2 * half + e] * D : 0.f;
                av[e] = in && i > j + e ? kk[n][2 * half + e] * D * sb[i] : 0.f;
            }
            *reinterpret_cast<float2*>(sA + i * C + j) = make_float2(av[0], av[1]);
            uint32_t hi, lo;
            split2(pv[0], pv[1], hi, lo);
            const uint32_t off = tile_at(0, i, n) + 4 * t;
            *reinterpret_cast<uint32_t*>(sT + 2 * kTile + off) = hi;
            *reinterpret_cast<uint32_t*>(sT + 3 * kTile + off) = lo;
        }
    __syncthreads();
    // Column j of T: x_i = [i = j] - sum_{m < i} A_im x_m.  Rows of A are read
    // by all threads at once (broadcast).
    if (tid < C) {
        float x[C];
#pragma unroll
        for (int i = 0; i < C; i++) {
            float s0 = tid == i ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 r = *reinterpret_cast<const float4*>(sA + i * C + m);
                s0 = fmaf(-r.x, x[m], s0);
                if (m + 1 < i) s1 = fmaf(-r.y, x[m + 1], s1);
                if (m + 2 < i) s2 = fmaf(-r.z, x[m + 2], s2);
                if (m + 3 < i) s3 = fmaf(-r.w, x[m + 3], s3);
            }
            x[i] = (s0 + s1) + (s2 + s3);
        }
#pragma unroll
        for (int i = 0; i < C; i++) {
            const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
            const __nv_bfloat16 lo = __float2bfloat16_rn(x[i] - __bfloat162float(hi));
            const uint32_t off = tile_at(0, i, tid >> 3) + 2 * (tid & 7);
            *reinterpret_cast<__nv_bfloat16*>(sT + off) = hi;
            *reinterpret_cast<__nv_bfloat16*>(sT + kTile + off) = lo;
        }
    }
    __syncthreads();
    uint4* dst = reinterpret_cast<uint4*>(tiles + ch * 4 * kTile);
    for (int i = tid; i < 4 * kTile / 16; i += kPrepThreads) dst[i] = reinterpret_cast<const uint4*>(sT)[i];
}

// --------------------------------------------------------------- the chain

constexpr int kWarps = 4;                            // 16 value columns each
constexpr int kChainThreads = (kWarps + 1) * 32;     // and the warp that loads

// What a pass writes: the output in bf16 or fp32, or (for the backward) the
// states before each chunk and the corrections.
enum : int { kOutBf16 = 0, kOutF32 = 1, kKeep = 2 };

template <int DK, int MODE>
struct Stage {
    static constexpr int K = C * DK * 2;
    static constexpr int Q = MODE == kKeep ? 0 : C * DK * 2;
    static constexpr int T = 2 * kTile;
    // a bf16 output needs no second term of P
    static constexpr int P = MODE == kKeep ? 0 : MODE == kOutF32 ? 2 * kTile : kTile;
    static constexpr int V = C * kSlice * 2;
    static constexpr int G = 1024;
    static constexpr int oQ = K, oT = K + Q, oP = oT + T, oV = oP + P, oG = oV + V;
    static constexpr int bytes = oG + G;
    static constexpr int loaded = K + Q + T + P + V + kGates;
    static constexpr int most = 225 * 1024;
    static constexpr int stages = most / bytes > 4 ? 4 : most / bytes;
    static constexpr int smem = stages * bytes + 1024 + 128;
};

struct ChainArgs {
    const uint8_t* tiles;
    const uint8_t* gates;
    const int* lengths;
    const float* initial_state;
    float* final_state;
    void* out;
    Kept kept;
    int N, nc, Hk, H, dv;
};

// The ring's barriers, behind its stages.
struct Ring {
    uint8_t* sm;
    uint64_t *full, *empty;
    __device__ __forceinline__ void init(int stages, int bytes) {
        extern __shared__ uint8_t raw[];
        sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
        full = reinterpret_cast<uint64_t*>(sm + stages * bytes);
        empty = full + stages;
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; i++) {
                tc::mbar_init(full + i, 1);
                tc::mbar_init(empty + i, kWarps);
            }
            tc::fence_barrier_init();
        }
        __syncthreads();
    }
};

template <int DK, int MODE>
__device__ __forceinline__ void chain_forward(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                              const ChainArgs& a, int b) {
    using St = Stage<DK, MODE>;
    constexpr int NS = St::stages;
    Ring ring;
    ring.init(NS, St::bytes);
    uint8_t* sm = ring.sm;
    uint64_t *full = ring.full, *empty = ring.empty;
    const int slice = blockIdx.x, h = blockIdx.y;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = length_of(a.lengths, b, a.N);
    const int n_chunks = (len + C - 1) / C;
    const size_t ch0 = ((size_t)b * a.H + h) * a.nc;

    if (w == kWarps) {  // loads
        if (lane != 0) return;
        const int hk = h / (a.H / a.Hk);
        for (int c = 0; c < n_chunks; c++) {
            const int st = c % NS;
            uint8_t* s = sm + st * St::bytes;
            if (c >= NS && !tc::mbar_wait(empty + st, ((c / NS) - 1) & 1)) {
                atomicExch(&g_delta_err, kErrTimeout);
                return;
            }
            tc::mbar_arrive_expect_tx(full + st, St::loaded);
#pragma unroll
            for (int i = 0; i < DK / 64; i++) tc::tma_load_4d(s + i * 8192, &mk, full + st, 64 * i, hk, c * C, b);
            const uint8_t* tl = a.tiles + (ch0 + c) * 4 * kTile;
            bulk_load(s + St::oT, tl, St::T, full + st);
            tc::tma_load_4d(s + St::oV, &mv, full + st, slice * kSlice, h, c * C, b);
            bulk_load(s + St::oG, a.gates + (ch0 + c) * kGateRow, kGates, full + st);
            if constexpr (MODE != kKeep) {
#pragma unroll
                for (int i = 0; i < DK / 64; i++)
                    tc::tma_load_4d(s + St::oQ + i * 8192, &mq, full + st, 64 * i, hk, c * C, b);
                bulk_load(s + St::oP, tl + 2 * kTile, St::P, full + st);
            }
        }
        return;
    }

    const int g = lane >> 2, t = lane & 3;
    const int col = slice * kSlice + 16 * w + g;  // this thread's columns: col and col + 8
    const size_t sb = ((size_t)b * a.H + h) * DK * a.dv;
    float S[DK / 8][4];
#pragma unroll
    for (int n = 0; n < DK / 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int r = 8 * n + 2 * t + (e & 1), cc = col + 8 * (e >> 1);
            S[n][e] = a.initial_state && cc < a.dv ? a.initial_state[sb + (size_t)r * a.dv + cc] : 0.f;
        }

    for (int c = 0; c < n_chunks; c++) {
        const int st = c % NS;
        if (!tc::mbar_wait(full + st, (c / NS) & 1)) {
            if (lane == 0) atomicExch(&g_delta_err, kErrTimeout);
            return;
        }
        uint8_t* s = sm + st * St::bytes;
        const uint32_t sK = tc::smem_u32(s), sQ = sK + St::oQ, sT = sK + St::oT, sP = sK + St::oP, sV = sK + St::oV;
        const float* gt = reinterpret_cast<const float*>(s + St::oG);
        const int L = min(C, len - c * C);
        if (L < C) {
            // rows behind the end may hold anything: every warp clears K's for
            // itself (all write the same zeros), V's are never selected
            clear_rows(s, L, DK / 8, lane);
            __syncwarp();
        }

        // X^T = S^T K^T
        float X[8][4];
#pragma unroll
        for (int n = 0; n < 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) X[n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DK / 16; kk++) {
            uint32_t hi[4], lo[4];
            split_a(S[2 * kk], S[2 * kk + 1], hi, lo);
            if constexpr (MODE == kKeep) {
                uint8_t* ks = a.kept.s + ((ch0 + c) * gridDim.x + slice) * (size_t)(4 * C * DK);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const uint32_t off = tile_at(0, 16 * w + g + 8 * (e & 1), 2 * kk + (e >> 1)) + 4 * t;
                    *reinterpret_cast<uint32_t*>(ks + off) = hi[e];
                    *reinterpret_cast<uint32_t*>(ks + 2 * C * DK + off) = lo[e];
                }
            }
#pragma unroll
            for (int p = 0; p < 4; p++) {
                uint32_t bk[4];
                ldsm4(bk, at_n(sK, 16 * p, 2 * kk, lane));
                mma(X[2 * p], hi, bk[0], bk[1]);
                mma(X[2 * p + 1], hi, bk[2], bk[3]);
                mma(X[2 * p], lo, bk[0], bk[1]);
                mma(X[2 * p + 1], lo, bk[2], bk[3]);
            }
        }

        // beta R^T, R = V - exp(G) X, split as the next product's A operand
        uint32_t rh[4][4], rl[4][4];
#pragma unroll
        for (int p = 0; p < 4; p++) {
            uint32_t v4[4];
            {
                const int m = lane >> 3, tok = 16 * p + 8 * (m >> 1) + (lane & 7);
                ldsm4_t(v4, tile_at(sV, tok, 2 * w + (m & 1)));
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int n = 2 * p + i, tok = 8 * n + 2 * t;
                const float2 eg = *reinterpret_cast<const float2*>(gt + tok);
                const float2 bt = *reinterpret_cast<const float2*>(gt + 2 * C + tok);
                const bool in0 = tok < L, in1 = tok + 1 < L;
                X[n][0] = in0 ? bt.x * (tc::bf16lo(v4[2 * i]) - eg.x * X[n][0]) : 0.f;
                X[n][1] = in1 ? bt.y * (tc::bf16hi(v4[2 * i]) - eg.y * X[n][1]) : 0.f;
                X[n][2] = in0 ? bt.x * (tc::bf16lo(v4[2 * i + 1]) - eg.x * X[n][2]) : 0.f;
                X[n][3] = in1 ? bt.y * (tc::bf16hi(v4[2 * i + 1]) - eg.y * X[n][3]) : 0.f;
            }
            split_a(X[2 * p], X[2 * p + 1], rh[p], rl[p]);
        }

        // U^T = (beta R)^T T^T; T is lower triangular: token i takes j <= i
        float U[8][4];
#pragma unroll
        for (int n = 0; n < 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) U[n][e] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int p = j; p < 4; p++) {
                uint32_t th[4], tl[4];
                ldsm4(th, at_n(sT, 16 * p, 2 * j, lane));
                ldsm4(tl, at_n(sT + kTile, 16 * p, 2 * j, lane));
                mma(U[2 * p], rh[j], th[0], th[1]);
                mma(U[2 * p + 1], rh[j], th[2], th[3]);
                mma(U[2 * p], rl[j], th[0], th[1]);
                mma(U[2 * p + 1], rl[j], th[2], th[3]);
                mma(U[2 * p], rh[j], tl[0], tl[1]);
                mma(U[2 * p + 1], rh[j], tl[2], tl[3]);
            }

        if constexpr (MODE == kKeep) {
            uint8_t* ku = a.kept.u + ((ch0 + c) * gridDim.x + slice) * (size_t)(2 * kTile);
#pragma unroll
            for (int n = 0; n < 8; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    uint32_t hi, lo;
                    split2(U[n][2 * e], U[n][2 * e + 1], hi, lo);
                    const uint32_t off = tile_at(0, 16 * w + g + 8 * e, n) + 4 * t;
                    *reinterpret_cast<uint32_t*>(ku + off) = hi;
                    *reinterpret_cast<uint32_t*>(ku + kTile + off) = lo;
                }
        } else {
            // O^T = exp(G) (S^T Q^T) + U^T P^T.  An output rounded to bf16
            // takes one bf16 term of S, U and P (each off by 2^-9 at most, as
            // the rounding of the output is); an fp32 one takes both.
            float O[8][4];
#pragma unroll
            for (int n = 0; n < 8; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) O[n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DK / 16; kk++) {
                uint32_t hi[4], lo[4];
                if constexpr (MODE == kOutF32) split_a(S[2 * kk], S[2 * kk + 1], hi, lo);
                else round_a(S[2 * kk], S[2 * kk + 1], hi);
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    uint32_t bq[4];
                    ldsm4(bq, at_n(sQ, 16 * p, 2 * kk, lane));
                    mma(O[2 * p], hi, bq[0], bq[1]);
                    mma(O[2 * p + 1], hi, bq[2], bq[3]);
                    if constexpr (MODE == kOutF32) {
                        mma(O[2 * p], lo, bq[0], bq[1]);
                        mma(O[2 * p + 1], lo, bq[2], bq[3]);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 8; n++) {
                const float2 eg = *reinterpret_cast<const float2*>(gt + 8 * n + 2 * t);
                O[n][0] *= eg.x;
                O[n][1] *= eg.y;
                O[n][2] *= eg.x;
                O[n][3] *= eg.y;
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t uh[4], ul[4];
                if constexpr (MODE == kOutF32) split_a(U[2 * j], U[2 * j + 1], uh, ul);
                else round_a(U[2 * j], U[2 * j + 1], uh);
#pragma unroll
                for (int p = j; p < 4; p++) {
                    uint32_t ph[4];
                    ldsm4(ph, at_n(sP, 16 * p, 2 * j, lane));
                    mma(O[2 * p], uh, ph[0], ph[1]);
                    mma(O[2 * p + 1], uh, ph[2], ph[3]);
                    if constexpr (MODE == kOutF32) {
                        uint32_t pl[4];
                        ldsm4(pl, at_n(sP + kTile, 16 * p, 2 * j, lane));
                        mma(O[2 * p], ul, ph[0], ph[1]);
                        mma(O[2 * p + 1], ul, ph[2], ph[3]);
                        mma(O[2 * p], uh, pl[0], pl[1]);
                        mma(O[2 * p + 1], uh, pl[2], pl[3]);
                    }
                }
            }
            const size_t row0 = (size_t)b * a.N + (size_t)c * C;
            if constexpr (MODE == kOutF32) {
                float* o = reinterpret_cast<float*>(a.out);
#pragma unroll
                for (int n = 0; n < 8; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int tok = 8 * n + 2 * t + (e & 1), cc = col + 8 * (e >> 1);
                        if (tok < L && cc < a.dv) o[((row0 + tok) * a.H + h) * a.dv + cc] = O[n][e];
                    }
            } else {
                // through this warp's columns of the V tile, which it has read
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    uint32_t r4[4];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        r4[2 * i] = tc::pack_bf16x2(O[2 * p + i][0], O[2 * p + i][1]);
                        r4[2 * i + 1] = tc::pack_bf16x2(O[2 * p + i][2], O[2 * p + i][3]);
                    }
                    const int m = lane >> 3, tok = 16 * p + 8 * (m >> 1) + (lane & 7);
                    stsm4_t(tile_at(sV, tok, 2 * w + (m & 1)), r4);
                }
                __syncwarp();
                __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.out);
                const int piece = lane & 1, c0 = slice * kSlice + 16 * w + 8 * piece;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int tok = 16 * i + (lane >> 1);
                    if (tok < L && c0 < a.dv)
                        *reinterpret_cast<uint4*>(o + ((row0 + tok) * a.H + h) * a.dv + c0) =
                            *reinterpret_cast<const uint4*>(s + St::oV + tile_at(0, tok, 2 * w + piece));
                }
            }
        }

        // S^T <- exp(G_C) S^T + (exp(G_C - G) U)^T K
        const float eC = gt[C - 1];
        uint32_t uh[4][4], ul[4][4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int n = 2 * j + i;
                const float2 e2 = *reinterpret_cast<const float2*>(gt + C + 8 * n + 2 * t);
                U[n][0] *= e2.x;
                U[n][1] *= e2.y;
                U[n][2] *= e2.x;
                U[n][3] *= e2.y;
            }
            split_a(U[2 * j], U[2 * j + 1], uh[j], ul[j]);
        }
#pragma unroll
        for (int d = 0; d < DK / 16; d += 2) {
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][e] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t b0[4], b1[4];
                ldsm4_t(b0, at_k(sK, 16 * j, 2 * d, lane));
                ldsm4_t(b1, at_k(sK, 16 * j, 2 * d + 2, lane));
                mma(acc[0], uh[j], b0[0], b0[1]);
                mma(acc[1], uh[j], b0[2], b0[3]);
                mma(acc[2], uh[j], b1[0], b1[1]);
                mma(acc[3], uh[j], b1[2], b1[3]);
                mma(acc[0], ul[j], b0[0], b0[1]);
                mma(acc[1], ul[j], b0[2], b0[3]);
                mma(acc[2], ul[j], b1[0], b1[1]);
                mma(acc[3], ul[j], b1[2], b1[3]);
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) S[2 * d + i][e] = fmaf(eC, S[2 * d + i][e], acc[i][e]);
        }
        // the stage goes back to the loads, which write it by another proxy
        __syncwarp();
        if (lane == 0) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(empty + st);
        }
    }
    if (a.final_state) {
#pragma unroll
        for (int n = 0; n < DK / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int r = 8 * n + 2 * t + (e & 1), cc = col + 8 * (e >> 1);
                if (cc < a.dv) a.final_state[sb + (size_t)r * a.dv + cc] = S[n][e];
            }
    }
}

// ------------------------------------------------------- the backward's chain
//
// With dS1 the gradient of the state after a chunk, and the same T, P:
//     dU = P^T dO + diag(exp(G_C - G)) K dS1,  dY = T^T dU,  dR = beta dY (= dV)
//     dS0 = exp(G_C) dS1 + (diag(exp(G)) Q)^T dO - (diag(exp(G)) K)^T dR,
// column by column as the forward, the chunks from the last to the first.

template <int DK>
struct BackStage {
    static constexpr int K = C * DK * 2, Q = K, T = 2 * kTile, P = 2 * kTile, O = C * kSlice * 2, G = 1024;
    static constexpr int oQ = K, oT = K + Q, oP = oT + T, oO = oP + P, oG = oO + O;
    static constexpr int bytes = oG + G;
    static constexpr int loaded = K + Q + T + P + O + kGates;
    static constexpr int stages = Stage<DK, kKeep>::most / bytes > 3 ? 3 : Stage<DK, kKeep>::most / bytes;
    static constexpr int smem = stages * bytes + 1024 + 128;
};

template <int DK>
__device__ __forceinline__ void chain_backward(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mo,
                                               const ChainArgs& a, const float* dfinal, float* dinitial, int b) {
    using St = BackStage<DK>;
    constexpr int NS = St::stages;
    Ring ring;
    ring.init(NS, St::bytes);
    uint8_t* sm = ring.sm;
    uint64_t *full = ring.full, *empty = ring.empty;
    const int slice = blockIdx.x, h = blockIdx.y;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = length_of(a.lengths, b, a.N);
    const int n_chunks = (len + C - 1) / C;
    const size_t ch0 = ((size_t)b * a.H + h) * a.nc;

    if (w == kWarps) {  // loads
        if (lane != 0) return;
        const int hk = h / (a.H / a.Hk);
        for (int it = 0; it < n_chunks; it++) {
            const int st = it % NS, c = n_chunks - 1 - it;
            uint8_t* s = sm + st * St::bytes;
            if (it >= NS && !tc::mbar_wait(empty + st, ((it / NS) - 1) & 1)) {
                atomicExch(&g_delta_err, kErrTimeout);
                return;
            }
            tc::mbar_arrive_expect_tx(full + st, St::loaded);
#pragma unroll
            for (int i = 0; i < DK / 64; i++) {
                tc::tma_load_4d(s + i * 8192, &mk, full + st, 64 * i, hk, c * C, b);
                tc::tma_load_4d(s + St::oQ + i * 8192, &mq, full + st, 64 * i, hk, c * C, b);
            }
            bulk_load(s + St::oT, a.tiles + (ch0 + c) * 4 * kTile, St::T + St::P, full + st);
            tc::tma_load_4d(s + St::oO, &mo, full + st, slice * kSlice, h, c * C, b);
            bulk_load(s + St::oG, a.gates + (ch0 + c) * kGateRow, kGates, full + st);
        }
        return;
    }

    const int g = lane >> 2, t = lane & 3;
    const int col = slice * kSlice + 16 * w + g;
    const size_t sb = ((size_t)b * a.H + h) * DK * a.dv;
    float S[DK / 8][4];
#pragma unroll
    for (int n = 0; n < DK / 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int r = 8 * n + 2 * t + (e & 1), cc = col + 8 * (e >> 1);
            S[n][e] = dfinal && cc < a.dv ? dfinal[sb + (size_t)r * a.dv + cc] : 0.f;
        }

    for (int it = 0; it < n_chunks; it++) {
        const int st = it % NS, c = n_chunks - 1 - it;
        if (!tc::mbar_wait(full + st, (it / NS) & 1)) {
            if (lane == 0) atomicExch(&g_delta_err, kErrTimeout);
            return;
        }
        uint8_t* s = sm + st * St::bytes;
        const uint32_t sK = tc::smem_u32(s), sQ = sK + St::oQ, sT = sK + St::oT, sP = sK + St::oP, sO = sK + St::oO;
        const float* gt = reinterpret_cast<const float*>(s + St::oG);
        const int L = min(C, len - c * C);
        if (L < C) {
            // the last chunk, the first one here: every warp clears what lies
            // behind the end for itself (all write the same zeros)
            clear_rows(s, L, DK / 8, lane);
            clear_rows(s + St::oQ, L, DK / 8, lane);
            clear_rows(s + St::oO, L, kSlice / 8, lane);
            __syncwarp();
        }

        // dU^T = (dS^T K^T) exp(G_C - G) + dO^T P
        float U[8][4];
#pragma unroll
        for (int n = 0; n < 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) U[n][e] = 0.f;
        uint8_t* ks = a.kept.ds + ((ch0 + c) * gridDim.x + slice) * (size_t)(4 * C * DK);
#pragma unroll
        for (int kk = 0; kk < DK / 16; kk++) {
            uint32_t hi[4], lo[4];
            split_a(S[2 * kk], S[2 * kk + 1], hi, lo);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t off = tile_at(0, 16 * w + g + 8 * (e & 1), 2 * kk + (e >> 1)) + 4 * t;
                *reinterpret_cast<uint32_t*>(ks + off) = hi[e];
                *reinterpret_cast<uint32_t*>(ks + 2 * C * DK + off) = lo[e];
            }
#pragma unroll
            for (int p = 0; p < 4; p++) {
                uint32_t bk[4];
                ldsm4(bk, at_n(sK, 16 * p, 2 * kk, lane));
                mma(U[2 * p], hi, bk[0], bk[1]);
                mma(U[2 * p + 1], hi, bk[2], bk[3]);
                mma(U[2 * p], lo, bk[0], bk[1]);
                mma(U[2 * p + 1], lo, bk[2], bk[3]);
            }
        }
#pragma unroll
        for (int n = 0; n < 8; n++) {
            const float2 e2 = *reinterpret_cast<const float2*>(gt + C + 8 * n + 2 * t);
            U[n][0] *= e2.x;
            U[n][1] *= e2.y;
            U[n][2] *= e2.x;
            U[n][3] *= e2.y;
        }
        uint32_t oh[4][4], ol[4][4];  // dO^T, later exp(G) dO^T in two terms
#pragma unroll
        for (int i = 0; i < 4; i++) {
            ldsm4_t(oh[i], at_n(sO, 16 * i, 2 * w, lane));
#pragma unroll
            for (int d = 0; d <= i; d++) {  // P is lower triangular: token j takes i >= j
                uint32_t ph[4], pl[4];
                ldsm4_t(ph, at_k(sP, 16 * i, 2 * d, lane));
                ldsm4_t(pl, at_k(sP + kTile, 16 * i, 2 * d, lane));
                mma(U[2 * d], oh[i], ph[0], ph[1]);
                mma(U[2 * d + 1], oh[i], ph[2], ph[3]);
                mma(U[2 * d], oh[i], pl[0], pl[1]);
                mma(U[2 * d + 1], oh[i], pl[2], pl[3]);
            }
        }

        // dY^T = dU^T T
        float Y[8][4];
#pragma unroll
        for (int n = 0; n < 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) Y[n][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t uh[4], ul[4];
            split_a(U[2 * i], U[2 * i + 1], uh, ul);
#pragma unroll
            for (int d = 0; d <= i; d++) {
                uint32_t th[4], tl[4];
                ldsm4_t(th, at_k(sT, 16 * i, 2 * d, lane));
                ldsm4_t(tl, at_k(sT + kTile, 16 * i, 2 * d, lane));
                mma(Y[2 * d], uh, th[0], th[1]);
                mma(Y[2 * d + 1], uh, th[2], th[3]);
                mma(Y[2 * d], ul, th[0], th[1]);
                mma(Y[2 * d + 1], ul, th[2], th[3]);
                mma(Y[2 * d], uh, tl[0], tl[1]);
                mma(Y[2 * d + 1], uh, tl[2], tl[3]);
            }
        }
        uint8_t* ky = a.kept.y + ((ch0 + c) * gridDim.x + slice) * (size_t)(2 * kTile);
#pragma unroll
        for (int n = 0; n < 8; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                uint32_t hi, lo;
                split2(Y[n][2 * e], Y[n][2 * e + 1], hi, lo);
                const uint32_t off = tile_at(0, 16 * w + g + 8 * e, n) + 4 * t;
                *reinterpret_cast<uint32_t*>(ky + off) = hi;
                *reinterpret_cast<uint32_t*>(ky + kTile + off) = lo;
            }

        // dS^T <- exp(G_C) dS^T + (exp(G) dO)^T Q - (exp(G) beta dY)^T K
        const float eC = gt[C - 1];
        uint32_t yh[4][4], yl[4][4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int n = 2 * i + j, tok = 8 * n + 2 * t;
                const float2 eg = *reinterpret_cast<const float2*>(gt + tok);
                const float2 bt = *reinterpret_cast<const float2*>(gt + 2 * C + tok);
                Y[n][0] *= -eg.x * bt.x;
                Y[n][1] *= -eg.y * bt.y;
                Y[n][2] *= -eg.x * bt.x;
                Y[n][3] *= -eg.y * bt.y;
#pragma unroll
                for (int r = 2 * j; r < 2 * j + 2; r++) {
                    const uint32_t x = oh[i][r];
                    split2(tc::bf16lo(x) * eg.x, tc::bf16hi(x) * eg.y, oh[i][r], ol[i][r]);
                }
            }
            split_a(Y[2 * i], Y[2 * i + 1], yh[i], yl[i]);
        }
#pragma unroll
        for (int d = 0; d < DK / 16; d++) {
            float acc[2][2][4];
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[0][i][e] = acc[1][i][e] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t bq[4], bk[4];
                ldsm4_t(bq, at_k(sQ, 16 * j, 2 * d, lane));
                ldsm4_t(bk, at_k(sK, 16 * j, 2 * d, lane));
                mma(acc[0][0], oh[j], bq[0], bq[1]);
                mma(acc[0][1], oh[j], bq[2], bq[3]);
                mma(acc[1][0], yh[j], bk[0], bk[1]);
                mma(acc[1][1], yh[j], bk[2], bk[3]);
                mma(acc[0][0], ol[j], bq[0], bq[1]);
                mma(acc[0][1], ol[j], bq[2], bq[3]);
                mma(acc[1][0], yl[j], bk[0], bk[1]);
                mma(acc[1][1], yl[j], bk[2], bk[3]);
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    S[2 * d + i][e] = fmaf(eC, S[2 * d + i][e], acc[0][i][e] + acc[1][i][e]);
        }
        __syncwarp();
        if (lane == 0) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(empty + st);
        }
    }
    if (dinitial) {
#pragma unroll
        for (int n = 0; n < DK / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int r = 8 * n + 2 * t + (e & 1), cc = col + 8 * (e >> 1);
                if (cc < a.dv) dinitial[sb + (size_t)r * a.dv + cc] = S[n][e];
            }
    }
}

// ------------------------------------------------------------------ kernels

template <int DK, int MODE>
__global__ void __launch_bounds__(kChainThreads, 1)
    k_delta_chain(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ ChainArgs a) {
    chain_forward<DK, MODE>(mq, mk, mv, a, blockIdx.z);
}

// The backward's two chains do not depend on each other: half of the blocks
// walk forward (states and corrections), half backward, side by side.
template <int DK>
__global__ void __launch_bounds__(kChainThreads, 1)
    k_delta_chains(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                   const __grid_constant__ ChainArgs a, const float* dfinal, float* dinitial) {
    if (blockIdx.z & 1) chain_forward<DK, kKeep>(mq, mk, mv, a, blockIdx.z >> 1);
    else chain_backward<DK>(mq, mk, mo, a, dfinal, dinitial, blockIdx.z >> 1);
}

template <int DK>
ret_status prep(const DeltaArgs& a, uint8_t* tiles, uint8_t* gates, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_delta_prep<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, prep_smem<DK>());
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule tables: %s", cudaGetErrorString(e));
    const int nc = chunks_of(a.N);
    k_delta_prep<DK><<<dim3(nc, a.H, a.B), kPrepThreads, prep_smem<DK>(), s>>>(a, tiles, gates, nc);
    return check_launch("delta rule: chunk tables");
}

template <int DK, int MODE>
ret_status chain(const DeltaArgs& a, ChainArgs c, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!chunk_map(&mq, a.q, a.B, a.N, a.Hk, DK) || !chunk_map(&mk, a.k, a.B, a.N, a.Hk, DK) ||
        !chunk_map(&mv, a.v, a.B, a.N, a.H, a.dv))
        return RET_ERR_CUDA;
    using St = Stage<DK, MODE>;
    cudaError_t e = cudaFuncSetAttribute(k_delta_chain<DK, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, St::smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule: %s", cudaGetErrorString(e));
    k_delta_chain<DK, MODE><<<dim3(slices_of(a.dv), a.H, a.B), kChainThreads, St::smem, s>>>(mq, mk, mv, c);
    return check_launch("delta rule: chain");
}

template <int MODE>
ret_status chain_dk(const DeltaArgs& a, const ChainArgs& c, cudaStream_t s) {
    return a.dk == 64 ? chain<64, MODE>(a, c, s) : a.dk == 128 ? chain<128, MODE>(a, c, s) : chain<256, MODE>(a, c, s);
}

ChainArgs chain_args(const DeltaArgs& a, const uint8_t* tiles, const uint8_t* gates) {
    ChainArgs c{};
    c.tiles = tiles;
    c.gates = gates;
    c.lengths = a.lengths;
    c.initial_state = a.initial_state;
    c.final_state = a.final_state;
    c.out = a.out;
    c.N = a.N;
    c.nc = chunks_of(a.N);
    c.Hk = a.Hk;
    c.H = a.H;
    c.dv = a.dv;
    return c;
}

}  // namespace

ret_status launch_prep(const DeltaArgs& a, uint8_t* tiles, uint8_t* gates, cudaStream_t s) {
    return a.dk == 64 ? prep<64>(a, tiles, gates, s) : a.dk == 128 ? prep<128>(a, tiles, gates, s) : prep<256>(a, tiles, gates, s);
}

template <int DK>
static ret_status chains(const DeltaArgs& a, const ChainArgs& c, cudaStream_t s) {
    CUtensorMap mq, mk, mv, mo;
    if (!chunk_map(&mq, a.q, a.B, a.N, a.Hk, DK) || !chunk_map(&mk, a.k, a.B, a.N, a.Hk, DK) ||
        !chunk_map(&mv, a.v, a.B, a.N, a.H, a.dv) || !chunk_map(&mo, a.dout, a.B, a.N, a.H, a.dv))
        return RET_ERR_CUDA;
    constexpr int smem = std::max(Stage<DK, kKeep>::smem, BackStage<DK>::smem);
    cudaError_t e = cudaFuncSetAttribute(k_delta_chains<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule: %s", cudaGetErrorString(e));
    k_delta_chains<DK><<<dim3(slices_of(a.dv), a.H, 2 * a.B), kChainThreads, smem, s>>>(mq, mk, mv, mo, c, a.dfinal_state,
                                                                                      a.dinitial_state);
    return check_launch("delta rule: the backward's chains");
}

ret_status launch_chains(const DeltaArgs& a, const uint8_t* tiles, const uint8_t* gates, const Kept& kept, cudaStream_t s) {
    ChainArgs c = chain_args(a, tiles, gates);
    c.final_state = nullptr;
    c.kept = kept;
    return a.dk == 64 ? chains<64>(a, c, s) : a.dk == 128 ? chains<128>(a, c, s) : chains<256>(a, c, s);
}

}  // namespace delta

using namespace delta;

bool delta_chunk_shape_ok(const DeltaArgs& a) {
    return a.in_dt == RET_BF16 && (a.dk == 64 || a.dk == 128 || a.dk == 256) && a.dv % 8 == 0;
}

size_t delta_forward_ws_bytes(const DeltaArgs& a) {
    return (size_t)a.B * a.H * chunks_of(a.N) * (4 * kTile + kGateRow);
}

ret_status launch_delta_forward(const DeltaArgs& a, void* ws, cudaStream_t s) {
    const size_t n = (size_t)a.B * a.H * chunks_of(a.N);
    uint8_t* tiles = reinterpret_cast<uint8_t*>(ws);
    uint8_t* gates = tiles + n * 4 * kTile;
    ret_status st = launch_prep(a, tiles, gates, s);
    if (st != RET_OK) return st;
    const ChainArgs c = chain_args(a, tiles, gates);
    return a.out_dt == RET_F32 ? chain_dk<kOutF32>(a, c, s) : chain_dk<kOutBf16>(a, c, s);
}

}  // namespace ret
