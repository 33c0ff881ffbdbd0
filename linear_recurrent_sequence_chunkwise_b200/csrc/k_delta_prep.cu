// k_delta_prep.cu -- the chunk tables of the gated delta rule (notation and
// number format: delta_util.cuh): scaled keys and queries in fp16, the gates,
// T = (I + diag(beta) M)^-1 and P, one block per (chunk, value head).
//
// Scores: K' K'^T by four warps and Q' K'^T by four more, 16 rows each and the
// columns up to the diagonal; a short row group of one shares an SM
// sub-partition with a long one of the other.  T by blocks of 16: the diagonal
// blocks by substitution (a thread per column, in registers), the others
// column by column of blocks, T_ij = -T_ii sum_{j <= m < i} A_im T_mj, on the
// tensor cores, a warp per block column.
//
// Bound by instruction issue and the barriers between its short phases: 1 x 8192,
// 16 heads of 256: 122 us for 2,048 chunks and heads; 4 x 2047 (1,472 chunks and
// heads of 128): 50 us with four blocks an SM, a fifth more with three.
#include "delta_util.cuh"

namespace ret {
namespace delta {

namespace {

constexpr int kThreads = 256;
constexpr int kDiag = 272;  // floats of a 16 x 16 diagonal block, off the next one's banks

template <int DK>
struct Smem {
    static constexpr int operands = 2 * C * DK * 2;
    static constexpr int tiles = 6 * kTile;  // T hi, T lo, P hi, P lo, A hi, A lo in the operands' place
    static constexpr int bytes = (operands > tiles ? operands : tiles) + 4 * kDiag * 4;
    static constexpr int diag = bytes - 4 * kDiag * 4;
};

// Exponent e that brings the largest element of a row spread over `width`
// lanes, eight values each, into [1, 2) (0 for a zero or non-finite row;
// `none`: a zero row).
template <int WIDTH>
__device__ __forceinline__ int row_exponent(const float (&x)[8], bool& none) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    none = m == 0.f;
    const int e = (__float_as_int(m) >> 23) & 255;
    return none || e == 255 ? 0 : min(max(e - 127, -60), 60);
}

template <int DK>
__global__ void __launch_bounds__(kThreads, DK == 256 ? 3 : 4) k_delta_prep(DeltaArgs a, Tables tb, int nc) {
    using Sm = Smem<DK>;
    launch_next();
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ double sG[C];
    // Decays between blocks of 16 rows, about row i's block's first row i0:
    // D_ij = exp(G_i - G_i0) exp(G_i0 - G_j) = row[i] col[i / 16][j], both at most
    // one.  With an exponential of a 64-bit difference for each element, and rows
    // scaled by their norms instead of their largest elements, the kernel took 137
    // us instead of 122 (dk 256, 128 chunks of 16 heads).
    __shared__ __align__(8) float row[C], col[4][C];
    __shared__ float sb[C], sk[C], sq[C];
    float* diag = reinterpret_cast<float*>(sm + Sm::diag);
    const int c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int L = min(C, length_of(a.lengths, b, a.N) - c * C);
    if (L <= 0) return;
    const int rep = a.H / a.Hk, hk = h / rep;
    const size_t ch = ((size_t)b * a.H + h) * nc + c;
    const size_t t0 = (size_t)b * a.N + (size_t)c * C;

    // running sum of g in 64 bits: differences of far larger sums stay exact
    if (w == 0) {
        double x[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int r = 2 * lane + i;
            const float gr = r < L ? a.g[(t0 + r) * a.H + h] : 0.f;
            x[i] = gr < kMinG ? kMinG : gr;  // a NaN stays one
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
    // K' and Q': rows scaled by powers of two, in fp16, zeros behind the end
    constexpr int kPieces = DK / 8;
    uint8_t* keys = h % rep == 0 ? tb.keys + (((size_t)b * a.Hk + hk) * nc + c) * (4 * C * DK) : nullptr;
    for (int i = tid; i < 2 * C * kPieces; i += kThreads) {
        const int which = i / (C * kPieces), r = (i / kPieces) % C, p = i % kPieces;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = 0.f;
        if (r < L) {
            const __nv_bfloat16* src = (const __nv_bfloat16*)(which ? a.q : a.k);
            const uint4 u = *reinterpret_cast<const uint4*>(src + ((t0 + r) * a.Hk + hk) * DK + 8 * p);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                x[2 * e] = tc::bf16lo(v[e]);
                x[2 * e + 1] = tc::bf16hi(v[e]);
            }
        }
        bool none;
        const int ex = row_exponent<kPieces>(x, none);
        const float inv = __int_as_float((127 - ex) << 23);
        uint4 o;
        o.x = pack_h2(x[0] * inv, x[1] * inv);
        o.y = pack_h2(x[2] * inv, x[3] * inv);
        o.z = pack_h2(x[4] * inv, x[5] * inv);
        o.w = pack_h2(x[6] * inv, x[7] * inv);
        const uint32_t off = which * 2 * C * DK + tile_at(r, p);
        *reinterpret_cast<uint4*>(sm + off) = o;
        if (keys) *reinterpret_cast<uint4*>(keys + off) = o;
        if (p == 0) (which ? sq : sk)[r] = none && !which ? 0.f : __int_as_float((127 + ex) << 23);
    }
    __syncthreads();
    if (tid < C) {
        // A zero key takes any scale: one that brings beta v, which such a token
        // has for its u, near v (beta |k|^2 sets no bound on beta there).
        float s = sk[tid];
        if (s == 0.f) s = __int_as_float((127 - min(max((__float_as_int(sb[tid]) >> 23 & 255) - 127, 0), 60)) << 23);
        const float bh = sb[tid] * s * s;
        float* gt = reinterpret_cast<float*>(tb.gates + ch * kGateRow);
        gt[gEG + tid] = expf((float)sG[tid]);
        gt[gEC + tid] = expf((float)(sG[C - 1] - sG[tid]));
        gt[gBeta + tid] = bh;
        gt[gIk + tid] = 1.f / s;
        gt[gSq + tid] = sq[tid];
        reinterpret_cast<double*>(gt + kGates / 4)[tid] = sG[tid];
        sb[tid] = bh;  // read by others after the next barrier
        const float m = warp_max(fabsf(bh));
        if (lane == 0) gt[gMax + w] = m;
    }

    {
        const int rb = tid >> 6, j = tid & 63;
        if (j < 16 * rb) col[rb][j] = expf((float)(sG[16 * rb] - sG[j]));
        if (rb == 0) row[j] = expf((float)(sG[j] - sG[j & 48]));
    }
    // scores
    const uint32_t sKs = tc::smem_u32(sm), sQs = sKs + 2 * C * DK;
    const bool isq = w >= 4;
    const int rg = isq ? 7 - w : w;
    float acc[8][4];
#pragma unroll
    for (int n = 0; n < 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[n][e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < DK / 16; s++) {
        uint32_t am[4];
        ldsm4(am, at_k(isq ? sQs : sKs, 16 * rg, 2 * s, lane));
#pragma unroll
        for (int p = 0; p < 4; p++)
            if (p <= rg) {
                uint32_t bk[4];
                ldsm4(bk, at_n(sKs, 16 * p, 2 * s, lane));
                mma(acc[2 * p], am, bk[0], bk[1]);
                mma(acc[2 * p + 1], am, bk[2], bk[3]);
            }
    }
    __syncthreads();  // the operands are done with
    uint8_t *sT = sm, *sP = sm + 2 * kTile, *sA = sm + 4 * kTile;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < 8; n++) {
        if (n / 2 > rg) continue;
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int i = 16 * rg + g + 8 * half, j = 8 * n + 2 * t;
            const float f = i >= L ? 0.f : isq ? 1.f : sb[i];
            float2 D;  // columns behind the end lie above the diagonal of the rows before it
            if (n / 2 < rg) {
                const float2 cj = *reinterpret_cast<const float2*>(&col[rg][j]);
                const float r = row[i] * f;
                D = make_float2(r * cj.x, r * cj.y);
            } else {
                D.x = (isq ? i >= j : i > j) ? f * expf((float)(sG[i] - sG[j])) : 0.f;
                D.y = (isq ? i > j : i > j + 1) ? f * expf((float)(sG[i] - sG[j + 1])) : 0.f;
            }
            // a score may be NaN or infinite where the factor is zero
            const float v0 = D.x != 0.f ? acc[n][2 * half] * D.x : 0.f, v1 = D.y != 0.f ? acc[n][2 * half + 1] * D.y : 0.f;
            uint32_t hi, lo;
            split2(v0, v1, hi, lo);
            const uint32_t off = tile_at(i, n) + 4 * t;
            uint8_t* dst = isq ? sP : sA;
            *reinterpret_cast<uint32_t*>(dst + off) = hi;
            *reinterpret_cast<uint32_t*>(dst + kTile + off) = lo;
            if (!isq && n / 2 == rg)
                *reinterpret_cast<float2*>(diag + rg * kDiag + (g + 8 * half) * 16 + (j & 15)) = make_float2(v0, v1);
        }
    }
    __syncthreads();
    uint4* dst = reinterpret_cast<uint4*>(tb.tiles + ch * 4 * kTile);
    if (tid < C) {
        // column j of a diagonal block: x_i = [i = j] - sum_{m < i} A_im x_m
        const int bl = tid >> 4, j = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
            float s0 = j == i ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 r = *reinterpret_cast<const float4*>(diag + bl * kDiag + i * 16 + m);
                s0 = fmaf(-r.x, x[m], s0);
                if (m + 1 < i) s1 = fmaf(-r.y, x[m + 1], s1);
                if (m + 2 < i) s0 = fmaf(-r.z, x[m + 2], s0);
                if (m + 3 < i) s1 = fmaf(-r.w, x[m + 3], s1);
            }
            x[i] = s0 + s1;
        }
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const __half hi = __float2half_rn(x[i]);
            const uint32_t off = tile_at(16 * bl + i, 2 * bl + (j >> 3)) + 2 * (j & 7);
            *reinterpret_cast<__half*>(sT + off) = hi;
            *reinterpret_cast<__half*>(sT + kTile + off) = __float2half_rn(x[i] - __half2float(hi));
        }
    } else if (w >= 4) {
        for (int i = tid - 128; i < 2 * kTile / 16; i += 128)
            dst[2 * kTile / 16 + i] = reinterpret_cast<const uint4*>(sP)[i];
    }
    __syncthreads();
    if (w < 3) {
        const int j = w;  // block column
        const uint32_t uT = sKs, uA = sKs + 4 * kTile;
        for (int i = j + 1; i < 4; i++) {
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) s[n][e] = 0.f;
            for (int m = j; m < i; m++) {
                uint32_t ah[4], al[4], bh[4], bl[4];
                ldsm4(ah, at_k(uA, 16 * i, 2 * m, lane));
                ldsm4(al, at_k(uA + kTile, 16 * i, 2 * m, lane));
                ldsm4_t(bh, at_k(uT, 16 * m, 2 * j, lane));
                ldsm4_t(bl, at_k(uT + kTile, 16 * m, 2 * j, lane));
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    mma(s[n], ah, bh[2 * n], bh[2 * n + 1]);
                    mma(s[n], al, bh[2 * n], bh[2 * n + 1]);
                    mma(s[n], ah, bl[2 * n], bl[2 * n + 1]);
                }
            }
            // the sum as a B operand: transpose its 8 x 8 blocks
            uint32_t xh[2][2], xl[2][2], th[4], tl[4];
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    uint32_t hi, lo;
                    split2(-s[n][2 * e], -s[n][2 * e + 1], hi, lo);
                    xh[n][e] = transpose8(hi);
                    xl[n][e] = transpose8(lo);
                }
            ldsm4(th, at_k(uT, 16 * i, 2 * i, lane));
            ldsm4(tl, at_k(uT + kTile, 16 * i, 2 * i, lane));
#pragma unroll
            for (int n = 0; n < 2; n++) {
                float y[4] = {0.f, 0.f, 0.f, 0.f};
                mma(y, th, xh[n][0], xh[n][1]);
                mma(y, tl, xh[n][0], xh[n][1]);
                mma(y, th, xl[n][0], xl[n][1]);
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    uint32_t hi, lo;
                    split2(y[2 * e], y[2 * e + 1], hi, lo);
                    const uint32_t off = tile_at(16 * i + g + 8 * e, 2 * j + n) + 4 * t;
                    *reinterpret_cast<uint32_t*>(sT + off) = hi;
                    *reinterpret_cast<uint32_t*>(sT + kTile + off) = lo;
                }
            }
            __syncwarp();
        }
    }
    __syncthreads();
    for (int i = tid; i < 2 * kTile / 16; i += kThreads) dst[i] = reinterpret_cast<const uint4*>(sT)[i];
}

template <int DK>
ret_status prep(const DeltaArgs& a, const Tables& t, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_delta_prep<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<DK>::bytes);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule tables: %s", cudaGetErrorString(e));
    const int nc = chunks_of(a.N);
    k_delta_prep<DK><<<dim3(nc, a.H, a.B), kThreads, Smem<DK>::bytes, s>>>(a, t, nc);
    return check_launch("delta rule: chunk tables");
}

}  // namespace

ret_status launch_prep(const DeltaArgs& a, const Tables& t, cudaStream_t s) {
    return a.dk == 64 ? prep<64>(a, t, s) : a.dk == 128 ? prep<128>(a, t, s) : prep<256>(a, t, s);
}

}  // namespace delta
}  // namespace ret
