// k_delta_chunk.cu -- the recurrence of the gated delta rule over the chunks of
// a sequence, forward and backward (notation and number format:
// delta_util.cuh; the tables come from k_delta_prep.cu).
//
// What bounds it is the chain: chunk c + 1 needs the state of chunk c, and a
// (sequence, head) has only its value columns to share out, which do not
// depend on each other.  Sixteen columns are the work of two warps.
// The first, the chain warp, carries them through the recurrence without a
// barrier: it holds the transposed state [16 x dk] as fp32 accumulator tiles,
// whose layout is that of the A operand of the next product (X^T = S^T K^T,
// U^T = R^T T^T, S^T += U^T K), so nothing it computes leaves its registers on
// the way.  Everything that the recurrence does not wait for is its helper's,
// on the same SM sub-partition, which fills the tensor pipe while the chain
// warp converts: the outputs (Q S and P U), or in the backward pass the terms
// of dO and the records.  The two hand over operand tiles through shared memory.
// The products run as mma.sync, not tcgen05: every operand is split into two
// fp16 terms between two products, in registers at once, where TMEM would cost
// a trip out and back for each of the four products of a chunk.
// K', Q', T, P come by bulk copies into a ring of stages, issued by a helper.
//
// %FIG%
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

// What a pass writes: the output in bf16 or fp32, or (for the backward) the
// states before each chunk and the corrections; and the backward's own chain.
enum : int { kOutBf16 = 0, kOutF32 = 1, kKeep = 2, kBack = 3 };

// Shared memory of a block of CG groups of 16 columns.
template <int DK, int CG, int MODE>
struct Plan {
    static constexpr int warps = 2 * CG;
    // a stage: K' (then Q'), T (then P), the gates
    static constexpr int keys = 2 * C * DK * (MODE == kKeep ? 1 : 2);
    static constexpr int tiles = MODE == kKeep ? 2 * kTile : MODE == kOutBf16 ? 3 * kTile : 4 * kTile;
    static constexpr int oT = keys, oGate = keys + tiles, stage = oGate + 2048;
    static constexpr uint32_t loaded = keys + tiles + kGates;
    // a group's: S in one or two terms, U (Y) the same way, staging of 64 x 16
    // bf16; the backward: Z in fp32, dU0 in fp32
    static constexpr int terms = MODE == kOutBf16 ? 1 : 2;
    static constexpr int sHalf = DK / 16 * 512, oU = terms * sHalf, uHalf = 4 * 512, oV = oU + terms * uHalf;
    static constexpr int oZ = oV + 2048, oD = oZ + (MODE == kBack ? DK * 64 : 0);
    static constexpr int group = oD + (MODE == kBack ? 4096 : 0);
    static constexpr int most = 226 * 1024 - 1024 - 512;
    static constexpr int fit = (most - CG * group) / stage;
    static constexpr int NS = fit > 3 ? 3 : fit;
    static_assert(NS >= 1, "tiles and exchange buffers exceed shared memory");
    static constexpr int oG = NS * stage, oBar = oG + CG * group;
    static constexpr int smem = oBar + 512 + 1024;
};

struct ChainArgs {
    Tables tb;
    const int* lengths;
    const float* initial_state;
    float* final_state;
    const __nv_bfloat16 *v, *dout;
    void* out;
    uint8_t* records;
    int N, nc, Hk, H, dv;
};

// Waits that give up: the error word is set, and the later waits of the warp
// are skipped, so that it comes to its end (with wrong results) soon.
struct Waits {
    bool ok = true;
    __device__ __forceinline__ void operator()(uint64_t* bar, int phase) {
        if (ok && !tc::mbar_wait(bar, phase & 1)) {
            ok = false;
            atomicExch(&g_delta_err, kErrTimeout);
        }
    }
};
__device__ __forceinline__ void signal(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}

// The block's shared memory and barriers: the stages', and for each group a
// pair (ready, free) for the tiles of S, those of U and the helper's fp32 terms.
struct Shared {
    uint8_t* sm;
    uint64_t *full, *empty, *s_ready, *s_free, *u_ready, *u_free, *z_ready, *z_free;
    float *s_inv, *u_inv;
    template <typename Pl, int CG>
    __device__ __forceinline__ void init() {
        extern __shared__ uint8_t raw[];
        sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
        full = reinterpret_cast<uint64_t*>(sm + Pl::oBar);
        empty = full + 3, s_ready = empty + 3, s_free = s_ready + 4, u_ready = s_free + 4, u_free = u_ready + 4;
        z_ready = u_free + 4, z_free = z_ready + 4;
        s_inv = reinterpret_cast<float*>(z_free + 4);
        u_inv = s_inv + 4;
        if (threadIdx.x == 0) {
            for (int i = 0; i < Pl::NS; i++) {
                tc::mbar_init(full + i, 1);
                tc::mbar_init(empty + i, Pl::warps);
            }
            for (int i = 0; i < CG; i++)
                for (uint64_t* b : {s_ready, s_free, u_ready, u_free, z_ready, z_free}) tc::mbar_init(b + i, 1);
            tc::fence_barrier_init();
        }
        __syncthreads();
    }
};

// One lane: chunk c of the sequence into its stage.
template <typename Pl, int DK>
__device__ __forceinline__ void load_stage(const Shared& r, const ChainArgs& a, size_t key_chunk, size_t chunk, int it,
                                           Waits& wait) {
    if (it >= Pl::NS) wait(r.empty + it % Pl::NS, it / Pl::NS - 1);
    if (!wait.ok) return;
    uint8_t* s = r.sm + (it % Pl::NS) * Pl::stage;
    uint64_t* bar = r.full + it % Pl::NS;
    tc::mbar_arrive_expect_tx(bar, Pl::loaded);
    bulk_load(s, a.tb.keys + key_chunk * (4 * C * DK), Pl::keys, bar);
    bulk_load(s + Pl::oGate, a.tb.gates + chunk * kGateRow, kGates, bar);
    bulk_load(s + Pl::oT, a.tb.tiles + chunk * 4 * kTile, Pl::tiles, bar);
}

__device__ __forceinline__ void put4(uint8_t* p, const uint32_t (&r)[4], int lane) {
    *reinterpret_cast<uint4*>(p + 16 * lane) = make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void get4(const uint8_t* p, uint32_t (&r)[4], int lane) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + 16 * lane);
    r[0] = u.x, r[1] = u.y, r[2] = u.z, r[3] = u.w;
}

// The scale of a warp's tiles.
template <int N>
__device__ __forceinline__ float tiles_scale(const float (&S)[N][4], float& inverse) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) m[e] = fmaxf(m[e], fabsf(S[n][e]));
    return scale_for(warp_max(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]))), inverse);
}
template <int N>
__device__ __forceinline__ void zero(float (&x)[N][4]) {
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) x[n][e] = 0.f;
}
// Columns (tokens) of tiles n = 0..7 times the token's factor.
__device__ __forceinline__ void scale_tokens(float (&x)[8][4], const float* f, float by, int t) {
#pragma unroll
    for (int n = 0; n < 8; n++) {
        float2 y = *reinterpret_cast<const float2*>(f + 8 * n + 2 * t);
        y.x *= by, y.y *= by;
        x[n][0] *= y.x, x[n][1] *= y.y, x[n][2] *= y.x, x[n][3] *= y.y;
    }
}
// The state's tile r = 8 n + 2 t + (e & 1), column g + 8 (e >> 1), from or to [dk, dv].
template <int N>
__device__ __forceinline__ void read_state(float (&S)[N][4], const float* p, int dv, int col, int t) {
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int cc = col + 8 * (e >> 1);
            S[n][e] = p && cc < dv ? p[(size_t)(8 * n + 2 * t + (e & 1)) * dv + cc] : 0.f;
        }
}
template <int N>
__device__ __forceinline__ void write_state(const float (&S)[N][4], float* p, int dv, int col, int t) {
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int cc = col + 8 * (e >> 1);
            if (cc < dv) p[(size_t)(8 * n + 2 * t + (e & 1)) * dv + cc] = S[n][e];
        }
}

// [16 x 16] bf16 (16 tokens, 16 columns) of a [B, N, H, dv] tensor, a 16-byte
// piece a lane.  A chunk ahead the address is clamped and nothing looks at the
// value (a branch or a select there would wait for the load); where it is used,
// what lies behind the sequence's end and behind dv becomes zero.
struct Rows {
    const __nv_bfloat16* p;  // of the (sequence, head), at this lane's columns
    size_t pitch;
    int len;
    bool cols;
    __device__ __forceinline__ uint4 load(int token) const {
        return *reinterpret_cast<const uint4*>(p + (size_t)min(token, len - 1) * pitch);
    }
    __device__ __forceinline__ uint4 use(uint4 x, int token) const {
        if (token >= len || !cols) x = make_uint4(0, 0, 0, 0);
        return x;
    }
};
__device__ __forceinline__ Rows rows_at(const __nv_bfloat16* t, const ChainArgs& a, int b, int h, int col, int len) {
    return Rows{t + ((size_t)b * a.N * a.H + h) * a.dv + min(col, a.dv - 8), (size_t)a.H * a.dv, len, col < a.dv};
}
// Such a piece, through 512 bytes of shared memory, as the transposed tiles
// (a row per column): e[0], e[1] tokens 0-7 of columns 0-7 and 8-15, e[2],
// e[3] tokens 8-15.
__device__ __forceinline__ void transpose16(uint8_t* slot, const uint4& x, int lane, uint32_t (&e)[4]) {
    *reinterpret_cast<uint4*>(slot + 16 * lane) = x;
    __syncwarp();
    const int m = lane >> 3, tok = 8 * (m >> 1) + (lane & 7);
    ldsm4_t(e, tc::smem_u32(slot) + tok * 32 + (m & 1) * 16);
}

// An operand tile of 16 columns of a record's [16][64 rows of 128 swizzled
// bytes], or of its [16][dk] in slabs of 64.
__device__ __forceinline__ void keep_tile(uint8_t* rec, int piece, int lane, const uint32_t (&r)[4]) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; e++)
        *reinterpret_cast<uint32_t*>(rec + tile_at<16>(g + 8 * (e & 1), piece + (e >> 1)) + 4 * t) = r[e];
}

template <int DK, int CG, int MODE>
__device__ __forceinline__ void chain_forward(const ChainArgs& a, int b) {
    using Pl = Plan<DK, CG, MODE>;
    constexpr int NS = Pl::NS, KK = DK / 16;
    Shared sh;
    sh.init<Pl, CG>();
    const int h = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = length_of(a.lengths, b, a.N), n_chunks = (len + C - 1) / C;
    const size_t ch0 = ((size_t)b * a.H + h) * a.nc;
    const int cg = w % CG, g = lane >> 2, t = lane & 3;
    const int group = blockIdx.x * CG + cg, col0 = group * 16;
    uint8_t* ex = sh.sm + Pl::oG + cg * Pl::group;
    uint8_t *sf = ex, *uf = ex + Pl::oU, *slot = ex + Pl::oV;
    Waits wait;

    if (w < CG) {  // the chain
        const size_t sb = ((size_t)b * a.H + h) * DK * a.dv;
        float S[DK / 8][4];
        read_state(S, a.initial_state ? a.initial_state + sb : nullptr, a.dv, col0 + g, t);
        const Rows vrows = rows_at(a.v, a, b, h, col0 + 8 * (lane & 1), len);
        uint4 vn[4];
        if (n_chunks)
#pragma unroll
            for (int i = 0; i < 4; i++) vn[i] = vrows.load(16 * i + (lane >> 1));
        for (int c = 0; c < n_chunks; c++) {
            uint8_t* st = sh.sm + (c % NS) * Pl::stage;
            const uint32_t sK = tc::smem_u32(st), sT = sK + Pl::oT;
            const float* gt = reinterpret_cast<const float*>(st + Pl::oGate);
#pragma unroll
            for (int i = 0; i < 4; i++)
                *reinterpret_cast<uint4*>(slot + 512 * i + 16 * lane) = vrows.use(vn[i], c * C + 16 * i + (lane >> 1));
#pragma unroll
            for (int i = 0; i < 4; i++) vn[i] = vrows.load((c + 1) * C + 16 * i + (lane >> 1));

            // X^T = S^T K^T; the helper gets the operand tiles
            float inv;
            const float ss = tiles_scale(S, inv);
            const float si = inv;
            float X[8][4];
            zero(X);
            wait(sh.full + c % NS, c / NS);
            if (c > 0) wait(sh.s_free + cg, c - 1);
#pragma unroll
            for (int kk = 0; kk < KK; kk++) {
                uint32_t hi[4], lo[4];
                split_a(S[2 * kk], S[2 * kk + 1], ss, hi, lo);
                put4(sf + kk * 512, hi, lane);
                if constexpr (Pl::terms == 2) put4(sf + Pl::sHalf + kk * 512, lo, lane);
                uint32_t bk[4][4];
#pragma unroll
                for (int p = 0; p < 4; p++) ldsm4(bk[p], at_n(sK, 16 * p, 2 * kk, lane));
                mma_row<0, 4>(X, hi, bk);
                mma_row<0, 4>(X, lo, bk);
            }
            if (lane == 0) sh.s_inv[cg] = si;
            signal(sh.s_ready + cg, lane);

            // R^T = beta' (V' - exp(G) X)
#pragma unroll
            for (int p = 0; p < 4; p++) {
                uint32_t v4[4];
                const int m = lane >> 3, tok = 8 * (m >> 1) + (lane & 7);
                ldsm4_t(v4, tc::smem_u32(slot) + 512 * p + tok * 32 + (m & 1) * 16);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int n = 2 * p + i, at = 8 * n + 2 * t;
                    float2 eg = *reinterpret_cast<const float2*>(gt + gEG + at);
                    const float2 bt = *reinterpret_cast<const float2*>(gt + gBeta + at);
                    const float2 ik = *reinterpret_cast<const float2*>(gt + gIk + at);
                    eg.x *= -si, eg.y *= -si;
                    X[n][0] = bt.x * fmaf(eg.x, X[n][0], tc::bf16lo(v4[2 * i]) * ik.x);
                    X[n][1] = bt.y * fmaf(eg.y, X[n][1], tc::bf16hi(v4[2 * i]) * ik.y);
                    X[n][2] = bt.x * fmaf(eg.x, X[n][2], tc::bf16lo(v4[2 * i + 1]) * ik.x);
                    X[n][3] = bt.y * fmaf(eg.y, X[n][3], tc::bf16hi(v4[2 * i + 1]) * ik.y);
                }
            }
            const float rs = tiles_scale(X, inv);
            const float ri = inv;

            // U^T = R^T T^T; T is lower triangular: token i takes j <= i
            float U[8][4];
            zero(U);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t rh[4], rl[4];
                split_a(X[2 * j], X[2 * j + 1], rs, rh, rl);
                uint32_t th[4][4], tl[4][4];
#pragma unroll
                for (int p = j; p < 4; p++) {
                    ldsm4(th[p], at_n(sT, 16 * p, 2 * j, lane));
                    ldsm4(tl[p], at_n(sT + kTile, 16 * p, 2 * j, lane));
                }
#pragma unroll
                for (int k = 0; k < 3; k++)
#pragma unroll
                    for (int p = j; p < 4; p++) {
                        const uint32_t(&b)[4] = k == 2 ? tl[p] : th[p];
                        mma(U[2 * p], k == 1 ? rl : rh, b[0], b[1]);
                        mma(U[2 * p + 1], k == 1 ? rl : rh, b[2], b[3]);
                    }
            }
            float ui = 0.f;
            const float us = tiles_scale(U, ui);  // of ri-scaled values: U is still times rs
            ui *= ri;
            if (c > 0) wait(sh.u_free + cg, c - 1);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t uh[4], ul[4];
                split_a(U[2 * j], U[2 * j + 1], us, uh, ul);
                put4(uf + j * 512, uh, lane);
                if constexpr (Pl::terms == 2) put4(uf + Pl::uHalf + j * 512, ul, lane);
            }
            if (lane == 0) sh.u_inv[cg] = ui;
            signal(sh.u_ready + cg, lane);

            // S^T <- exp(G_C) S^T + (exp(G_C - G) U)^T K
            const float eC = gt[gEG + C - 1];
            scale_tokens(U, gt + gEC, us, t);
            uint32_t uh[4][4], ul[4][4];
#pragma unroll
            for (int j = 0; j < 4; j++) split_a(U[2 * j], U[2 * j + 1], 1.f, uh[j], ul[j]);
#pragma unroll
            for (int d = 0; d < KK; d += 4) {
                float acc[8][4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t b[4][4];
#pragma unroll
                    for (int i = 0; i < 4; i++) ldsm4_t(b[i], at_k(sK, 16 * j, 2 * (d + i), lane));
                    if (j == 0) {
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            mma0(acc[2 * i], uh[j], b[i][0], b[i][1]);
                            mma0(acc[2 * i + 1], uh[j], b[i][2], b[i][3]);
                        }
                    } else {
                        mma_row<0, 4>(acc, uh[j], b);
                    }
                    mma_row<0, 4>(acc, ul[j], b);
                }
#pragma unroll
                for (int i = 0; i < 8; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) S[2 * d + i][e] = fmaf(ui, acc[i][e], eC * S[2 * d + i][e]);
            }
            signal(sh.empty + c % NS, lane);
        }
        if (a.final_state) write_state(S, a.final_state + sb, a.dv, col0 + g, t);
        return;
    }

    // the helper; the first one also feeds the stages
    const int hk = h / (a.H / a.Hk);
    const size_t kc0 = ((size_t)b * a.Hk + hk) * a.nc;
    const bool feeds = w == CG && lane == 0;
    if (feeds)
        for (int c = 0; c < NS - 1 && c < n_chunks; c++) load_stage<Pl, DK>(sh, a, kc0 + c, ch0 + c, c, wait);
    for (int c = 0; c < n_chunks; c++) {
        if (feeds && c + NS - 1 < n_chunks)
            load_stage<Pl, DK>(sh, a, kc0 + c + NS - 1, ch0 + c + NS - 1, c + NS - 1, wait);
        __syncwarp();
        uint8_t* st = sh.sm + (c % NS) * Pl::stage;
        if constexpr (MODE == kKeep) {
            // the operand tiles into the chunk's record
            uint8_t* rec = a.records + ((ch0 + c) * groups_of(a.dv) + group) * Record<DK>::bytes;
            float* rf = reinterpret_cast<float*>(rec + Record<DK>::f);
            const bool keeps = col0 < a.dv;
            wait(sh.s_ready + cg, c);
            if (keeps) {
#pragma unroll 4
                for (int kk = 0; kk < KK; kk++) {
                    uint32_t r[4];
                    get4(sf + kk * 512, r, lane);
                    keep_tile(rec + Record<DK>::s, 2 * kk, lane, r);
                    get4(sf + Pl::sHalf + kk * 512, r, lane);
                    keep_tile(rec + Record<DK>::s + 32 * DK, 2 * kk, lane, r);
                }
                if (lane == 0) rf[fS] = sh.s_inv[cg];
            }
            signal(sh.s_free + cg, lane);
            wait(sh.u_ready + cg, c);
            if (keeps) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t r[4];
                    get4(uf + j * 512, r, lane);
                    keep_tile(rec + Record<DK>::u, 2 * j, lane, r);
                    get4(uf + Pl::uHalf + j * 512, r, lane);
                    keep_tile(rec + Record<DK>::u + 2048, 2 * j, lane, r);
                }
                if (lane == 0) rf[fU] = sh.u_inv[cg];
            }
            signal(sh.u_free + cg, lane);
        } else {
            // O^T = s_q (exp(G) S^T Q^T + U^T P^T).  A bf16 output takes one term
            // of S, U and P (off by 2^-12 at most each, against its own 2^-9).
            const uint32_t sQ = tc::smem_u32(st) + 2 * C * DK, sP = tc::smem_u32(st) + Pl::oT + 2 * kTile;
            const float* gt = reinterpret_cast<const float*>(st + Pl::oGate);
            float O[8][4];
            zero(O);
            wait(sh.full + c % NS, c / NS);
            wait(sh.s_ready + cg, c);
#pragma unroll 4
            for (int kk = 0; kk < KK; kk++) {
                uint32_t hi[4], lo[4];
                get4(sf + kk * 512, hi, lane);
                if constexpr (Pl::terms == 2) get4(sf + Pl::sHalf + kk * 512, lo, lane);
                uint32_t bq[4][4];
#pragma unroll
                for (int p = 0; p < 4; p++) ldsm4(bq[p], at_n(sQ, 16 * p, 2 * kk, lane));
                mma_row<0, 4>(O, hi, bq);
                if constexpr (Pl::terms == 2) mma_row<0, 4>(O, lo, bq);
            }
            const float si = sh.s_inv[cg];
            signal(sh.s_free + cg, lane);
            wait(sh.u_ready + cg, c);
            const float ui = sh.u_inv[cg];
            // in units of U's tiles, so that both products share an accumulator
            scale_tokens(O, gt + gEG, si / ui, t);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t uh[4], ul[4];
                get4(uf + j * 512, uh, lane);
                if constexpr (Pl::terms == 2) get4(uf + Pl::uHalf + j * 512, ul, lane);
#pragma unroll
                for (int p = j; p < 4; p++) {
                    uint32_t ph[4];
                    ldsm4(ph, at_n(sP, 16 * p, 2 * j, lane));
                    mma(O[2 * p], uh, ph[0], ph[1]);
                    mma(O[2 * p + 1], uh, ph[2], ph[3]);
                    if constexpr (Pl::terms == 2) {
                        uint32_t pl[4];
                        ldsm4(pl, at_n(sP + kTile, 16 * p, 2 * j, lane));
                        mma(O[2 * p], ul, ph[0], ph[1]);
                        mma(O[2 * p + 1], ul, ph[2], ph[3]);
                        mma(O[2 * p], uh, pl[0], pl[1]);
                        mma(O[2 * p + 1], uh, pl[2], pl[3]);
                    }
                }
            }
            scale_tokens(O, gt + gSq, ui, t);
            const size_t row0 = (size_t)b * a.N + (size_t)c * C;
            const int L = len - c * C;
            if constexpr (MODE == kOutF32) {
                signal(sh.u_free + cg, lane);
                float* o = reinterpret_cast<float*>(a.out);
#pragma unroll
                for (int n = 0; n < 8; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int tok = 8 * n + 2 * t + (e & 1), cc = col0 + g + 8 * (e >> 1);
                        if (tok < L && cc < a.dv) o[((row0 + tok) * a.H + h) * a.dv + cc] = O[n][e];
                    }
            } else {
                // rows of 32 bytes through U's tiles, which have been read
                __syncwarp();
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    uint32_t r4[4];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        r4[2 * i] = tc::pack_bf16x2(O[2 * p + i][0], O[2 * p + i][1]);
                        r4[2 * i + 1] = tc::pack_bf16x2(O[2 * p + i][2], O[2 * p + i][3]);
                    }
                    const int m = lane >> 3;
                    stsm4_t(tc::smem_u32(uf) + 512 * p + (8 * (m >> 1) + (lane & 7)) * 32 + (m & 1) * 16, r4);
                }
                __syncwarp();
                const int cc = col0 + 8 * (lane & 1);
                uint4 o4[4];
#pragma unroll
                for (int p = 0; p < 4; p++) o4[p] = *reinterpret_cast<const uint4*>(uf + 512 * p + 16 * lane);
                signal(sh.u_free + cg, lane);
                __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.out);
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    const int tok = 16 * p + (lane >> 1);
                    if (tok < L && cc < a.dv) *reinterpret_cast<uint4*>(o + ((row0 + tok) * a.H + h) * a.dv + cc) = o4[p];
                }
            }
        }
        signal(sh.empty + c % NS, lane);
    }
}

// ------------------------------------------------------- the backward's chain
//
// With dS1 the gradient of the state after a chunk, and the same T, P:
//     dU = P^T dO' + diag(exp(G_C - G)) K dS1,  Y = T^T dU,  dR = beta' Y
//     dS0 = exp(G_C) dS1 + (diag(exp(G)) Q)^T dO' - (diag(exp(G)) K)^T dR,
// column by column as the forward, the chunks from the last to the first.  The
// helper computes the two terms of dO' ahead of the chain warp.

template <int DK, int CG>
__device__ __forceinline__ void chain_backward(const ChainArgs& a, const float* dfinal, float* dinitial, int b) {
    using Pl = Plan<DK, CG, kBack>;
    constexpr int NS = Pl::NS, KK = DK / 16;
    Shared sh;
    sh.init<Pl, CG>();
    const int h = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = length_of(a.lengths, b, a.N), n_chunks = (len + C - 1) / C;
    const size_t ch0 = ((size_t)b * a.H + h) * a.nc;
    const int cg = w % CG, g = lane >> 2, t = lane & 3;
    const int group = blockIdx.x * CG + cg, col0 = group * 16;
    uint8_t* ex = sh.sm + Pl::oG + cg * Pl::group;
    uint8_t *sf = ex, *uf = ex + Pl::oU, *slot = ex + Pl::oV;
    float4 *zf = reinterpret_cast<float4*>(ex + Pl::oZ) + lane, *df = reinterpret_cast<float4*>(ex + Pl::oD) + lane;
    Waits wait;

    if (w < CG) {
        const size_t sb = ((size_t)b * a.H + h) * DK * a.dv;
        float S[DK / 8][4];
        read_state(S, dfinal ? dfinal + sb : nullptr, a.dv, col0 + g, t);
        for (int it = 0; it < n_chunks; it++) {
            uint8_t* st = sh.sm + (it % NS) * Pl::stage;
            const uint32_t sK = tc::smem_u32(st), sT = sK + Pl::oT;
            const float* gt = reinterpret_cast<const float*>(st + Pl::oGate);

            // dS^T K^T
            float inv;
            const float ss = tiles_scale(S, inv);
            const float si = inv;
            float U[8][4];
            zero(U);
            wait(sh.full + it % NS, it / NS);
            if (it > 0) wait(sh.s_free + cg, it - 1);
#pragma unroll
            for (int kk = 0; kk < KK; kk++) {
                uint32_t hi[4], lo[4];
                split_a(S[2 * kk], S[2 * kk + 1], ss, hi, lo);
                put4(sf + kk * 512, hi, lane);
                put4(sf + Pl::sHalf + kk * 512, lo, lane);
                uint32_t bk[4][4];
#pragma unroll
                for (int p = 0; p < 4; p++) ldsm4(bk[p], at_n(sK, 16 * p, 2 * kk, lane));
                mma_row<0, 4>(U, hi, bk);
                mma_row<0, 4>(U, lo, bk);
            }
            if (lane == 0) sh.s_inv[cg] = si;
            signal(sh.s_ready + cg, lane);
            scale_tokens(U, gt + gEC, si, t);
            wait(sh.z_ready + cg, it);
#pragma unroll
            for (int n = 0; n < 8; n++) {
                const float4 d = df[32 * n];
                U[n][0] += d.x, U[n][1] += d.y, U[n][2] += d.z, U[n][3] += d.w;
            }
            const float us = tiles_scale(U, inv);
            const float ui = inv;

            // Y^T = dU^T T: token j takes i >= j
            float Y[8][4];
            zero(Y);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t uh[4], ul[4];
                split_a(U[2 * i], U[2 * i + 1], us, uh, ul);
                uint32_t th[4][4], tl[4][4];
#pragma unroll
                for (int d = 0; d <= i; d++) {
                    ldsm4_t(th[d], at_k(sT, 16 * i, 2 * d, lane));
                    ldsm4_t(tl[d], at_k(sT + kTile, 16 * i, 2 * d, lane));
                }
#pragma unroll
                for (int k = 0; k < 3; k++)
#pragma unroll
                    for (int d = 0; d <= i; d++) {
                        const uint32_t(&b)[4] = k == 2 ? tl[d] : th[d];
                        mma(Y[2 * d], k == 1 ? ul : uh, b[0], b[1]);
                        mma(Y[2 * d + 1], k == 1 ? ul : uh, b[2], b[3]);
                    }
            }
            const float ys = tiles_scale(Y, inv);  // of us-scaled values
            const float yi = inv * ui;
            if (it > 0) wait(sh.u_free + cg, it - 1);
            uint32_t yh[4][4], yl[4][4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                split_a(Y[2 * j], Y[2 * j + 1], ys, yh[j], yl[j]);
                put4(uf + j * 512, yh[j], lane);
                put4(uf + Pl::uHalf + j * 512, yl[j], lane);
            }
            if (lane == 0) sh.u_inv[cg] = yi;
            signal(sh.u_ready + cg, lane);

            // dS^T <- exp(G_C) dS^T + Z - (exp(G) beta' Y)^T K
            const float eC = gt[gEG + C - 1];
            scale_tokens(Y, gt + gEG, -ys, t);
            scale_tokens(Y, gt + gBeta, 1.f, t);
#pragma unroll
            for (int j = 0; j < 4; j++) split_a(Y[2 * j], Y[2 * j + 1], 1.f, yh[j], yl[j]);
#pragma unroll
            for (int d = 0; d < KK; d += 4) {
                float acc[8][4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t b[4][4];
#pragma unroll
                    for (int i = 0; i < 4; i++) ldsm4_t(b[i], at_k(sK, 16 * j, 2 * (d + i), lane));
                    if (j == 0) {
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            mma0(acc[2 * i], yh[j], b[i][0], b[i][1]);
                            mma0(acc[2 * i + 1], yh[j], b[i][2], b[i][3]);
                        }
                    } else {
                        mma_row<0, 4>(acc, yh[j], b);
                    }
                    mma_row<0, 4>(acc, yl[j], b);
                }
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float4 z = zf[32 * (2 * d + i)];
                    S[2 * d + i][0] = fmaf(yi, acc[i][0], fmaf(eC, S[2 * d + i][0], z.x));
                    S[2 * d + i][1] = fmaf(yi, acc[i][1], fmaf(eC, S[2 * d + i][1], z.y));
                    S[2 * d + i][2] = fmaf(yi, acc[i][2], fmaf(eC, S[2 * d + i][2], z.z));
                    S[2 * d + i][3] = fmaf(yi, acc[i][3], fmaf(eC, S[2 * d + i][3], z.w));
                }
            }
            signal(sh.z_free + cg, lane);
            signal(sh.empty + it % NS, lane);
        }
        if (dinitial) write_state(S, dinitial + sb, a.dv, col0 + g, t);
        return;
    }

    const int hk = h / (a.H / a.Hk);
    const size_t kc0 = ((size_t)b * a.Hk + hk) * a.nc;
    const bool feeds = w == CG && lane == 0, keeps = col0 < a.dv;
    auto load = [&](int it) {
        const int c = n_chunks - 1 - it;
        load_stage<Pl, DK>(sh, a, kc0 + c, ch0 + c, it, wait);
    };
    if (feeds)
        for (int it = 0; it < NS - 1 && it < n_chunks; it++) load(it);
    const Rows orows = rows_at(a.dout, a, b, h, col0 + 8 * (lane & 1), len);
    uint4 on[4];
    if (n_chunks)
#pragma unroll
        for (int i = 0; i < 4; i++) on[i] = orows.load((n_chunks - 1) * C + 16 * i + (lane >> 1));
    for (int it = 0; it < n_chunks; it++) {
        if (feeds && it + NS - 1 < n_chunks) load(it + NS - 1);
        __syncwarp();
        {  // dO' of this chunk: its record's tile, dU0 and Z
            const int c = n_chunks - 1 - it;
            uint8_t* st = sh.sm + (it % NS) * Pl::stage;
            const uint32_t sQ = tc::smem_u32(st) + 2 * C * DK, sP = tc::smem_u32(st) + Pl::oT + 2 * kTile;
            const float* gt = reinterpret_cast<const float*>(st + Pl::oGate);
            uint8_t* rec = a.records + ((ch0 + c) * groups_of(a.dv) + group) * Record<DK>::bytes;
            float* rf = reinterpret_cast<float*>(rec + Record<DK>::f);
            float o[8][4];
            wait(sh.full + it % NS, it / NS);
#pragma unroll
            for (int p = 0; p < 4; p++) {
                uint32_t v4[4];
                transpose16(slot + 512 * p, orows.use(on[p], c * C + 16 * p + (lane >> 1)), lane, v4);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    o[2 * p + i][0] = tc::bf16lo(v4[2 * i]);
                    o[2 * p + i][1] = tc::bf16hi(v4[2 * i]);
                    o[2 * p + i][2] = tc::bf16lo(v4[2 * i + 1]);
                    o[2 * p + i][3] = tc::bf16hi(v4[2 * i + 1]);
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; i++) on[i] = orows.load(max(c - 1, 0) * C + 16 * i + (lane >> 1));
            scale_tokens(o, gt + gSq, 1.f, t);
            float oi;
            const float os = tiles_scale(o, oi);
            uint32_t oh[4][4], ol[4][4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                split_a(o[2 * i], o[2 * i + 1], os, oh[i], ol[i]);  // exact in one term, up to its range
                if (keeps) keep_tile(rec + Record<DK>::o, 2 * i, lane, oh[i]);
            }
            if (keeps && lane == 0) rf[fO] = oi;
            // dU0^T = dO'^T P: token j takes i >= j
            float U[8][4];
            zero(U);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int k = 0; k < 2; k++)
#pragma unroll
                    for (int d = 0; d <= i; d++) {
                        uint32_t b[4];
                        ldsm4_t(b, at_k(sP + k * kTile, 16 * i, 2 * d, lane));
                        mma(U[2 * d], oh[i], b[0], b[1]);
                        mma(U[2 * d + 1], oh[i], b[2], b[3]);
                    }
            scale_tokens(o, gt + gEG, os, t);
#pragma unroll
            for (int i = 0; i < 4; i++) split_a(o[2 * i], o[2 * i + 1], 1.f, oh[i], ol[i]);
            if (it > 0) wait(sh.z_free + cg, it - 1);
#pragma unroll
            for (int n = 0; n < 8; n++) df[32 * n] = make_float4(U[n][0] * oi, U[n][1] * oi, U[n][2] * oi, U[n][3] * oi);
            // Z^T = (exp(G) dO')^T Q
#pragma unroll 1
            for (int d = 0; d < KK; d += 4) {
                float acc[8][4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t b[4][4];
#pragma unroll
                    for (int i = 0; i < 4; i++) ldsm4_t(b[i], at_k(sQ, 16 * j, 2 * (d + i), lane));
                    if (j == 0) {
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            mma0(acc[2 * i], oh[j], b[i][0], b[i][1]);
                            mma0(acc[2 * i + 1], oh[j], b[i][2], b[i][3]);
                        }
                    } else {
                        mma_row<0, 4>(acc, oh[j], b);
                    }
                    mma_row<0, 4>(acc, ol[j], b);
                }
#pragma unroll
                for (int i = 0; i < 8; i++)
                    zf[32 * (2 * d + i)] = make_float4(acc[i][0] * oi, acc[i][1] * oi, acc[i][2] * oi, acc[i][3] * oi);
            }
            signal(sh.z_ready + cg, lane);
            signal(sh.empty + it % NS, lane);
        }
        {  // the chain's tiles of this chunk into its record
            uint8_t* rec = a.records + ((ch0 + n_chunks - 1 - it) * groups_of(a.dv) + group) * Record<DK>::bytes;
            float* rf = reinterpret_cast<float*>(rec + Record<DK>::f);
            wait(sh.s_ready + cg, it);
            if (keeps) {
#pragma unroll 4
                for (int kk = 0; kk < KK; kk++) {
                    uint32_t r[4];
                    get4(sf + kk * 512, r, lane);
                    keep_tile(rec + Record<DK>::ds, 2 * kk, lane, r);
                    get4(sf + Pl::sHalf + kk * 512, r, lane);
                    keep_tile(rec + Record<DK>::ds + 32 * DK, 2 * kk, lane, r);
                }
                if (lane == 0) rf[fDs] = sh.s_inv[cg];
            }
            signal(sh.s_free + cg, lane);
            wait(sh.u_ready + cg, it);
            if (keeps) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t r[4];
                    get4(uf + j * 512, r, lane);
                    keep_tile(rec + Record<DK>::y, 2 * j, lane, r);
                    get4(uf + Pl::uHalf + j * 512, r, lane);
                    keep_tile(rec + Record<DK>::y + 2048, 2 * j, lane, r);
                }
                if (lane == 0) rf[fY] = sh.u_inv[cg];
            }
            signal(sh.u_free + cg, lane);
        }
    }
}

// ------------------------------------------------------------------ kernels

template <int DK, int CG, int MODE>
__global__ void __launch_bounds__(Plan<DK, CG, MODE>::warps * 32, 1) k_delta_chain(const __grid_constant__ ChainArgs a) {
    chain_forward<DK, CG, MODE>(a, blockIdx.z);
}

// The backward's two chains do not depend on each other: half of the blocks
// walk forward (states and corrections), half backward, side by side.
template <int DK, int CG>
__global__ void __launch_bounds__(Plan<DK, CG, kBack>::warps * 32, 1)
    k_delta_chains(const __grid_constant__ ChainArgs a, const float* dfinal, float* dinitial) {
    if (blockIdx.z & 1) chain_forward<DK, CG, kKeep>(a, blockIdx.z >> 1);
    else chain_backward<DK, CG>(a, dfinal, dinitial, blockIdx.z >> 1);
}

// Groups of 16 columns a block takes: as many as share the tiles (fewer loads)
// while every one of the 148 SMs that can be busy is.
int groups_of_block(const DeltaArgs& a, int most, int chains) {
    int cg = most;
    const long long all = (long long)a.B * a.H * chains;
    while (cg > 1 && all * ((groups_of(a.dv) + cg / 2 - 1) / (cg / 2)) <= 148) cg /= 2;
    return cg;
}

template <int DK, int CG, int MODE>
ret_status chain(const DeltaArgs& a, const ChainArgs& c, cudaStream_t s) {
    using Pl = Plan<DK, CG, MODE>;
    cudaError_t e = cudaFuncSetAttribute(k_delta_chain<DK, CG, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Pl::smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule: %s", cudaGetErrorString(e));
    const dim3 grid((groups_of(a.dv) + CG - 1) / CG, a.H, a.B);
    k_delta_chain<DK, CG, MODE><<<grid, Pl::warps * 32, Pl::smem, s>>>(c);
    return check_launch("delta rule: chain");
}

template <int DK>
ret_status chain_dk(const DeltaArgs& a, const ChainArgs& c, cudaStream_t s) {
    if (a.out_dt == RET_F32) {
        const int cg = groups_of_block(a, 2, 1);
        return cg == 2 ? chain<DK, 2, kOutF32>(a, c, s) : chain<DK, 1, kOutF32>(a, c, s);
    }
    const int cg = groups_of_block(a, 4, 1);
    return cg == 4   ? chain<DK, 4, kOutBf16>(a, c, s)
           : cg == 2 ? chain<DK, 2, kOutBf16>(a, c, s)
                     : chain<DK, 1, kOutBf16>(a, c, s);
}

ChainArgs chain_args(const DeltaArgs& a, const Tables& t) {
    ChainArgs c{};
    c.tb = t;
    c.lengths = a.lengths;
    c.initial_state = a.initial_state;
    c.final_state = a.final_state;
    c.v = (const __nv_bfloat16*)a.v;
    c.dout = (const __nv_bfloat16*)a.dout;
    c.out = a.out;
    c.N = a.N;
    c.nc = chunks_of(a.N);
    c.Hk = a.Hk;
    c.H = a.H;
    c.dv = a.dv;
    return c;
}

template <int DK, int CG>
ret_status chains(const DeltaArgs& a, const ChainArgs& c, cudaStream_t s) {
    constexpr int smem = std::max(Plan<DK, CG, kKeep>::smem, Plan<DK, CG, kBack>::smem);
    cudaError_t e = cudaFuncSetAttribute(k_delta_chains<DK, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail(RET_ERR_CUDA, "delta rule: %s", cudaGetErrorString(e));
    const dim3 grid((groups_of(a.dv) + CG - 1) / CG, a.H, 2 * a.B);
    k_delta_chains<DK, CG><<<grid, Plan<DK, CG, kBack>::warps * 32, smem, s>>>(c, a.dfinal_state, a.dinitial_state);
    return check_launch("delta rule: the backward's chains");
}
template <int DK>
ret_status chains_dk(const DeltaArgs& a, const ChainArgs& c, cudaStream_t s) {
    return groups_of_block(a, 2, 2) == 2 ? chains<DK, 2>(a, c, s) : chains<DK, 1>(a, c, s);
}

}  // namespace

ret_status launch_chains(const DeltaArgs& a, const Tables& t, uint8_t* records, cudaStream_t s) {
    ChainArgs c = chain_args(a, t);
    c.final_state = nullptr;
    c.records = records;
    return a.dk == 64 ? chains_dk<64>(a, c, s) : a.dk == 128 ? chains_dk<128>(a, c, s) : chains_dk<256>(a, c, s);
}

}  // namespace delta

using namespace delta;

bool delta_chunk_shape_ok(const DeltaArgs& a) {
    return a.in_dt == RET_BF16 && (a.dk == 64 || a.dk == 128 || a.dk == 256) && a.dv % 8 == 0;
}

size_t delta_forward_ws_bytes(const DeltaArgs& a) { return table_bytes(a); }

ret_status launch_delta_forward(const DeltaArgs& a, void* ws, cudaStream_t s) {
    const Tables t = tables_at(a, ws);
    ret_status st = launch_prep(a, t, s);
    if (st != RET_OK) return st;
    const ChainArgs c = chain_args(a, t);
    return a.dk == 64 ? chain_dk<64>(a, c, s) : a.dk == 128 ? chain_dk<128>(a, c, s) : chain_dk<256>(a, c, s);
}

}  // namespace ret
