// k_delta_chunk.cu -- the recurrence of the gated delta rule over the chunks of
// a sequence, forward and backward (notation and number format:
// delta_util.cuh; the tables come from k_delta_prep.cu).
//
// What bounds it is the chain: chunk c + 1 needs the state of chunk c, and a
// (sequence, head) has only its value columns to share out, which do not
// depend on each other.  Sixteen columns are the work of three warps.
// Two chain warps carry them through the recurrence: each holds half of dk of
// the transposed state, [16 x dk/2] as fp32 accumulator tiles, whose layout is
// that of the A operand of the next product (X^T = S^T K^T, U^T = R^T T^T,
// S^T += U^T K), and owns two of the four quarters of the chunk's tokens between
// the products over dk (the first and the last, or the two between: T is
// triangular, so both have the same work).  They exchange parts of X, R and U
// through shared memory, with three barriers of 64 threads in a chunk.  (One
// warp alone takes 8,700 clocks for a chunk of dk = 128, of which the tensor pipe
// needs 2,600; the halves took 898 to 800 us at 1 x 8192 x 16 x 256 x 512.)
// Everything that the recurrence does not wait for is the third warp's, the
// helper: the outputs (Q S and P U), or in the backward pass the terms of dO,
// where a fourth warp writes the records.  They get the operand tiles of S and U
// as they are.
// The products run as mma.sync, not tcgen05: every operand is split into two
// fp16 terms between two products, in registers at once, where TMEM would cost
// a trip out and back for each of the four products of a chunk.
// K', Q', T, P come by bulk copies into a ring of stages, issued by a helper.
//
// A stage is handed back behind a proxy fence (see release) and every wait of a
// warp ends in a vote (see Waits).
//
// 1 x 8192, 16 heads of 256 / 512: 128 blocks of four groups, 1,030 us, 8.1 us a
// chunk; with one term of S, U and P for the outputs a sixth less (the helper's
// products share the tensor pipe, and tiles of two terms leave the rings one stage
// each).
// 4 x 2047, 16 heads of 128 / 128: 166 us, 5.2 us a chunk of the longest sequence.
// The backward's chains of 1 x 4096, 16 heads of 128 / 128: 64 blocks of two groups a
// way, 300 us.
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
    // 2 CG warps of the chains, CG helpers, and CG that write the records
    static constexpr int warps = MODE == kKeep || MODE == kBack ? 4 * CG : 3 * CG;
    // Two rings: the chain warps' K', T and gates, and the helpers' Q', P and gates.
    static constexpr int kGateRoom = 1536, keys = 2 * C * DK;
    static constexpr int oT = keys, aGate = oT + 2 * kTile, A = aGate + kGateRoom;
    static constexpr int oP = keys, bGate = oP + 2 * kTile, B = MODE == kKeep ? 0 : bGate + kGateRoom;
    // a group's: S in two terms, U (Y) the same way, staging of 64 x 16 bf16;
    // between the chain warps parts of X, in whose place each later puts its R (dU),
    // and exp(G_C - G) U (exp(G) beta' Y) in fp32; the backward: Z in fp32, dU0 in fp32
    static constexpr int sHalf = DK / 16 * 512, oU = 2 * sHalf, uHalf = 4 * 512, oV = oU + 2 * uHalf;
    static constexpr int oX = oV + 2048, oE = oX + 4096;
    static constexpr int oZ = oE + 4096, oD = oZ + (MODE == kBack ? DK * 64 : 0);
    static constexpr int group = oD + (MODE == kBack ? 4096 : 0);
    static constexpr int most = 226 * 1024 - 1024 - 512, left = most - CG * group;
    static constexpr int NA = 2 * A + B <= left ? 2 : 1, NB = NA * A + 2 * B <= left ? 2 : 1;
    static_assert(NA * A + NB * B <= left, "tiles and exchange buffers exceed shared memory");
    static constexpr int oB = NA * A, oG = oB + NB * B, oBar = oG + CG * group;
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
// A wait is the whole warp's and ends in a vote.  Polling ends lane by lane, and
// what comes after it (ldmatrix, mma.sync) is defined only for a warp whose lanes
// execute it together.
struct Waits {
    bool ok = true;  // the same in all lanes, but for the feeding lane between `lane` and `together`
    __device__ __forceinline__ void operator()(uint64_t* bar, int phase) {
        if (!__all_sync(0xffffffffu, !ok || tc::mbar_wait(bar, phase & 1))) give_up();
    }
    // One lane's, while the others wait in `together`.
    __device__ __forceinline__ void lane(uint64_t* bar, int phase) {
        if (ok && !tc::mbar_wait(bar, phase & 1)) give_up();
    }
    __device__ __forceinline__ void together() { ok = __all_sync(0xffffffffu, ok); }

private:
    __device__ __forceinline__ void give_up() {
        ok = false;
        atomicExch(&g_delta_err, kErrTimeout);
    }
};
__device__ __forceinline__ void signal(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}
// Hands a stage back to the bulk copies.  The warp has read it through the generic
// proxy and the copy writes through the async proxy: an mbarrier alone does not
// order the two, and the last ldmatrix could find rows of the stage's next tiles.
__device__ __forceinline__ void release(uint64_t* bar, int lane) {
    tc::fence_proxy_async_smem();
    signal(bar, lane);
}

// The block's shared memory and barriers: the stages', and for each group a
// pair (ready, free) for the tiles of S, those of U and the helper's fp32 terms.
struct Shared {
    uint8_t* sm;
    uint64_t *fa, *ea, *fb, *eb, *s_ready, *s_free, *u_ready, *u_free, *z_ready, *z_free;
    float *s_inv, *u_inv, *s_max, *v_max, *e_max;  // [2] a group, u_inv one
    template <typename Pl, int CG>
    __device__ __forceinline__ void init() {
        extern __shared__ uint8_t raw[];
        sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
        fa = reinterpret_cast<uint64_t*>(sm + Pl::oBar);
        ea = fa + 2, fb = ea + 2, eb = fb + 2, s_ready = eb + 2, s_free = s_ready + 4, u_ready = s_free + 4, u_free = u_ready + 4;
        z_ready = u_free + 4, z_free = z_ready + 4;
        s_inv = reinterpret_cast<float*>(z_free + 4);
        u_inv = s_inv + 8, s_max = u_inv + 4, v_max = s_max + 8, e_max = v_max + 8;
        if (threadIdx.x == 0) {
            for (int i = 0; i < 2; i++) {
                tc::mbar_init(fa + i, 1), tc::mbar_init(fb + i, 1);
                tc::mbar_init(ea + i, 2 * CG), tc::mbar_init(eb + i, CG);
            }
            for (int i = 0; i < CG; i++) {
                for (uint64_t* b : {s_free, u_free, z_ready}) tc::mbar_init(b + i, 1);
                for (uint64_t* b : {s_ready, u_ready, z_free}) tc::mbar_init(b + i, 2);
            }
            tc::fence_barrier_init();
        }
        __syncthreads();
    }
};

// One lane: the tiles of a chunk, the it-th that is walked, into the rings; `to`
// counts the chunks under way.
template <typename Pl, int DK>
__device__ __forceinline__ void load_a(const Shared& r, const ChainArgs& a, size_t key_chunk, size_t chunk, int it,
                                       Waits& wait, int& to) {
    if (it >= Pl::NA) wait.lane(r.ea + it % Pl::NA, it / Pl::NA - 1);
    if (!wait.ok) return;
    to = it + 1;
    uint8_t* s = r.sm + (it % Pl::NA) * Pl::A;
    uint64_t* bar = r.fa + it % Pl::NA;
    tc::mbar_arrive_expect_tx(bar, Pl::keys + 2 * kTile + kGates);
    bulk_load(s, a.tb.keys + key_chunk * (4 * C * DK), Pl::keys, bar);
    bulk_load(s + Pl::aGate, a.tb.gates + chunk * kGateRow, kGates, bar);
    bulk_load(s + Pl::oT, a.tb.tiles + chunk * 4 * kTile, 2 * kTile, bar);
}
template <typename Pl, int DK>
__device__ __forceinline__ void load_b(const Shared& r, const ChainArgs& a, size_t key_chunk, size_t chunk, int it,
                                       Waits& wait, int& to) {
    if (it >= Pl::NB) wait.lane(r.eb + it % Pl::NB, it / Pl::NB - 1);
    if (!wait.ok) return;
    to = it + 1;
    uint8_t* s = r.sm + Pl::oB + (it % Pl::NB) * Pl::B;
    uint64_t* bar = r.fb + it % Pl::NB;
    tc::mbar_arrive_expect_tx(bar, Pl::keys + 2 * kTile + kGates);
    bulk_load(s, a.tb.keys + key_chunk * (4 * C * DK) + Pl::keys, Pl::keys, bar);
    bulk_load(s + Pl::oP, a.tb.tiles + chunk * 4 * kTile + 2 * kTile, 2 * kTile, bar);
    bulk_load(s + Pl::bGate, a.tb.gates + chunk * kGateRow, kGates, bar);
}
// The feeding lane, last: no copy of the block's is in flight when it ends, not even
// where a warp gave up a wait and did not see its tiles come.
template <typename Pl>
__device__ __forceinline__ void settle(const Shared& r, int to_a, int to_b) {
    for (int i = max(to_a - Pl::NA, 0); i < to_a; i++) tc::mbar_wait(r.fa + i % Pl::NA, (i / Pl::NA) & 1);
    for (int i = max(to_b - Pl::NB, 0); i < to_b; i++) tc::mbar_wait(r.fb + i % Pl::NB, (i / Pl::NB) & 1);
}

__device__ __forceinline__ void put4(uint8_t* p, const uint32_t (&r)[4], int lane) {
    *reinterpret_cast<uint4*>(p + 16 * lane) = make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void get4(const uint8_t* p, uint32_t (&r)[4], int lane) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + 16 * lane);
    r[0] = u.x, r[1] = u.y, r[2] = u.z, r[3] = u.w;
}

// The largest magnitude of a warp's tiles, and the scale for it.
template <int N>
__device__ __forceinline__ float tiles_max(const float (&S)[N][4]) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) m[e] = fmaxf(m[e], fabsf(S[n][e]));
    return warp_max(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
}
template <int N>
__device__ __forceinline__ float tiles_scale(const float (&S)[N][4], float& inverse) {
    return scale_for(tiles_max(S), inverse);
}
// The parts of a product over dk: the other warp's quarters (its first and
// second) go to it, the own ones (hf and 3 - hf) are returned.
__device__ __forceinline__ void hand_over(uint8_t* buf, const float (&x)[8][4], int hf, float s, int lane, float (&mine)[4][4]) {
    float4* dst = reinterpret_cast<float4*>(buf + (1 - hf) * 2048) + lane;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        // tiles of quarters 0, 3 (hf 0) and 1, 2 (hf 1), in that order
        const int t0 = i < 2 ? i : 4 + i, t1 = 2 + i;
        const float(&give)[4] = hf ? x[t0] : x[t1];
        const float(&keep)[4] = hf ? x[t1] : x[t0];
        dst[32 * i] = make_float4(give[0] * s, give[1] * s, give[2] * s, give[3] * s);
#pragma unroll
        for (int e = 0; e < 4; e++) mine[i][e] = keep[e] * s;
    }
}
__device__ __forceinline__ void take_over(const uint8_t* buf, int hf, int lane, float (&mine)[4][4]) {
    const float4* src = reinterpret_cast<const float4*>(buf + hf * 2048) + lane;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float4 y = src[32 * i];
        mine[i][0] += y.x, mine[i][1] += y.y, mine[i][2] += y.z, mine[i][3] += y.w;
    }
}
// acc = sum over the tokens of (hi + lo)^T B, B's 16 D columns from piece 2 d on.
template <int D>
__device__ __forceinline__ void state_product(float (&acc)[8][4], const uint32_t (&hi)[4][4], const uint32_t (&lo)[4][4],
                                              uint32_t sB, int d, int lane) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint32_t b[4][4];
#pragma unroll
        for (int i = 0; i < D; i++) ldsm4_t(b[i], at_k(sB, 16 * j, 2 * (d + i), lane));
        if (j == 0) {
#pragma unroll
            for (int i = 0; i < D; i++) {
                mma0(acc[2 * i], lo[j], b[i][0], b[i][1]);
                mma0(acc[2 * i + 1], lo[j], b[i][2], b[i][3]);
            }
        } else {
            mma_row<0, D>(acc, lo[j], b);
        }
        mma_row<0, D>(acc, hi[j], b);
    }
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
// What a chunk adds to the state, tokens times factors in [0, 1]: behind a strong
// decay far below the tiles that it was computed from, so it is exchanged in fp32
// and split with a scale of its own.  The own quarters' tiles into the exchange;
// their largest magnitude.
__device__ __forceinline__ float put_gated(uint8_t* buf, const float (&x)[4][4], int qa, int qb, int lane) {
    float m = 0.f;
#pragma unroll
    for (int n = 0; n < 4; n++) {
        *reinterpret_cast<float4*>(buf + (n < 2 ? qa : qb) * 1024 + (n & 1) * 512 + 16 * lane) =
            make_float4(x[n][0], x[n][1], x[n][2], x[n][3]);
#pragma unroll
        for (int e = 0; e < 4; e++) m = fmaxf(m, fabsf(x[n][e]));
    }
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}
__device__ __forceinline__ void get_gated(const uint8_t* buf, float s, int lane, uint32_t (&hi)[4][4], uint32_t (&lo)[4][4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float4 u = *reinterpret_cast<const float4*>(buf + j * 1024 + 16 * lane);
        const float4 v = *reinterpret_cast<const float4*>(buf + j * 1024 + 512 + 16 * lane);
        const float x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
        split_a(x, y, s, hi[j], lo[j]);
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
    constexpr int NA = Pl::NA, NB = Pl::NB, KK = DK / 16;
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

    if (w < 2 * CG) {  // the chain: half `hf` of dk, quarters qa and qb of the tokens
        constexpr int KH = KK / 2;
        const int hf = w / CG, qa = hf, qb = 3 - hf;
        const size_t sb = (((size_t)b * a.H + h) * DK + hf * (DK / 2)) * a.dv;
        float S[DK / 16][4];
        read_state(S, a.initial_state ? a.initial_state + sb : nullptr, a.dv, col0 + g, t);
        const Rows vrows = rows_at(a.v, a, b, h, col0 + 8 * (lane & 1), len);
        const int tok_a = 16 * qa + (lane >> 1), tok_b = 16 * qb + (lane >> 1);
        uint4 va = make_uint4(0, 0, 0, 0), vb = va;
        if (n_chunks) va = vrows.load(tok_a), vb = vrows.load(tok_b);
        float m_own = tiles_max(S);
        uint8_t *xf = ex + Pl::oX, *ef = ex + Pl::oE;
        // R of quarter q, in its owner's part of the exchange of X: quarters 0, 3, 1, 2
        auto rf = [&](int q) { return xf + 1024 * (q == 0 ? 0 : q == 3 ? 1 : q == 1 ? 2 : 3); };
        for (int c = 0; c < n_chunks; c++) {
            uint8_t* st = sh.sm + (c % NA) * Pl::A;
            const uint32_t sK = tc::smem_u32(st), sT = sK + Pl::oT;
            const float* gt = reinterpret_cast<const float*>(st + Pl::aGate);
            // V of the own quarters, transposed
            uint32_t v4[2][4];
            transpose16(slot + 512 * qa, vrows.use(va, c * C + tok_a), lane, v4[0]);
            transpose16(slot + 512 * qb, vrows.use(vb, c * C + tok_b), lane, v4[1]);
            va = vrows.load((c + 1) * C + tok_a);
            vb = vrows.load((c + 1) * C + tok_b);

            // the half's X^T = S^T K^T; the helper gets the operand tiles
            float si;
            const float ss = scale_for(m_own, si);
            float X[8][4];
            zero(X);
            wait(sh.fa + c % NA, c / NA);
            if (c > 0) wait(sh.s_free + cg, c - 1);
#pragma unroll
            for (int kk = 0; kk < KH; kk++) {
                uint32_t hi[4], lo[4];
                split_a(S[2 * kk], S[2 * kk + 1], ss, hi, lo);
                put4(sf + (hf * KH + kk) * 512, hi, lane);
                put4(sf + Pl::sHalf + (hf * KH + kk) * 512, lo, lane);
                uint32_t bk[4][4];
#pragma unroll
                for (int p = 0; p < 4; p++) ldsm4(bk[p], at_n(sK, 16 * p, 2 * (hf * KH + kk), lane));
                mma_row<0, 4>(X, hi, bk);
                mma_row<0, 4>(X, lo, bk);
            }
            // beta' V' of the own quarters and its largest value
            float vq[4][4], vm = 0.f;
#pragma unroll
            for (int n = 0; n < 4; n++) {
                const int at = 16 * (n < 2 ? qa : qb) + 8 * (n & 1) + 2 * t;
                float2 ik = *reinterpret_cast<const float2*>(gt + gIk + at);
                const float2 bt = *reinterpret_cast<const float2*>(gt + gBeta + at);
                ik.x *= bt.x, ik.y *= bt.y;
                const uint32_t x = v4[n / 2][2 * (n & 1)], y = v4[n / 2][2 * (n & 1) + 1];
                vq[n][0] = tc::bf16lo(x) * ik.x, vq[n][1] = tc::bf16hi(x) * ik.y;
                vq[n][2] = tc::bf16lo(y) * ik.x, vq[n][3] = tc::bf16hi(y) * ik.y;
#pragma unroll
                for (int e = 0; e < 4; e++) vm = fmaxf(vm, fabsf(vq[n][e]));
            }
            vm = warp_max(vm);
            if (lane == 0) {
                sh.s_inv[2 * cg + hf] = si;
                sh.s_max[2 * cg + hf] = m_own;
                sh.v_max[2 * cg + hf] = vm;
            }
            signal(sh.s_ready + cg, lane);
            float R[4][4];  // quarters qa, qb
            hand_over(xf, X, hf, si, lane, R);
            tc::barrier(1 + cg, 64);
            take_over(xf, hf, lane, R);

            // R^T = beta' (V' - exp(G) X); one scale for R and U of the group
            const float bound = fmaxf(fmaxf(sh.v_max[2 * cg], sh.v_max[2 * cg + 1]),
                                      fmaxf(sh.s_max[2 * cg], sh.s_max[2 * cg + 1]) * fmaxf(1.f, fmaxf(gt[gMax], gt[gMax + 1])));
            float ui;
            const float us = bound_scale(bound, ui);
#pragma unroll
            for (int n = 0; n < 4; n++) {
                const int at = 16 * (n < 2 ? qa : qb) + 8 * (n & 1) + 2 * t;
                const float2 eg = *reinterpret_cast<const float2*>(gt + gEG + at);
                const float2 bt = *reinterpret_cast<const float2*>(gt + gBeta + at);
                R[n][0] = fmaf(-bt.x * eg.x, R[n][0], vq[n][0]);
                R[n][1] = fmaf(-bt.y * eg.y, R[n][1], vq[n][1]);
                R[n][2] = fmaf(-bt.x * eg.x, R[n][2], vq[n][2]);
                R[n][3] = fmaf(-bt.y * eg.y, R[n][3], vq[n][3]);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                uint32_t hi[4], lo[4];
                const int q = i ? qb : qa;
                split_a(R[2 * i], R[2 * i + 1], us, hi, lo);
                put4(rf(q), hi, lane);
                put4(rf(q) + 512, lo, lane);
            }
            tc::barrier(1 + cg, 64);

            // U^T = R^T T^T; T is lower triangular: token i takes j <= i
            float U[4][4];
            zero(U);
            // the small products, then the large ones; for the gradients in passes of
            // their own (which would cost the forward 2% at dk 256)
            constexpr int kPasses = MODE == kKeep ? 2 : 1;
#pragma unroll
            for (int pass = 0; pass < kPasses; pass++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (j > qb) continue;
                    uint32_t rh[4], rl[4], th[2][4], tl[2][4];
                    get4(rf(j), rh, lane);
                    if (pass == 0) get4(rf(j) + 512, rl, lane);
#pragma unroll
                    for (int i = 0; i < 2; i++)
                        if (i || j <= qa) {
                            ldsm4(th[i], at_n(sT, 16 * (i ? qb : qa), 2 * j, lane));
                            if (pass == 0) ldsm4(tl[i], at_n(sT + kTile, 16 * (i ? qb : qa), 2 * j, lane));
                        }
#pragma unroll
                    for (int k = pass * 2; k < (kPasses == 1 || pass ? 3 : 2); k++)
#pragma unroll
                        for (int i = 0; i < 2; i++)
                            if (i || j <= qa) {
                                const uint32_t(&x)[4] = k == 1 ? tl[i] : th[i];
                                mma(U[2 * i], k == 0 ? rl : rh, x[0], x[1]);
                                mma(U[2 * i + 1], k == 0 ? rl : rh, x[2], x[3]);
                            }
                }
            if (c > 0) wait(sh.u_free + cg, c - 1);
            // U for the helper, exp(G_C - G) U for the state
#pragma unroll
            for (int i = 0; i < 2; i++) {
                uint32_t hi[4], lo[4];
                const int q = i ? qb : qa;
                split_a(U[2 * i], U[2 * i + 1], 1.f, hi, lo);
                put4(uf + q * 512, hi, lane);
                put4(uf + Pl::uHalf + q * 512, lo, lane);
            }
            if (lane == 0 && hf == 0) sh.u_inv[cg] = ui;
            signal(sh.u_ready + cg, lane);
#pragma unroll
            for (int n = 0; n < 4; n++) {
                const float2 e2 = *reinterpret_cast<const float2*>(gt + gEC + 16 * (n < 2 ? qa : qb) + 8 * (n & 1) + 2 * t);
                U[n][0] *= e2.x, U[n][1] *= e2.y, U[n][2] *= e2.x, U[n][3] *= e2.y;
            }
            const float em = put_gated(ef, U, qa, qb, lane);
            if (lane == 0) sh.e_max[2 * cg + hf] = em;
            tc::barrier(1 + cg, 64);

            // the half's S^T <- exp(G_C) S^T + (exp(G_C - G) U)^T K
            const float eC = gt[gEG + C - 1];
            float ei;
            const float es = scale_for(fmaxf(sh.e_max[2 * cg], sh.e_max[2 * cg + 1]), ei);
            ei *= ui;
            uint32_t uh[4][4], ul[4][4];
            get_gated(ef, es, lane, uh, ul);
            float m[4] = {0.f, 0.f, 0.f, 0.f};
            constexpr int D = KH < 4 ? KH : 4;
#pragma unroll
            for (int d = 0; d < KH; d += D) {
                float acc[8][4];
                state_product<D>(acc, uh, ul, sK, hf * KH + d, lane);
#pragma unroll
                for (int i = 0; i < 2 * D; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        S[2 * d + i][e] = fmaf(ei, acc[i][e], eC * S[2 * d + i][e]);
                        m[e] = fmaxf(m[e], fabsf(S[2 * d + i][e]));
                    }
            }
            release(sh.ea + c % NA, lane);
            m_own = warp_max(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
        }
        if (a.final_state) write_state(S, a.final_state + sb, a.dv, col0 + g, t);
        return;
    }

    // the helper; the first one also feeds the stages
    const int hk = h / (a.H / a.Hk);
    const size_t kc0 = ((size_t)b * a.Hk + hk) * a.nc;
    const bool feeds = w == 2 * CG && lane == 0;
    int to_a = 0, to_b = 0;
    if (feeds)
        for (int c = 0; c < NA - 1 && c < n_chunks; c++) load_a<Pl, DK>(sh, a, kc0 + c, ch0 + c, c, wait, to_a);
    if (MODE != kKeep && feeds)
        for (int c = 0; c < NB - 1 && c < n_chunks; c++) load_b<Pl, DK>(sh, a, kc0 + c, ch0 + c, c, wait, to_b);
    for (int c = 0; c < n_chunks; c++) {
        if (feeds) {
            const int na = c + NA - 1, nb = c + NB - 1;
            if (MODE != kKeep && nb < n_chunks) load_b<Pl, DK>(sh, a, kc0 + nb, ch0 + nb, nb, wait, to_b);
            if (na < n_chunks) load_a<Pl, DK>(sh, a, kc0 + na, ch0 + na, na, wait, to_a);
        }
        wait.together();
        if (MODE == kKeep && w < 3 * CG) continue;  // only feeds
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
                if (lane < 2) rf[fS + lane] = sh.s_inv[2 * cg + lane];
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
            // O^T = s_q (exp(G) S^T Q^T + U^T P^T)
            uint8_t* st = sh.sm + Pl::oB + (c % NB) * Pl::B;
            const uint32_t sQ = tc::smem_u32(st), sP = sQ + Pl::oP;
            const float* gt = reinterpret_cast<const float*>(st + Pl::bGate);
            float O[8][4];
            zero(O);
            wait(sh.fb + c % NB, c / NB);
            wait(sh.s_ready + cg, c);
            // The halves have their own scales.  The smaller one's goes first: its sums
            // shrink to the larger one's units, where the other way round they could
            // pass fp32's range.
            const float s0 = sh.s_inv[2 * cg], s1 = sh.s_inv[2 * cg + 1], si = fmaxf(s0, s1);
            const int first = s0 <= s1 ? 0 : KK / 2;
#pragma unroll 4
            for (int i = 0; i < KK; i++) {
                if (i == KK / 2) {
                    const float f = fminf(s0, s1) / si;
#pragma unroll
                    for (int n = 0; n < 8; n++)
#pragma unroll
                        for (int e = 0; e < 4; e++) O[n][e] *= f;
                }
                const int kk = i ^ first;
                uint32_t hi[4], lo[4];
                get4(sf + kk * 512, hi, lane);
                get4(sf + Pl::sHalf + kk * 512, lo, lane);
                uint32_t bq[4][4];
#pragma unroll
                for (int p = 0; p < 4; p++) ldsm4(bq[p], at_n(sQ, 16 * p, 2 * kk, lane));
                mma_row<0, 4>(O, hi, bq);
                mma_row<0, 4>(O, lo, bq);
            }
            signal(sh.s_free + cg, lane);
            wait(sh.u_ready + cg, c);
            const float ui = sh.u_inv[cg];
            // in units of U's tiles, so that both products share an accumulator
            scale_tokens(O, gt + gEG, si / ui, t);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t uh[4], ul[4];
                get4(uf + j * 512, uh, lane);
                get4(uf + Pl::uHalf + j * 512, ul, lane);
#pragma unroll
                for (int p = j; p < 4; p++) {
                    uint32_t ph[4];
                    ldsm4(ph, at_n(sP, 16 * p, 2 * j, lane));
                    {
                        uint32_t pl[4];
                        ldsm4(pl, at_n(sP + kTile, 16 * p, 2 * j, lane));
                        mma(O[2 * p], ul, ph[0], ph[1]);
                        mma(O[2 * p + 1], ul, ph[2], ph[3]);
                        mma(O[2 * p], uh, pl[0], pl[1]);
                        mma(O[2 * p + 1], uh, pl[2], pl[3]);
                    }
                    mma(O[2 * p], uh, ph[0], ph[1]);
                    mma(O[2 * p + 1], uh, ph[2], ph[3]);
                }
            }
            scale_tokens(O, gt + gSq, ui, t);
            release(sh.eb + c % NB, lane);
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
    }
    if (feeds) settle<Pl>(sh, to_a, to_b);
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
    constexpr int NA = Pl::NA, NB = Pl::NB, KK = DK / 16;
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

    if (w < 2 * CG) {
        constexpr int KH = KK / 2;
        const int hf = w / CG, qa = hf, qb = 3 - hf;
        const size_t sb = (((size_t)b * a.H + h) * DK + hf * (DK / 2)) * a.dv;
        float S[DK / 16][4];
        read_state(S, dfinal ? dfinal + sb : nullptr, a.dv, col0 + g, t);
        float m_own = tiles_max(S);
        uint8_t *xf = ex + Pl::oX, *ef = ex + Pl::oE;
        // R of quarter q, in its owner's part of the exchange of X: quarters 0, 3, 1, 2
        auto rf = [&](int q) { return xf + 1024 * (q == 0 ? 0 : q == 3 ? 1 : q == 1 ? 2 : 3); };
        for (int it = 0; it < n_chunks; it++) {
            uint8_t* st = sh.sm + (it % NA) * Pl::A;
            const uint32_t sK = tc::smem_u32(st), sT = sK + Pl::oT;
            const float* gt = reinterpret_cast<const float*>(st + Pl::aGate);

            // the half's dS^T K^T
            float si;
            const float ss = scale_for(m_own, si);
            float X[8][4];
            zero(X);
            wait(sh.fa + it % NA, it / NA);
            if (it > 0) wait(sh.s_free + cg, it - 1);
#pragma unroll
            for (int kk = 0; kk < KH; kk++) {
                uint32_t hi[4], lo[4];
                split_a(S[2 * kk], S[2 * kk + 1], ss, hi, lo);
                put4(sf + (hf * KH + kk) * 512, hi, lane);
                put4(sf + Pl::sHalf + (hf * KH + kk) * 512, lo, lane);
                uint32_t bk[4][4];
#pragma unroll
                for (int p = 0; p < 4; p++) ldsm4(bk[p], at_n(sK, 16 * p, 2 * (hf * KH + kk), lane));
                mma_row<0, 4>(X, lo, bk);
                mma_row<0, 4>(X, hi, bk);
            }
            if (lane == 0) {
                sh.s_inv[2 * cg + hf] = si;
                sh.s_max[2 * cg + hf] = m_own;
            }
            signal(sh.s_ready + cg, lane);
            float U[4][4];
            hand_over(xf, X, hf, si, lane, U);
            wait(sh.z_ready + cg, it);
            tc::barrier(1 + cg, 64);
            take_over(xf, hf, lane, U);
            const float bound = fmaxf(sh.v_max[2 * cg], fmaxf(sh.s_max[2 * cg], sh.s_max[2 * cg + 1])) *
                                fmaxf(1.f, fmaxf(gt[gMax], gt[gMax + 1]));
            float ui;
            const float us = bound_scale(bound, ui);
#pragma unroll
            for (int n = 0; n < 4; n++) {
                const int tile = 2 * (n < 2 ? qa : qb) + (n & 1);
                const float2 e2 = *reinterpret_cast<const float2*>(gt + gEC + 8 * tile + 2 * t);
                const float4 d = df[32 * tile];
                U[n][0] = fmaf(U[n][0], e2.x, d.x), U[n][1] = fmaf(U[n][1], e2.y, d.y);
                U[n][2] = fmaf(U[n][2], e2.x, d.z), U[n][3] = fmaf(U[n][3], e2.y, d.w);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                uint32_t hi[4], lo[4];
                const int q = i ? qb : qa;
                split_a(U[2 * i], U[2 * i + 1], us, hi, lo);
                put4(rf(q), hi, lane);
                put4(rf(q) + 512, lo, lane);
            }
            tc::barrier(1 + cg, 64);

            // Y^T = dU^T T: token j takes i >= j
            float Y[4][4];
            zero(Y);
#pragma unroll
            for (int pass = 0; pass < 2; pass++)  // the small products, then the large ones
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (i < qa) continue;
                    uint32_t uh[4], ul[4], th[2][4], tl[2][4];
                    get4(rf(i), uh, lane);
                    if (pass == 0) get4(rf(i) + 512, ul, lane);
#pragma unroll
                    for (int k = 0; k < 2; k++)
                        if (!k || i >= qb) {
                            ldsm4_t(th[k], at_k(sT, 16 * i, 2 * (k ? qb : qa), lane));
                            if (pass == 0) ldsm4_t(tl[k], at_k(sT + kTile, 16 * i, 2 * (k ? qb : qa), lane));
                        }
#pragma unroll
                    for (int m = pass * 2; m < 2 + pass; m++)
#pragma unroll
                        for (int k = 0; k < 2; k++)
                            if (!k || i >= qb) {
                                const uint32_t(&x)[4] = m == 1 ? tl[k] : th[k];
                                mma(Y[2 * k], m == 0 ? ul : uh, x[0], x[1]);
                                mma(Y[2 * k + 1], m == 0 ? ul : uh, x[2], x[3]);
                            }
                }
            if (it > 0) wait(sh.u_free + cg, it - 1);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                uint32_t hi[4], lo[4];
                const int q = i ? qb : qa;
                split_a(Y[2 * i], Y[2 * i + 1], 1.f, hi, lo);
                put4(uf + q * 512, hi, lane);
                put4(uf + Pl::uHalf + q * 512, lo, lane);
            }
            if (lane == 0 && hf == 0) sh.u_inv[cg] = ui;
            signal(sh.u_ready + cg, lane);
#pragma unroll
            for (int n = 0; n < 4; n++) {
                const int at = 16 * (n < 2 ? qa : qb) + 8 * (n & 1) + 2 * t;
                const float2 eg = *reinterpret_cast<const float2*>(gt + gEG + at);
                const float2 bt = *reinterpret_cast<const float2*>(gt + gBeta + at);
                Y[n][0] *= -eg.x * bt.x, Y[n][1] *= -eg.y * bt.y, Y[n][2] *= -eg.x * bt.x, Y[n][3] *= -eg.y * bt.y;
            }
            const float em = put_gated(ef, Y, qa, qb, lane);
            if (lane == 0) sh.e_max[2 * cg + hf] = em;
            tc::barrier(1 + cg, 64);

            // the half's dS^T <- exp(G_C) dS^T + Z - (exp(G) beta' Y)^T K
            const float eC = gt[gEG + C - 1];
            float ei;
            const float es = scale_for(fmaxf(sh.e_max[2 * cg], sh.e_max[2 * cg + 1]), ei);
            ei *= ui;
            uint32_t yh[4][4], yl[4][4];
            get_gated(ef, es, lane, yh, yl);
            float m[4] = {0.f, 0.f, 0.f, 0.f};
            constexpr int D = KH < 4 ? KH : 4;
#pragma unroll
            for (int d = 0; d < KH; d += D) {
                float acc[8][4];
                state_product<D>(acc, yh, yl, sK, hf * KH + d, lane);
#pragma unroll
                for (int i = 0; i < 2 * D; i++) {
                    const float4 z4 = zf[32 * (2 * (hf * KH + d) + i)];
                    const float z[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        S[2 * d + i][e] = fmaf(ei, acc[i][e], fmaf(eC, S[2 * d + i][e], z[e]));
                        m[e] = fmaxf(m[e], fabsf(S[2 * d + i][e]));
                    }
                }
            }
            signal(sh.z_free + cg, lane);
            release(sh.ea + it % NA, lane);
            m_own = warp_max(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
        }
        if (dinitial) write_state(S, dinitial + sb, a.dv, col0 + g, t);
        return;
    }

    const bool keeps = col0 < a.dv;
    if (w >= 3 * CG) {  // the chain's tiles of every chunk into its record
        for (int it = 0; it < n_chunks; it++) {
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
                if (lane < 2) rf[fDs + lane] = sh.s_inv[2 * cg + lane];
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
        return;
    }
    const int hk = h / (a.H / a.Hk);
    const size_t kc0 = ((size_t)b * a.Hk + hk) * a.nc;
    const bool feeds = w == 2 * CG && lane == 0;
    int to_a = 0, to_b = 0;
    auto load = [&](int na, int nb) {
        if (na < n_chunks) load_a<Pl, DK>(sh, a, kc0 + n_chunks - 1 - na, ch0 + n_chunks - 1 - na, na, wait, to_a);
        if (nb < n_chunks) load_b<Pl, DK>(sh, a, kc0 + n_chunks - 1 - nb, ch0 + n_chunks - 1 - nb, nb, wait, to_b);
    };
    if (feeds) {
        for (int it = 0; it < NB - 1; it++) load(n_chunks, it);
        for (int it = 0; it < NA - 1; it++) load(it, n_chunks);
    }
    const Rows orows = rows_at(a.dout, a, b, h, col0 + 8 * (lane & 1), len);
    uint4 on[4];
    if (n_chunks)
#pragma unroll
        for (int i = 0; i < 4; i++) on[i] = orows.load((n_chunks - 1) * C + 16 * i + (lane >> 1));
    for (int it = 0; it < n_chunks; it++) {
        if (feeds) {  // the helper's own first: the chain's may wait for the chain
            load(n_chunks, it + NB - 1);
            load(it + NA - 1, n_chunks);
        }
        wait.together();
        {  // dO' of this chunk: its record's tile, dU0 and Z
            const int c = n_chunks - 1 - it;
            uint8_t* st = sh.sm + Pl::oB + (it % NB) * Pl::B;
            const uint32_t sQ = tc::smem_u32(st), sP = sQ + Pl::oP;
            const float* gt = reinterpret_cast<const float*>(st + Pl::bGate);
            uint8_t* rec = a.records + ((ch0 + c) * groups_of(a.dv) + group) * Record<DK>::bytes;
            float* rf = reinterpret_cast<float*>(rec + Record<DK>::f);
            float o[8][4];
            wait(sh.fb + it % NB, it / NB);
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
            for (int k = 1; k >= 0; k--)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int d = 0; d <= i; d++) {
                        uint32_t b[4];
                        ldsm4_t(b, at_k(sP + k * kTile, 16 * i, 2 * d, lane));
                        mma(U[2 * d], oh[i], b[0], b[1]);
                        mma(U[2 * d + 1], oh[i], b[2], b[3]);
                    }
            scale_tokens(o, gt + gEG, 1.f, t);
            float zi;  // of the gated rows: behind a strong decay far below dO'
            const float zs = tiles_scale(o, zi);
#pragma unroll
            for (int i = 0; i < 4; i++) split_a(o[2 * i], o[2 * i + 1], zs, oh[i], ol[i]);
            const float um = tiles_max(U) * oi;
            if (it > 0) wait(sh.z_free + cg, it - 1);
#pragma unroll
            for (int n = 0; n < 8; n++) df[32 * n] = make_float4(U[n][0] * oi, U[n][1] * oi, U[n][2] * oi, U[n][3] * oi);
            // Z^T = (exp(G) dO')^T Q
#pragma unroll 1
            for (int d = 0; d < KK; d += 4) {
                float acc[8][4];
                state_product<4>(acc, oh, ol, sQ, d, lane);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    zf[32 * (2 * d + i)] = make_float4(acc[i][0] * zi, acc[i][1] * zi, acc[i][2] * zi, acc[i][3] * zi);
            }
            if (lane == 0) sh.v_max[2 * cg] = um;
            signal(sh.z_ready + cg, lane);
            release(sh.eb + it % NB, lane);
        }
    }
    if (feeds) settle<Pl>(sh, to_a, to_b);
}

// ------------------------------------------------------------------ kernels

template <int DK, int CG, int MODE>
__global__ void __launch_bounds__(Plan<DK, CG, MODE>::warps * 32, 1) k_delta_chain(const __grid_constant__ ChainArgs a) {
    wait_previous();
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
    return launch_after(k_delta_chain<DK, CG, MODE>, grid, Pl::warps * 32, Pl::smem, s, "delta rule: chain", c);
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
    // (Set up beside the kernel before, as the forward's chain is, this one and the
    // next took a third longer on 1 x 4096 x 16 x 128 x 128: 689 us against 526.)
    k_delta_chains<DK, CG><<<grid, Plan<DK, CG, kBack>::warps * 32, smem, s>>>(c, a.dfinal_state, a.dinitial_state);
    return check_launch("delta rule: the backward's chains");
}
template <int DK>
ret_status chains_dk(const DeltaArgs& a, const ChainArgs& c, cudaStream_t s) {
    // two groups share the tiles where they leave no SM idle: 1 x 4096, 16 heads of
    // 128 / 128, the whole backward 550 us, with one group 666
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
