// k_delta_step.cu -- the gated delta rule token by token: one decode step, and
// a whole sequence on the CUDA cores.  Per value head, S [dk, dv] fp32:
//     S' = exp(g) S,  u = beta (v - S'^T k),  S <- S' + k u^T,  o = S^T q.
// Both dot products run on the old state, so a step needs one reduction:
//     u = beta (v - a S^T k),  o = a S^T q + (q . k) u,  a = exp(g).
#include <algorithm>

#include "kernels.h"

namespace ret {

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
    float4* S = reinterpret_cast<float4*>(state + bh * dk * dv + c);
    const size_t ld = dv / 4;

    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int r = rl + i * RL;
        s[i] = live && r < dk ? __ldcs(S + (size_t)r * ld) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i = tid; i < kDeltaMaxDk; i += WARPS * 32) {
        ks[i] = i < dk ? ld_as_float(k, kb + i) : 0.f;
        qs[i] = i < dk ? ld_as_float(q, kb + i) : 0.f;
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

template <typename Tin, typename Tout>
void step(const DeltaArgs& a, float* state, cudaStream_t s) {
    const unsigned bh = (unsigned)(a.B * a.H), wide = (a.dv + 63) / 64, narrow = (a.dv + 15) / 16;
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
    if (a.in_dt == RET_F32) a.out_dt == RET_F32 ? step<float, float>(a, state, s) : step<float, __nv_bfloat16>(a, state, s);
    else a.out_dt == RET_F32 ? step<__nv_bfloat16, float>(a, state, s) : step<__nv_bfloat16, __nv_bfloat16>(a, state, s);
    return check_launch("ret_delta_decode_step");
}

ret_status launch_delta_recurrent(const DeltaArgs& a, cudaStream_t s) {
    if (a.in_dt == RET_F32) a.out_dt == RET_F32 ? recurrent<float, float>(a, s) : recurrent<float, __nv_bfloat16>(a, s);
    else a.out_dt == RET_F32 ? recurrent<__nv_bfloat16, float>(a, s) : recurrent<__nv_bfloat16, __nv_bfloat16>(a, s);
    return check_launch("ret_delta_forward_chunkwise: token by token");
}

}  // namespace ret
