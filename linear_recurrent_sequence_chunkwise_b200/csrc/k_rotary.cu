// k_rotary.cu -- rotary positions on q and k: pair p of a row at position n is
// turned by n * f_p and multiplied by `scale`,
//     [a', b'] = scale [a cos - b sin, a sin + b cos],
// where the pair is (2p, 2p+1) (interleaved) or (p, p + r/2) (half), r the
// turned part of the head; the other d - r components are copied.  The
// transpose (the gradient) turns by -n f_p.
//
// Bound by memory: every element is read and written once.  A warp takes one
// token and walks its heads; a lane stays on the same pairs of every head, so
// their sines and cosines, computed once per (token, pair), sit in registers
// and a head costs its loads, its products and its stores, eight vectors in
// flight.  The angle is a 64-bit product reduced to [-pi, pi] (a far position
// times a frequency has no exact digits left in 32 bits).
// 8192 tokens x 32 heads of 256 in bf16, 268 MB: 46 us (a block per token with
// the table in shared memory, read again for every head: 133 us; this form with
// a branch around each load, which then waits for it: 108 us).
#include <algorithm>

#include "kernels.h"

namespace ret {

namespace {

constexpr int kRotWarps = 4;    // warps of a block, one token each
constexpr int kRotLoads = 8;    // vectors in flight in a lane

struct RotFreqs {
    double f[kMaxRotaryDim / 2];
};

template <typename T, int V>
struct alignas(sizeof(T) * V == 16 ? 16 : alignof(T)) Pack {
    T e[V];
};

// V elements, aligned to V * sizeof(T).
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> ld_pack(const T* p) {
    Pack<T, V> r;
    if constexpr (sizeof(T) * V == 16) {
        *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) r.e[i] = p[i];
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void st_pack(T* p, const Pack<T, V>& r) {
    if constexpr (sizeof(T) * V == 16) {
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) p[i] = r.e[i];
    }
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// A row (token, head) is cut into units: V elements of each half of the turned
// part (half layout, `parts` = 2) or V consecutive elements (interleaved); what
// follows the turned part is cut the same way and copied.  turned = units that
// rotate, units = all of a row.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kRotWarps * 32) k_rotary(RotaryArgs a, const __grid_constant__ RotFreqs fr, int tokens,
                                                          int units, int turned, int rows_split) {
    constexpr int PARTS = HALF ? 2 : 1, kRotUnroll = kRotLoads / PARTS;
    constexpr int PV = HALF ? V : (V + 1) / 2;  // pairs of a unit
    __shared__ float2 table[kRotWarps][kMaxRotaryDim / 2];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int tok = (int)blockIdx.x * kRotWarps + w;
    if (tok >= tokens) return;  // no barrier of the block below
    const int b = tok / a.N, n = tok - b * a.N;
    const int r2 = a.rotary_dim / 2, rows = a.H + a.Hk;
    const int row0 = (int)((long long)rows * blockIdx.y / rows_split);
    const int row1 = (int)((long long)rows * (blockIdx.y + 1) / rows_split);
    float2* cs = table[w];
    const long long pos = a.positions ? (long long)a.positions[tok] : a.pos_offset + n;
    for (int p = lane; p < r2; p += 32) {
        float s, c;
        sincosf(rot_angle(pos, fr.f[p]), &s, &c);
        cs[p] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
    }
    __syncwarp();

    const T* q = reinterpret_cast<const T*>(a.q.p) + b * a.q.sb + n * a.q.sn;
    const T* k = reinterpret_cast<const T*>(a.k.p) + b * a.k.sb + n * a.k.sn;
    T* qo = reinterpret_cast<T*>(a.qo.p) + b * a.qo.sb + n * a.qo.sn;
    T* ko = reinterpret_cast<T*>(a.ko.p) + b * a.ko.sb + n * a.ko.sn;
    const int width = min(units, 32), heads = 32 / width;  // lanes of a row, rows of a warp
    if (lane >= width * heads) return;
    for (int un = lane % width; un < units; un += width) {
        const bool turn = un < turned;
        const int c = turn ? un * V : a.rotary_dim + (un - turned) * V;
        const int second = turn ? r2 : (a.d - a.rotary_dim) / 2;  // distance of the second part
        float2 t[PV];
#pragma unroll
        for (int i = 0; i < PV; i++) t[i] = turn ? cs[HALF ? c + i : c / 2 + i] : make_float2(1.f, 0.f);
        for (int r = row0 + lane / width; r < row1; r += kRotUnroll * heads) {
            Pack<T, V> x[kRotUnroll][PARTS];
#pragma unroll
            for (int u = 0; u < kRotUnroll; u++) {
                const int row = min(r + u * heads, row1 - 1);  // no branch around a load
                const T* src = (row < a.H ? q + row * a.q.sh : k + (row - a.H) * a.k.sh) + c;
#pragma unroll
                for (int i = 0; i < PARTS; i++) x[u][i] = ld_pack<T, V>(src + i * second);
            }
#pragma unroll
            for (int u = 0; u < kRotUnroll; u++) {
                const int row = r + u * heads;
                if (row >= row1) continue;
                if (turn) {
#pragma unroll
                    for (int i = 0; i < PV; i++) {
                        T& lo = HALF ? x[u][0].e[i] : x[u][0].e[2 * i];
                        T& hi = HALF ? x[u][PARTS - 1].e[i] : x[u][0].e[(2 * i + 1) % V];
                        const float f = to_f(lo), g = to_f(hi);
                        from_f(lo, f * t[i].x - g * t[i].y);
                        from_f(hi, f * t[i].y + g * t[i].x);
                    }
                }
                T* dst = (row < a.H ? qo + row * a.qo.sh : ko + (row - a.H) * a.ko.sh) + c;
#pragma unroll
                for (int i = 0; i < PARTS; i++) st_pack<T, V>(dst + i * second, x[u][i]);
            }
        }
    }
}

template <typename T, int V, bool HALF>
void launch(const RotaryArgs& a, const RotFreqs& fr, cudaStream_t s) {
    const int unit = HALF ? 2 * V : V;
    const int units = a.d / unit, turned = a.rotary_dim / unit;
    const int rows = a.H + a.Hk, heads = 32 / std::min(units, 32);
    const long long tokens = (long long)a.B * a.N, blocks = (tokens + kRotWarps - 1) / kRotWarps;
    // Few tokens: a token's heads go to several warps, each with its own
    // sines, until there are eight warps for each of the 148 SMs.
    const long long want = 8 * 148 / tokens;
    const int split = (int)std::max<long long>(1, std::min<long long>((rows + heads - 1) / heads, want));
    k_rotary<T, V, HALF><<<dim3((unsigned)blocks, split), kRotWarps * 32, 0, s>>>(a, fr, (int)tokens, units, turned, split);
}

}  // namespace

ret_status launch_rotary(const RotaryArgs& a, const double* freqs, cudaStream_t s) {
    RotFreqs fr;
    for (int p = 0; p < a.rotary_dim / 2; p++) fr.f[p] = freqs[p];
    for (int p = a.rotary_dim / 2; p < kMaxRotaryDim / 2; p++) fr.f[p] = 0.0;
    const int es = a.dt == RET_F32 ? 4 : 2, V = 16 / es;
    // 16-byte accesses need whole vectors in every part of the row and
    // 16-byte rows in every view; else element by element.
    const int unit = a.half ? 2 * V : V;
    bool wide = a.rotary_dim % unit == 0 && a.d % unit == 0;
    const RotaryView* views[4] = {&a.q, &a.qo, a.Hk ? &a.k : nullptr, a.Hk ? &a.ko : nullptr};
    for (const RotaryView* v : views)
        if (v) wide = wide && aligned(v->p, 16) && v->sb % V == 0 && v->sn % V == 0 && v->sh % V == 0;
    if (a.dt == RET_F32) {
        if (wide) a.half ? launch<float, 4, true>(a, fr, s) : launch<float, 4, false>(a, fr, s);
        else a.half ? launch<float, 1, true>(a, fr, s) : launch<float, 2, false>(a, fr, s);
    } else {
        if (wide) a.half ? launch<__nv_bfloat16, 8, true>(a, fr, s) : launch<__nv_bfloat16, 8, false>(a, fr, s);
        else a.half ? launch<__nv_bfloat16, 1, true>(a, fr, s) : launch<__nv_bfloat16, 2, false>(a, fr, s);
    }
    return check_launch("ret_rotary");
}

}  // namespace ret
