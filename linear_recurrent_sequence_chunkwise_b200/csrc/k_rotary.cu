// k_rotary.cu -- rotary positions on q and k: pair p of a row at position n is
// turned by n * f_p and multiplied by `scale`,
//     [a', b'] = scale [a cos - b sin, a sin + b cos],
// where the pair is (2p, 2p+1) (interleaved) or (p, p + r/2) (half), r the
// turned part of the head; the other d - r components are copied.  The
// transpose (the gradient) turns by -n f_p.
//
// Bound by memory: every element is read and written once.  The angle is a
// 64-bit product reduced to [-pi, pi] (a far position times a frequency has
// no exact digits left in 32 bits); its sine and cosine are computed once per
// (token, pair) into shared memory and serve every head of q and k.  A block
// takes about 1,024 16-byte vectors (so a thread has four loads in flight
// over the sine pass) of one or several tokens.
#include <algorithm>

#include "kernels.h"

namespace ret {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotUnroll = 4;
constexpr int kRotTable = 4096;  // (cos, sin) pairs of a block's tokens: 32 KB

struct RotFreqs {
    double f[kMaxRotaryDim / 2];
};

template <typename T, int V>
struct Pack {
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

// A row (token, head) is cut into units: V consecutive elements of the two
// halves (half layout), 2V consecutive elements (interleaved), or 2V elements
// to copy.  turned = units that rotate, units = all of a row.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kRotThreads) k_rotary(RotaryArgs a, const __grid_constant__ RotFreqs fr, int tokens,
                                                       int tb, int units, int turned, int rows_split) {
    __shared__ float2 cs[kRotTable];
    const int r2 = a.rotary_dim / 2;
    const int rows = a.H + a.Hk;
    const int row0 = (int)((long long)rows * blockIdx.y / rows_split);
    const int row1 = (int)((long long)rows * (blockIdx.y + 1) / rows_split);
    const int per_token = (row1 - row0) * units;
    const int t0 = (int)blockIdx.x * tb;
    const int nt = min(tb, tokens - t0);
    const int items = nt * per_token;

    Pack<T, V> x[kRotUnroll], y[kRotUnroll];
    T* dst[kRotUnroll];
    int off2[kRotUnroll];  // distance of the unit's second part from its first
    int tab[kRotUnroll];   // table index of its first pair, -1: copy

    auto locate = [&](int it, int u, const T*& src) {
        const int tl = it / per_token, rem = it - tl * per_token;
        const int row = row0 + rem / units, un = rem % units;
        const int tok = t0 + tl;
        const int b = tok / a.N, n = tok - b * a.N;
        int c;
        if (un < turned) {
            c = HALF ? un * V : 2 * un * V;
            off2[u] = HALF ? r2 : V;
            tab[u] = tl * r2 + un * V;
        } else {
            c = a.rotary_dim + 2 * (un - turned) * V;
            off2[u] = V;
            tab[u] = -1;
        }
        const bool isq = row < a.H;
        const int h = isq ? row : row - a.H;
        const RotaryView& vi = isq ? a.q : a.k;
        const RotaryView& vo = isq ? a.qo : a.ko;
        src = reinterpret_cast<const T*>(vi.p) + b * vi.sb + n * vi.sn + h * vi.sh + c;
        dst[u] = reinterpret_cast<T*>(vo.p) + b * vo.sb + n * vo.sn + h * vo.sh + c;
    };
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kRotUnroll; u++) {
            const int it = base + u * kRotThreads + threadIdx.x;
            if (it < items) {
                const T* src;
                locate(it, u, src);
                x[u] = ld_pack<T, V>(src);
                y[u] = ld_pack<T, V>(src + off2[u]);
            }
        }
    };
    auto finish = [&](int base) {
#pragma unroll
        for (int u = 0; u < kRotUnroll; u++) {
            const int it = base + u * kRotThreads + threadIdx.x;
            if (it >= items) continue;
            if (tab[u] >= 0) {
                if constexpr (HALF) {
#pragma unroll
                    for (int i = 0; i < V; i++) {
                        const float2 t = cs[tab[u] + i];
                        const float p = to_f(x[u].e[i]), q = to_f(y[u].e[i]);
                        from_f(x[u].e[i], p * t.x - q * t.y);
                        from_f(y[u].e[i], p * t.y + q * t.x);
                    }
                } else {
                    // the 2V consecutive elements hold V pairs
#pragma unroll
                    for (int i = 0; i < V; i++) {
                        T& lo = 2 * i < V ? x[u].e[(2 * i) % V] : y[u].e[(2 * i) % V];
                        T& hi = 2 * i + 1 < V ? x[u].e[(2 * i + 1) % V] : y[u].e[(2 * i + 1) % V];
                        const float2 t = cs[tab[u] + i];
                        const float p = to_f(lo), q = to_f(hi);
                        from_f(lo, p * t.x - q * t.y);
                        from_f(hi, p * t.y + q * t.x);
                    }
                }
            }
            st_pack<T, V>(dst[u], x[u]);
            st_pack<T, V>(dst[u] + off2[u], y[u]);
        }
    };

    load(0);
    for (int i = threadIdx.x; i < nt * r2; i += kRotThreads) {
        const int tl = i / r2, p = i - tl * r2;
        const int tok = t0 + tl;
        const long long pos = a.positions ? (long long)a.positions[tok] : a.pos_offset + tok % a.N;
        float s, c;
        sincosf(rot_angle(pos, fr.f[p]), &s, &c);
        cs[i] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
    }
    __syncthreads();
    finish(0);
    for (int base = kRotUnroll * kRotThreads; base < items; base += kRotUnroll * kRotThreads) {
        load(base);
        finish(base);
    }
}

template <typename T, int V, bool HALF>
void launch(const RotaryArgs& a, const RotFreqs& fr, cudaStream_t s) {
    const int units = a.d / (2 * V), turned = a.rotary_dim / (2 * V);
    const int rows = a.H + a.Hk;
    const long long tokens = (long long)a.B * a.N;
    const int want = kRotUnroll * kRotThreads / 2;  // units of two vectors: the block's share
    int tb = std::max(1, want / (rows * units));
    tb = std::max(1, std::min(tb, kRotTable / (a.rotary_dim / 2)));
    // Few tokens: a token's heads go to several blocks, each with its own
    // sines, until there are two blocks for each of the 148 SMs.
    long long blocks = (tokens + tb - 1) / tb;
    int split = 1;
    if (blocks < 296) {
        tb = 1;
        blocks = tokens;
        split = (int)std::min<long long>(rows, std::max<long long>(1, 296 / blocks));
    }
    k_rotary<T, V, HALF><<<dim3((unsigned)blocks, split), kRotThreads, 0, s>>>(a, fr, (int)tokens, tb, units, turned,
                                                                             split);
}

}  // namespace

ret_status launch_rotary(const RotaryArgs& a, const double* freqs, cudaStream_t s) {
    RotFreqs fr;
    for (int p = 0; p < a.rotary_dim / 2; p++) fr.f[p] = freqs[p];
    for (int p = a.rotary_dim / 2; p < kMaxRotaryDim / 2; p++) fr.f[p] = 0.0;
    const int es = a.dt == RET_F32 ? 4 : 2, V = 16 / es;
    // 16-byte accesses need whole vectors in every part of the row and
    // 16-byte rows in every view; else element by element.
    bool wide = a.rotary_dim % (2 * V) == 0 && a.d % (2 * V) == 0;
    const RotaryView* views[4] = {&a.q, &a.qo, a.Hk ? &a.k : nullptr, a.Hk ? &a.ko : nullptr};
    for (const RotaryView* v : views)
        if (v) wide = wide && aligned(v->p, 16) && v->sb % V == 0 && v->sn % V == 0 && v->sh % V == 0;
    if (a.dt == RET_F32) {
        if (wide) a.half ? launch<float, 4, true>(a, fr, s) : launch<float, 4, false>(a, fr, s);
        else a.half ? launch<float, 1, true>(a, fr, s) : launch<float, 1, false>(a, fr, s);
    } else {
        if (wide) a.half ? launch<__nv_bfloat16, 8, true>(a, fr, s) : launch<__nv_bfloat16, 8, false>(a, fr, s);
        else a.half ? launch<__nv_bfloat16, 1, true>(a, fr, s) : launch<__nv_bfloat16, 1, false>(a, fr, s);
    }
    return check_launch("ret_rotary");
}

}  // namespace ret
