// k_layernorm.cu -- layer norm over the last dimension and its gradients.
//     y = (x - mean) rstd gain + bias,  rstd = 1 / sqrt(var + eps)   (biased variance)
//     with h = (x - mean) rstd and t = dy gain:
//     dx = rstd (t - avg(t) - h avg(t h)),  dgain = sum_rows dy h,  dbias = sum_rows dy
//
// The bytes (x, dy read once, y, dx written once) are the floor, the
// instructions are close behind: on 2,048 bf16 columns a sum over the threads
// of a row costs a warp as much as eight elements of each of its lanes.  So a
// lane takes 16 elements of a row (the backward: of its two inputs, with the
// weights and two columns' sums), and a group of 32 to 512 threads the row.  The
// groups walk the rows with the next one's loads in flight.  The forward takes
// the variance about the mean (two reductions), which keeps rows with a large
// mean exact.
//
// The backward's column sums: a group keeps its columns' partial sums of dgain
// and dbias in registers; the groups of a block add theirs in shared memory,
// every block writes one partial row, and a second kernel adds those in a fixed
// order (the result does not depend on timing).  Sums are fp32, those of the partial
// rows 64-bit: a column's longest chain of fp32 additions is a group's rows and a
// block's groups.
//
// 8192 x 2048 bf16: forward 16.5 us (a warp to a row, 64 elements in a lane: 24
// us; eight warps, 8 elements: 28 us), backward 23 + 4 us for the columns (eight
// warps, 8 elements: 39 us).
#include <algorithm>
#include <atomic>

#include "kernels.h"

namespace ret {

namespace {

constexpr int kBwdElems = 16;    // elements of a row in a thread of the backward
constexpr int kBwdMost = 512;    // threads of a block of the backward
constexpr int kBwdBlocks = 296;  // most blocks of the backward, and so partial rows
constexpr int kSms = 148;

__device__ __forceinline__ float f_of(float x) { return x; }
__device__ __forceinline__ float f_of(__nv_bfloat16 x) { return __bfloat162float(x); }

// VEC consecutive elements as they lie in memory; VEC * sizeof(T) is 16
// (aligned) or VEC is 1.  A load behind the row's end reads the row's last
// elements instead and is cleared where it is used: a branch around a load
// waits for the load where it ends.
template <typename T, int VEC>
struct alignas(VEC == 1 ? sizeof(T) : 16) Raw {
    T e[VEC];
    __device__ __forceinline__ void keep_if(bool in) {
        if constexpr (VEC == 1) {
            if (!in) st_from_float(e, 0, 0.f);
        } else {
            uint4& u = *reinterpret_cast<uint4*>(e);
            if (!in) u = make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC == 1) e[0] = p[0];
        else *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
    }
};
// Elements 2 i and 2 i + 1 of an array in its own dtype.
__device__ __forceinline__ float2 pair_of(const float* e, int i) { return make_float2(e[2 * i], e[2 * i + 1]); }
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* e, int i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(e)[i];
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T, int VEC, int NV>
__device__ __forceinline__ float2 pair_of(const Raw<T, VEC> (&r)[NV], int p) {
    if constexpr (VEC == 1) return make_float2(f_of(r[2 * p].e[0]), f_of(r[2 * p + 1].e[0]));
    else return pair_of(r[2 * p / VEC].e, p % (VEC / 2));
}
template <typename W, int VEC, int NV>
__device__ __forceinline__ float2 pair_of(const W (&w)[NV][VEC], int p) {
    if constexpr (VEC == 1) return make_float2(f_of(w[2 * p][0]), f_of(w[2 * p + 1][0]));
    else return pair_of(w[2 * p / VEC], p % (VEC / 2));
}
// VEC elements from the pairs at f, rounded once.
template <typename T, int VEC>
__device__ __forceinline__ void st_vec(T* p, const float2* f) {
    static_assert(VEC > 1, "");
    uint4 u;
    if constexpr (sizeof(T) == 4) {
        u = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].x, f[i].y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(p) = u;
}
// The row's elements from the thread's pairs.
template <typename T, int VEC, int NV, bool FULL>
__device__ __forceinline__ void st_row(T* p, const float2 (&f)[VEC * NV / 2], int d, int group, int lane) {
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = (i * group + lane) * VEC;
        if (FULL || c < d) {
            if constexpr (VEC == 1) st_from_float(p, c, i & 1 ? f[i / 2].y : f[i / 2].x);
            else st_vec<T, VEC>(p + c, f + i * VEC / 2);
        }
    }
}
// VEC weights at column c, in their own dtype (kept so in registers).
template <typename W, int VEC>
__device__ __forceinline__ void ld_w(const W* w, int c, W* f) {
    if constexpr (VEC * sizeof(W) >= 16) {
#pragma unroll
        for (int i = 0; i < VEC; i += 16 / (int)sizeof(W))
            *reinterpret_cast<uint4*>(f + i) = *reinterpret_cast<const uint4*>(w + c + i);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i++) f[i] = w[c + i];
    }
}

// Sums over the T threads of a group; every thread gets them.  `red`: words of
// the group (zero at the start for `one`), alternating between two halves so that one
// barrier per sum is enough.  `bar`: the group's named barrier, 0 for a group
// that is the block (a block with a variable one holds 16 of an SM's 64
// barriers: four blocks).
__host__ __device__ constexpr int red_words(int T) { return (T / 32 + 3) / 4 * 4; }
struct GroupSum {
    float* red;  // two halves, 16-byte aligned
    int T, bar, half;
    // For a group of a warp or of the whole block.
    __device__ __forceinline__ float one(float x) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (T == 32) return x;
        const int n = red_words(T);
        float* r = next(n);
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = x;
        __syncthreads();
        float4 t = *reinterpret_cast<const float4*>(r);
        for (int i = 4; i < n; i += 4) {
            const float4 u = *reinterpret_cast<const float4*>(r + i);
            t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
        }
        return (t.x + t.y) + (t.z + t.w);
    }
    // Two sums: half of the lanes goes on with each.
    __device__ __forceinline__ float2 two(float x, float y) {
        const bool up = threadIdx.x & 16;
        float s = (up ? y : x) + __shfl_xor_sync(0xffffffffu, up ? x : y, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (T == 32) {
            const float other = __shfl_xor_sync(0xffffffffu, s, 16);
            return up ? make_float2(other, s) : make_float2(s, other);
        }
        const int nw = T / 32;
        float* r = next(2 * nw);
        if ((threadIdx.x & 15) == 0) r[(threadIdx.x % T) >> 4] = s;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(T) : "memory");
        float2 t = *reinterpret_cast<const float2*>(r);
        for (int i = 1; i < nw; i++) {
            const float2 u = *reinterpret_cast<const float2*>(r + 2 * i);
            t.x += u.x, t.y += u.y;
        }
        return t;
    }
    __device__ __forceinline__ float* next(int n) {
        float* r = red + half * n;
        half ^= 1;
        return r;
    }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ unsigned long long u64(float2 x) { return *reinterpret_cast<unsigned long long*>(&x); }
__device__ __forceinline__ float2 f2(unsigned long long x) { return *reinterpret_cast<float2*>(&x); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(u64(a)), "l"(u64(b)), "l"(u64(c)));
    return f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(u64(a)), "l"(u64(b)));
    return f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(u64(a)), "l"(u64(b)));
    return f2(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// FULL: the group's loads cover the row exactly and both weights are given.
// A group is a warp or the block.
template <typename T, typename W, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(512) k_ln_forward(const T* __restrict__ x, const W* __restrict__ gain,
                                                   const W* __restrict__ bias, T* __restrict__ y,
                                                   float* __restrict__ mean_out, float* __restrict__ rstd_out,
                                                   long long rows, int d, float eps, int group) {
    constexpr int P = VEC * NV / 2;
    __shared__ __align__(16) float red[2 * red_words(512)];
    const int gi = threadIdx.x / group, lane = threadIdx.x % group, ng = blockDim.x / group;
    GroupSum sum{red, group, 0, 0};
    if (threadIdx.x < 2 * red_words(512)) red[threadIdx.x] = 0.f;  // before the first sum's barrier by its own writers
    if (group > 32) __syncthreads();
    const float inv_d = 1.f / d;
    const long long stride = (long long)gridDim.x * ng;
    Raw<T, VEC> raw[NV];
    const T* xr = x + (long long)(blockIdx.x * ng + gi) * d;  // of the row whose loads come next
    auto load = [&](bool there) {  // the last row again where there is none: no branch around a load
        if (!there) xr = x + (rows - 1) * d;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * group + lane) * VEC;
            raw[i].load(xr + (FULL ? c : min(c, d - VEC)));
        }
        xr += stride * d;
    };
    // behind the row's end: zero
    auto inside = [&](float2 f, int p) {
        if (!FULL) {
            if ((2 * p / VEC * group + lane) * VEC >= d) f.x = 0.f;
            if (((2 * p + 1) / VEC * group + lane) * VEC >= d) f.y = 0.f;
        }
        return f;
    };
    long long row = (long long)blockIdx.x * ng + gi;
    load(row < rows);
    for (; row < rows; row += stride) {
        float2 f[P], s = both(0.f), v = s;
#pragma unroll
        for (int p = 0; p < P; p++) {
            f[p] = inside(pair_of<T, VEC, NV>(raw, p), p);
            s = add2(s, f[p]);
        }
        load(row + stride < rows);
        const float mean = sum.one(s.x + s.y) * inv_d;
        const float2 m2 = both(-mean);
#pragma unroll
        for (int p = 0; p < P; p++) {
            f[p] = inside(add2(f[p], m2), p);
            v = fma2(f[p], f[p], v);
        }
        const float rstd = rsqrtf(sum.one(v.x + v.y) * inv_d + eps);  // good to 2 units
        if (lane == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
        const float2 r2 = both(rstd);
        alignas(16) W g[NV][VEC], b[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * group + lane) * VEC, at = FULL ? c : min(c, d - VEC);
            if (FULL || gain) ld_w<W, VEC>(gain, at, g[i]);
            if (FULL || bias) ld_w<W, VEC>(bias, at, b[i]);
        }
#pragma unroll
        for (int p = 0; p < P; p++) {
            f[p] = mul2(f[p], r2);
            if (FULL) {
                f[p] = fma2(f[p], pair_of<W, VEC, NV>(g, p), pair_of<W, VEC, NV>(b, p));
            } else {
                if (gain) f[p] = mul2(f[p], pair_of<W, VEC, NV>(g, p));
                if (bias) f[p] = add2(f[p], pair_of<W, VEC, NV>(b, p));
            }
        }
        st_row<T, VEC, NV, FULL>(y + row * d, f, d, group, lane);
    }
}

// part: [gridDim.x][2][d] column sums of each block, or null.
// FULL: the group's loads cover the row exactly and a gain is given.
template <typename T, typename W, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kBwdMost) k_ln_backward(const T* __restrict__ dy, const T* __restrict__ x,
                                                         const float* __restrict__ mean_in,
                                                         const float* __restrict__ rstd_in, const W* __restrict__ gain,
                                                         T* __restrict__ dx, float* __restrict__ part, long long rows,
                                                         int d, int group) {
    constexpr int E = VEC * NV, P = E / 2;
    launch_next();
    // the next row's loads in flight, where they fit the registers
    constexpr bool kAhead = (FULL && sizeof(T) == 2) || E == 8;
    __shared__ __align__(8) float red[64];
    extern __shared__ float cols[];  // [2][group * E]: the block's column sums
    const int gi = threadIdx.x / group, lane = threadIdx.x % group, ng = blockDim.x / group;
    GroupSum sum{red + gi * 4 * (group / 32), group, 1 + gi, 0};
    const long long stride = (long long)gridDim.x * ng;
    long long row = (long long)blockIdx.x * ng + gi;
    // element e of the thread: column ((e / VEC) * group + lane) * VEC + e % VEC
    alignas(16) W g[NV][VEC];
    float2 ag[P], ab[P];
    Raw<T, VEC> nx[NV], ny[NV];
    float nm = 0.f, nr = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++) st_from_float(&g[i][e], 0, 1.f);
    auto load = [&](long long r) {
        if (r >= rows) return;
        nm = mean_in[r];
        nr = rstd_in[r];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * group + lane) * VEC, at = FULL ? c : min(c, d - VEC);
            nx[i].load(x + r * d + at);
            ny[i].load(dy + r * d + at);
        }
    };
    if (kAhead) load(row);
#pragma unroll
    for (int p = 0; p < P; p++) ag[p] = ab[p] = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = (i * group + lane) * VEC;
        if (FULL || (gain && c < d)) ld_w<W, VEC>(gain, c, g[i]);
    }
    const float inv_d = 1.f / d;
    for (; row < rows; row += stride) {
        if (!kAhead) load(row);
        const float rstd = nr;
        const float2 r2 = both(nr), m2 = both(-nm);
        float2 h[P], t[P], sx = both(0.f), sy = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (!FULL) ny[i].keep_if((i * group + lane) * VEC < d);  // so every sum stays as it is
#pragma unroll
        for (int p = 0; p < P; p++) {
            h[p] = mul2(add2(pair_of<T, VEC, NV>(nx, p), m2), r2);
            t[p] = pair_of<T, VEC, NV>(ny, p);
            ag[p] = fma2(t[p], h[p], ag[p]);
            ab[p] = add2(ab[p], t[p]);
            if (FULL || gain) t[p] = mul2(t[p], pair_of<W, VEC, NV>(g, p));
            sx = add2(sx, t[p]);
            sy = fma2(t[p], h[p], sy);
        }
        if (kAhead) load(row + stride);
        const float2 s = sum.two(sx.x + sx.y, sy.x + sy.y);
        if (dx) {
            // rstd (t - c0 - h c1)
            const float2 c0 = both(-s.x * inv_d * rstd), c1 = both(-s.y * inv_d * rstd);
#pragma unroll
            for (int p = 0; p < P; p++) t[p] = fma2(t[p], r2, fma2(h[p], c1, c0));
            st_row<T, VEC, NV, FULL>(dx + row * d, t, d, group, lane);
        }
    }
    if (!part) return;
    // the groups of the block add their columns one after the other
    const int width = group * E;
    const float *fg = reinterpret_cast<const float*>(ag), *fb = reinterpret_cast<const float*>(ab);
    for (int k = 0; k < ng; k++) {
        __syncthreads();
        if (gi == k) {
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const int c = (i * group + lane) * VEC + e;
                    cols[c] = k ? cols[c] + fg[i * VEC + e] : fg[i * VEC + e];
                    cols[width + c] = k ? cols[width + c] + fb[i * VEC + e] : fb[i * VEC + e];
                }
        }
    }
    __syncthreads();
    float* mine = part + (size_t)blockIdx.x * 2 * d;
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
        mine[c] = cols[c];
        mine[d + c] = cols[width + c];
    }
}

// Adds the partial rows: a block takes 32 columns, warp w the partial rows
// w, w + 32, ... (all loads of a thread in flight), then the warps' sums in order; in
// 64 bits, which costs nothing beside the loads.
constexpr int kColWarps = 32;
__global__ void __launch_bounds__(kColWarps * 32) k_ln_columns(const float* __restrict__ part, int parts, int d,
                                                              float* __restrict__ dgain, float* __restrict__ dbias) {
    __shared__ double s[kColWarps][33];
    wait_previous();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, n = 2 * d;
    double t = 0.0;
    if (c < n) {
        constexpr int kLoads = (kBwdBlocks + kColWarps - 1) / kColWarps;
        float x[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int p = w + i * kColWarps;
            x[i] = p < parts ? part[(size_t)p * n + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kLoads; i++) t += x[i];
    }
    s[w][lane] = t;
    __syncthreads();
    if (w == 0 && c < n) {
        t = 0.0;
#pragma unroll
        for (int i = 0; i < kColWarps; i++) t += s[i][lane];
        float* out = c < d ? dgain : dbias;
        if (out) out[c < d ? c : c - d] = (float)t;
    }
}

// The group of threads of a row: the smallest of 32, 64, ... that holds it.
int group_for(int d, int elems) {
    int t = 32;
    while (t * elems < d) t *= 2;
    return t;
}

bool wide_rows(const LayerNormArgs& a) {
    const int V = a.dt == RET_F32 ? 4 : 8;
    bool ok = a.d % V == 0;
    for (const void* p : {a.x, (const void*)a.y, a.gain, a.bias, a.dy, (const void*)a.dx})
        ok = ok && (!p || aligned(p, 16));
    return ok;
}

template <typename T, typename W, int VEC, int ELEMS>
ret_status fwd_go(const LayerNormArgs& a, cudaStream_t s) {
    const int group = group_for(a.d, ELEMS), threads = group == 32 ? 128 : group, ng = threads / group;
    // The blocks that fit at once walk the rows.  How many is a matter of the form's
    // registers (64 to 128 a thread) and asked for once: with 1,024 threads an SM for
    // every form some had a second, short round of blocks (8192 x 2000 bf16: 24.2 us
    // instead of 20.7; where all of them fit, 8192 x 2048, no difference).
    auto go = [&](auto kern, bool full) -> ret_status {
        static std::atomic<int> known[2][5];
        int size = 0;  // of the group: 32 << size
        while (32 << size < group) size++;
        std::atomic<int>& fit = known[full][size];
        int an_sm = fit.load(std::memory_order_relaxed);
        if (!an_sm) {
            const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&an_sm, kern, threads, 0);
            if (e != cudaSuccess) return fail(RET_ERR_CUDA, "ret_layernorm_forward: %s", cudaGetErrorString(e));
            fit.store(an_sm, std::memory_order_relaxed);
        }
        const unsigned blocks = (unsigned)std::min<long long>((long long)kSms * an_sm, (a.rows + ng - 1) / ng);
        kern<<<blocks, threads, 0, s>>>((const T*)a.x, (const W*)a.gain, (const W*)a.bias, (T*)a.y, a.mean, a.rstd, a.rows,
                                        a.d, (float)a.eps, group);
        return check_launch("ret_layernorm_forward");
    };
    if constexpr (VEC > 1)
        if (a.d == group * ELEMS && a.gain && a.bias) return go(k_ln_forward<T, W, VEC, ELEMS / VEC, true>, true);
    return go(k_ln_forward<T, W, VEC, ELEMS / VEC, false>, false);
}
template <typename T, typename W>
ret_status fwd(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    if (!wide_rows(a)) return fwd_go<T, W, 1, 16>(a, s);
    return fwd_go<T, W, V, 16>(a, s);
}

template <typename T, typename W>
ret_status bwd(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    // element by element eight in a thread leave room for the next row's loads
    const bool wide = wide_rows(a);
    const int elems = wide || a.d > 8 * kBwdMost ? kBwdElems : 8, group = group_for(a.d, elems);
    // Few large blocks when there are rows for all of them (fewer partial rows
    // to write and add), small ones to spread few rows.
    const bool many = a.rows >= (long long)kSms * (kBwdMost / group);
    const int threads = many ? kBwdMost : std::max(128, group), ng = threads / group;
    const int blocks = (int)std::min<long long>(many ? kSms : kBwdBlocks, (a.rows + ng - 1) / ng);
    float* part = a.dgain || a.dbias ? (float*)a.workspace : nullptr;
    const size_t smem = part ? (size_t)2 * group * elems * sizeof(float) : 0;  // at most 64 KB
    auto go = [&](auto kern) -> ret_status {
        if (smem > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return fail(RET_ERR_CUDA, "ret_layernorm_backward: %s", cudaGetErrorString(e));
        }
        kern<<<blocks, threads, smem, s>>>((const T*)a.dy, (const T*)a.x, a.mean, a.rstd, (const W*)a.gain, (T*)a.dx, part,
                                           a.rows, a.d, group);
        return check_launch("ret_layernorm_backward");
    };
    ret_status st = !wide ? (elems == 8 ? go(k_ln_backward<T, W, 1, 8, false>) : go(k_ln_backward<T, W, 1, kBwdElems, false>))
                    : a.d == group * kBwdElems && a.gain ? go(k_ln_backward<T, W, V, kBwdElems / V, true>)
                                                         : go(k_ln_backward<T, W, V, kBwdElems / V, false>);
    if (st != RET_OK || !part) return st;
    return launch_after(k_ln_columns, dim3((2 * a.d + 31) / 32), kColWarps * 32, 0, s, "ret_layernorm_backward: columns", part, blocks, a.d,
                        a.dgain, a.dbias);
}

}  // namespace

size_t layernorm_bwd_workspace_bytes(long long rows, int d) {
    return (size_t)std::min<long long>(kBwdBlocks, rows) * 2 * d * sizeof(float);
}

ret_status launch_layernorm_forward(const LayerNormArgs& a, cudaStream_t s) {
    if (a.dt == RET_F32) return a.w_dt == RET_F32 ? fwd<float, float>(a, s) : fwd<float, __nv_bfloat16>(a, s);
    return a.w_dt == RET_F32 ? fwd<__nv_bfloat16, float>(a, s) : fwd<__nv_bfloat16, __nv_bfloat16>(a, s);
}

ret_status launch_layernorm_backward(const LayerNormArgs& a, cudaStream_t s) {
    if (a.dt == RET_F32) return a.w_dt == RET_F32 ? bwd<float, float>(a, s) : bwd<float, __nv_bfloat16>(a, s);
    return a.w_dt == RET_F32 ? bwd<__nv_bfloat16, float>(a, s) : bwd<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace ret
