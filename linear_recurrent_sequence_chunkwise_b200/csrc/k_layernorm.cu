// k_layernorm.cu -- layer norm over the last dimension and its gradients.
//     y = (x - mean) rstd gain + bias,  rstd = 1 / sqrt(var + eps)   (biased variance)
//     with h = (x - mean) rstd and t = dy gain:
//     dx = rstd (t - avg(t) - h avg(t h)),  dgain = sum_rows dy h,  dbias = sum_rows dy
//
// Bound by memory: x (and dy) are read once and y (dx) written once.  A row is
// held in the registers of a group of T threads, the smallest power of two
// (32 to 1,024) whose 16-byte vectors cover it; a group of one warp needs no
// barrier, a larger one a named barrier of its own, so the groups of a block
// run apart.  The forward takes the variance about the mean (two reductions),
// which keeps rows with a large mean exact.
//
// The backward's column sums: a group walks many rows and keeps its columns'
// partial sums of dgain and dbias in registers, the groups of a block add
// theirs in shared memory, every block writes one partial row, and a second
// kernel adds those in a fixed order (the result does not depend on timing).
// All sums are fp32.
#include <algorithm>

#include "kernels.h"

namespace ret {

namespace {

__device__ __forceinline__ float f_of(float x) { return x; }
__device__ __forceinline__ float f_of(__nv_bfloat16 x) { return __bfloat162float(x); }

// VEC consecutive elements as fp32; VEC * sizeof(T) is 16 (aligned) or VEC is 1.
template <typename T, int VEC>
__device__ __forceinline__ void ld_vec(const T* p, float* f) {
    if constexpr (VEC == 1) {
        f[0] = f_of(p[0]);
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int i = 0; i < VEC; i++) f[i] = f_of(e[i]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void st_vec(T* p, const float* f) {
    if constexpr (VEC == 1) {
        st_from_float(p, 0, f[0]);
    } else {
        uint4 u;
        T* e = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int i = 0; i < VEC; i++) st_from_float(e, i, f[i]);
        *reinterpret_cast<uint4*>(p) = u;
    }
}
// VEC weights at column c (their own dtype; not necessarily 16-byte wide).
template <typename W, int VEC>
__device__ __forceinline__ void ld_w(const W* w, int c, float* f) {
    if constexpr (VEC * sizeof(W) >= 16) {
#pragma unroll
        for (int i = 0; i < VEC; i += 16 / (int)sizeof(W)) ld_vec<W, 16 / (int)sizeof(W)>(w + c + i, f + i);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i++) f[i] = f_of(w[c + i]);
    }
}

// Sum over the T threads of a group; every thread gets it.  `red`: the
// group's 32 words, alternating between two halves so that one barrier per
// sum is enough.
struct GroupSum {
    float2* red;  // [2][T / 32]
    int T, bar, half;
    __device__ __forceinline__ float2 operator()(float2 x) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        }
        if (T == 32) return x;
        const int nw = T / 32, w = (threadIdx.x % T) >> 5;
        float2* r = red + half * nw;
        half ^= 1;
        if ((threadIdx.x & 31) == 0) r[w] = x;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(T) : "memory");
        float2 s = r[0];
        for (int i = 1; i < nw; i++) {
            s.x += r[i].x;
            s.y += r[i].y;
        }
        return s;
    }
};

template <typename T, typename W, int VEC, int NV>
__global__ void __launch_bounds__(1024) k_ln_forward(const T* __restrict__ x, const W* __restrict__ gain,
                                                    const W* __restrict__ bias, T* __restrict__ y,
                                                    float* __restrict__ mean_out, float* __restrict__ rstd_out,
                                                    long long rows, int d, float eps, int group) {
    __shared__ float2 red[64];
    const int gi = threadIdx.x / group, lane = threadIdx.x % group, ng = blockDim.x / group;
    const long long row = (long long)blockIdx.x * ng + gi;
    if (row >= rows) return;  // the whole group
    GroupSum sum{red + gi * 2 * (group / 32), group, 1 + gi, 0};
    const T* xr = x + row * d;
    float f[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = (i * group + lane) * VEC;
        if (c < d) {
            ld_vec<T, VEC>(xr + c, f[i]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; e++) f[i][e] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++) s += f[i][e];
    const float mean = sum(make_float2(s, 0.f)).x / d;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if ((i * group + lane) * VEC < d) {
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                f[i][e] -= mean;
                v = fmaf(f[i][e], f[i][e], v);
            }
        }
    const float rstd = 1.f / sqrtf(sum(make_float2(v, 0.f)).x / d + eps);
    if (lane == 0) {
        if (mean_out) mean_out[row] = mean;
        if (rstd_out) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = (i * group + lane) * VEC;
        if (c >= d) continue;
        float g[VEC], b[VEC];
        if (gain) ld_w<W, VEC>(gain, c, g);
        if (bias) ld_w<W, VEC>(bias, c, b);
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            float t = f[i][e] * rstd;
            if (gain) t *= g[e];
            if (bias) t += b[e];
            f[i][e] = t;
        }
        st_vec<T, VEC>(y + row * d + c, f[i]);
    }
}

// part: [gridDim.x][2][d] column sums of each block, or null.
template <typename T, typename W, int VEC, int NV>
__global__ void __launch_bounds__(512) k_ln_backward(const T* __restrict__ dy, const T* __restrict__ x,
                                                    const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                                                    const W* __restrict__ gain, T* __restrict__ dx,
                                                    float* __restrict__ part, long long rows, int d, int group) {
    __shared__ float2 red[32];
    extern __shared__ float cols[];  // [2][group * NV * VEC]: the block's column sums
    const int gi = threadIdx.x / group, lane = threadIdx.x % group, ng = blockDim.x / group;
    GroupSum sum{red + gi * 2 * (group / 32), group, 1 + gi, 0};
    float g[NV][VEC], ag[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = (i * group + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            g[i][e] = 1.f;
            ag[i][e] = ab[i][e] = 0.f;
        }
        if (gain && c < d) ld_w<W, VEC>(gain, c, g[i]);
    }
    const float inv_d = 1.f / d;
    for (long long row = (long long)blockIdx.x * ng + gi; row < rows; row += (long long)gridDim.x * ng) {
        const float mean = mean_in[row], rstd = rstd_in[row];
        float h[NV][VEC], t[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * group + lane) * VEC;
            if (c < d) {
                ld_vec<T, VEC>(x + row * d + c, h[i]);
                ld_vec<T, VEC>(dy + row * d + c, t[i]);
            }
        }
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if ((i * group + lane) * VEC < d) {
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    h[i][e] = (h[i][e] - mean) * rstd;
                    ag[i][e] = fmaf(t[i][e], h[i][e], ag[i][e]);
                    ab[i][e] += t[i][e];
                    t[i][e] *= g[i][e];
                    s.x += t[i][e];
                    s.y = fmaf(t[i][e], h[i][e], s.y);
                }
            }
        s = sum(s);
        const float c0 = s.x * inv_d, c1 = s.y * inv_d;
        if (dx) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = (i * group + lane) * VEC;
                if (c >= d) continue;
#pragma unroll
                for (int e = 0; e < VEC; e++) t[i][e] = rstd * (t[i][e] - c0 - h[i][e] * c1);
                st_vec<T, VEC>(dx + row * d + c, t[i]);
            }
        }
    }
    if (!part) return;
    // the groups of the block add their columns one after the other
    const int width = group * NV * VEC;
    for (int k = 0; k < ng; k++) {
        __syncthreads();
        if (gi == k) {
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const int c = (i * group + lane) * VEC + e;
                    cols[c] = k ? cols[c] + ag[i][e] : ag[i][e];
                    cols[width + c] = k ? cols[width + c] + ab[i][e] : ab[i][e];
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

// Adds the partial rows: a block takes 32 columns, its warps the partial rows
// w, w + 8, ..., then the warps' sums in order.
__global__ void __launch_bounds__(256) k_ln_columns(const float* __restrict__ part, int parts, int d,
                                                   float* __restrict__ dgain, float* __restrict__ dbias) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, n = 2 * d;
    float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
    if (c < n) {
        int p = w;
        for (; p + 24 < parts; p += 32) {
            a0 += part[(size_t)p * n + c];
            a1 += part[(size_t)(p + 8) * n + c];
            a2 += part[(size_t)(p + 16) * n + c];
            a3 += part[(size_t)(p + 24) * n + c];
        }
        for (; p < parts; p += 8) a0 += part[(size_t)p * n + c];
    }
    s[w][lane] = (a0 + a1) + (a2 + a3);
    __syncthreads();
    if (w == 0 && c < n) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) t += s[i][lane];
        float* out = c < d ? dgain : dbias;
        if (out) out[c < d ? c : c - d] = t;
    }
}

// The group of threads of a row: the smallest of 32, 64, ... 1,024 that
// holds it, 0 if none does.
int group_for(int d, int vec, int nv, int most) {
    for (int t = 32; t <= most; t *= 2)
        if ((long long)t * vec * nv >= d) return t;
    return 0;
}

constexpr int kFwdVec = 4, kFwdScalar = 8;  // loads of a thread of the forward
constexpr int kBwdElems = 16;               // elements of a thread of the backward
constexpr int kFwdMost = 1024, kBwdMost = 512;
// Blocks of the backward: two for each of the 148 SMs.
constexpr int kBwdBlocks = 296;

bool wide_rows(const LayerNormArgs& a) {
    const int V = a.dt == RET_F32 ? 4 : 8;
    bool ok = a.d % V == 0;
    for (const void* p : {a.x, (const void*)a.y, a.gain, a.bias, a.dy, (const void*)a.dx})
        ok = ok && (!p || aligned(p, 16));
    return ok;
}

struct BwdPlan {
    int group, threads, blocks;
};
BwdPlan bwd_plan(const LayerNormArgs& a, bool wide) {
    BwdPlan p;
    p.group = wide ? group_for(a.d, a.dt == RET_F32 ? 4 : 8, kBwdElems / (a.dt == RET_F32 ? 4 : 8), kBwdMost)
                   : group_for(a.d, 1, kBwdElems, kBwdMost);
    p.threads = std::max(256, p.group);
    const long long ng = p.group ? p.threads / p.group : 1;
    p.blocks = (int)std::min<long long>(kBwdBlocks, (a.rows + ng - 1) / ng);
    return p;
}

template <typename T, typename W>
ret_status fwd(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = wide_rows(a);
    int group = wide ? group_for(a.d, V, kFwdVec, kFwdMost) : group_for(a.d, 1, kFwdScalar, kFwdMost);
    const int threads = std::max(128, group), ng = threads / group;
    const long long blocks = (a.rows + ng - 1) / ng;
    if (wide)
        k_ln_forward<T, W, V, kFwdVec><<<(unsigned)blocks, threads, 0, s>>>(
            (const T*)a.x, (const W*)a.gain, (const W*)a.bias, (T*)a.y, a.mean, a.rstd, a.rows, a.d, (float)a.eps, group);
    else
        k_ln_forward<T, W, 1, kFwdScalar><<<(unsigned)blocks, threads, 0, s>>>(
            (const T*)a.x, (const W*)a.gain, (const W*)a.bias, (T*)a.y, a.mean, a.rstd, a.rows, a.d, (float)a.eps, group);
    return check_launch("ret_layernorm_forward");
}

template <typename T, typename W>
ret_status bwd(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = wide_rows(a);
    const BwdPlan p = bwd_plan(a, wide);
    float* part = a.dgain || a.dbias ? (float*)a.workspace : nullptr;
    const int width = p.group * kBwdElems;
    const size_t smem = part ? (size_t)2 * width * sizeof(float) : 0;  // at most 64 KB
    auto go = [&](auto kern) -> ret_status {
        if (smem > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return fail(RET_ERR_CUDA, "ret_layernorm_backward: %s", cudaGetErrorString(e));
        }
        kern<<<p.blocks, p.threads, smem, s>>>((const T*)a.dy, (const T*)a.x, a.mean, a.rstd, (const W*)a.gain, (T*)a.dx,
                                               part, a.rows, a.d, p.group);
        return check_launch("ret_layernorm_backward");
    };
    ret_status st = wide ? go(k_ln_backward<T, W, V, kBwdElems / V>) : go(k_ln_backward<T, W, 1, kBwdElems>);
    if (st != RET_OK || !part) return st;
    k_ln_columns<<<(2 * a.d + 31) / 32, 256, 0, s>>>(part, p.blocks, a.d, a.dgain, a.dbias);
    return check_launch("ret_layernorm_backward: columns");
}

}  // namespace

bool layernorm_fits(int d) { return d <= kLayerNormMaxDim; }

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
