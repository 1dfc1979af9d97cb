// The transition forward for a few rows (one token and up), in groups of at most 8:
// bound by reading the weights, so the work is spread by weight rows over every SM
// instead of by row tiles.  Two kernels: H, a warp a feature (both projections, the activation
// and the product), then Y, one to eight warps a channel.  X and H lie in shared
// memory in fp32: nothing is rounded before Y.  The second kernel starts beside the
// first (programmatic dependent launch) and has its first weights on their way
// before it waits for H.  One row, C = 384, F = 1536, bf16: 5.8 us a call in a replayed
// graph for 3.5 MB of weights (L2 holds them: two launches and two rounds of L2
// latency are the rest), 15 us called from Python, which the host's side bounds.
#pragma once

#include "transition_common.cuh"

namespace evo {

constexpr int kTrFewThreads = 256;
constexpr int kTrFewRows = 8;              // most rows of a group (grid y: groups)
constexpr int kTrFewBytes = 128 * 1024;    // most bytes of X or H in shared memory

template <typename T>
struct TrFewParams {
    const T *x, *wg, *wu, *wd;
    T* y;
    float* h;  // [M, F]
    int M, C, F;
    int split;  // warps of a channel: 1, 2, 4 or 8
};

template <typename T>
__device__ __forceinline__ float tr_f32(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
    else return __bfloat162float(v);
}

// VE weights from p: 16 bytes at once, or one
template <typename T, int VE>
__device__ __forceinline__ void tr_few_load(const T* p, float (&w)[VE]) {
    if constexpr (VE == 1) {
        w[0] = tr_f32(*p);
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int e = 0; e < VE; ++e) w[e] = tr_f32(t[e]);
    }
}

template <typename T, int ACT, int MB, int VE>
__global__ void __launch_bounds__(kTrFewThreads) evo_tr_few_gate_kernel(const TrFewParams<T> p) {
    extern __shared__ __align__(16) float few_smem[];  // [MB][C]
    // first the wait: the kernel after this one reads weights before its own wait, so it
    // may start only once every kernel before this one has ended
    ptx::pdl_wait();
    ptx::pdl_launch();
    const int m0 = blockIdx.y * MB, M = min(MB, p.M - m0);
    const T* x = p.x + (long long)m0 * p.C;
    float* h = p.h + (long long)m0 * p.F;
    for (int i = threadIdx.x; i < MB * p.C; i += kTrFewThreads) few_smem[i] = i < M * p.C ? tr_f32(x[i]) : 0.0f;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int f = (blockIdx.x * kTrFewThreads + threadIdx.x) >> 5; f < p.F; f += gridDim.x * (kTrFewThreads / 32)) {
        const T *wg = p.wg + (long long)f * p.C, *wu = p.wu + (long long)f * p.C;
        float g[MB] = {}, u[MB] = {};
#pragma unroll 2
        for (int c = lane * VE; c < p.C; c += 32 * VE) {
            float a[VE], b[VE];
            tr_few_load<T, VE>(wg + c, a);
            tr_few_load<T, VE>(wu + c, b);
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float xv = few_smem[m * p.C + c + e];
                    g[m] = fmaf(xv, a[e], g[m]);
                    u[m] = fmaf(xv, b[e], u[m]);
                }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                g[m] += __shfl_xor_sync(0xffffffffu, g[m], o);
                u[m] += __shfl_xor_sync(0xffffffffu, u[m], o);
            }
            if (lane == m && m < M) h[(long long)m * p.F + f] = tr_act<ACT>(g[m]) * u[m];
        }
    }
}

template <typename T, int MB, int VE>
__global__ void __launch_bounds__(kTrFewThreads) evo_tr_few_out_kernel(const TrFewParams<T> p) {
    extern __shared__ __align__(16) float few_smem[];  // [MB][F]
    __shared__ float part[kTrFewThreads / 32][MB];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = (kTrFewThreads / 32) / p.split;  // channels at once
    const int sub = warp % p.split, c = blockIdx.x * per + warp / p.split;
    const T* wd = p.wd + (long long)min(c, p.C - 1) * p.F;
    const int step = 32 * VE * p.split;
    int f = (sub * 32 + lane) * VE;
    float w[VE] = {};
    ptx::pdl_launch();
    if (f < p.F) tr_few_load<T, VE>(wd + f, w);  // no result of the kernel before
    ptx::pdl_wait();
    const int m0 = blockIdx.y * MB, M = min(MB, p.M - m0);
    const float* h = p.h + (long long)m0 * p.F;
    T* out = p.y + (long long)m0 * p.C;
    for (int i = threadIdx.x; i < MB * p.F; i += kTrFewThreads) few_smem[i] = i < M * p.F ? h[i] : 0.0f;
    __syncthreads();
    float y[MB] = {};
    while (f < p.F) {
        float next[VE] = {};
        if (f + step < p.F) tr_few_load<T, VE>(wd + f + step, next);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int e = 0; e < VE; ++e) y[m] = fmaf(few_smem[m * p.F + f + e], w[e], y[m]);
#pragma unroll
        for (int e = 0; e < VE; ++e) w[e] = next[e];
        f += step;
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) y[m] += __shfl_xor_sync(0xffffffffu, y[m], o);
        if (lane == 0) part[warp][m] = y[m];
    }
    __syncthreads();
    if (threadIdx.x < per * MB) {
        const int k = threadIdx.x / MB, m = threadIdx.x % MB, ck = blockIdx.x * per + k;
        float s = 0.0f;
        for (int i = 0; i < p.split; ++i) s += part[k * p.split + i][m];
        if (ck < p.C && m < M) {
            if constexpr (sizeof(T) == 4) out[(long long)m * p.C + ck] = s;
            else tr_store(out + (long long)m * p.C + ck, s);
        }
    }
}

}  // namespace evo
