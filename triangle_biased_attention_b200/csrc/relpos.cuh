// The learned relative-position bias: a pair bias looked up in a table by the
// bucket of the residue distance, and the table's gradient.
//
//     P[b, 0, h, i, j]  = table[r(b, i, j), h]  (+ base[b, 0, h, i, j])
//     dtable[r, h]      = sum of dP[b, 0, h, i, j] over the (b, i, j) with r(b, i, j) = r
//     r(b, i, j)        = the number of borders <= pos_q[b, i] - pos_k[b, j],
//                         or num_borders + 1 where the chains of i and j differ
//
// A thread owns eight key columns j and walks the query rows i, so the key
// positions stay in registers.  A distance finds its row in one shared-memory
// read when the borders span at most kRelLut - 2 distances (every distance between the
// first and the last border has an entry), else by a binary search in the
// borders.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "common.cuh"

namespace evo {

constexpr int kRelThreads = 256;      // forward
constexpr int kRelBwdThreads = 128;   // backward
constexpr int kRelCols = 8;           // key columns of a thread
constexpr int kRelLut = 2048;         // entries of the distance table
constexpr int kRelMaxBorders = 2048;
constexpr int kRelBins = 256;         // table rows that one backward block sums

template <typename T>
struct RelParams {
    const T* table;       // [rows, H]
    const int *borders, *pos_q, *pos_k, *chain_q, *chain_k;
    const T* base;        // [B, 1, H, Sq, Sk] or null
    T* pair;              // forward: written
    const T* dpair;       // backward: read
    float* part;          // backward: [tiles][H][rows] partial sums
    int B, Sq, Sk, H, nb, rows;
    int ti;               // query rows of a block
    int lane_cols;        // log2 of the threads along j
};

// difference of two positions, held at the ends of the 32-bit range
__device__ __forceinline__ int rel_distance(int q, int k) {
    int d;
    asm("sub.sat.s32 %0, %1, %2;" : "=r"(d) : "r"(q), "r"(k));
    return d;
}

// Distances to table rows, in shared memory.
struct RelLookup {
    const uint16_t* lut;
    const int* borders;
    int lo, last;  // first and last distance with an entry of its own in the lut
    int nb;
    bool direct;

    __device__ __forceinline__ int search(int d) const {
        int a = 0, n = nb;  // the answer lies in [a, a + n]
        while (n > 0) {
            const int half = n >> 1;
            if (borders[a + half] <= d) {
                a += half + 1;
                n -= half + 1;
            } else {
                n = half;
            }
        }
        return a;
    }
    __device__ __forceinline__ int row(int d) const {
        return direct ? int(lut[min(max(d, lo), last) - lo]) : search(d);
    }
};

// Fills the block's shared copies; every thread of the block calls it.
__device__ __forceinline__ RelLookup rel_setup(const int* __restrict__ borders, int nb, int* sborders, uint16_t* lut) {
    for (int i = threadIdx.x; i < nb; i += blockDim.x) sborders[i] = borders[i];
    __syncthreads();
    RelLookup L;
    L.borders = sborders;
    L.lut = lut;
    L.nb = nb;
    // one entry below the first border, one for each distance up to the last
    const long long first = nb > 0 ? sborders[0] : 0, last = nb > 0 ? sborders[nb - 1] : 0;
    const long long span = last - first + 2;
    L.direct = span >= 2 && span <= kRelLut && first > -2147483647ll;
    L.lo = L.direct ? int(first) - 1 : 0;
    L.last = int(last);
    if (L.direct)
        for (int e = threadIdx.x; e < int(span); e += blockDim.x) lut[e] = uint16_t(L.search(L.lo + e));
    __syncthreads();
    return L;
}

template <typename T>
__device__ __forceinline__ float rel_f32(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
    else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T rel_from(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// One block: `ti` query rows x 256 or more key columns x every head.
template <typename T>
__global__ void __launch_bounds__(kRelThreads) evo_relpos_fwd_kernel(const RelParams<T> p) {
    __shared__ int sborders[kRelMaxBorders];
    __shared__ uint16_t lut[kRelLut];
    const RelLookup L = rel_setup(p.borders, p.nb, sborders, lut);
    const int lanes = 1 << p.lane_cols, tx = threadIdx.x & (lanes - 1), ty = threadIdx.x >> p.lane_cols;
    const int b = blockIdx.z, j0 = blockIdx.x * lanes * kRelCols + tx;
    const int i_end = min(p.Sq, int(blockIdx.y + 1) * p.ti);
    int pk[kRelCols], ck[kRelCols];
#pragma unroll
    for (int e = 0; e < kRelCols; ++e) {
        const int j = j0 + e * lanes;
        pk[e] = j < p.Sk ? p.pos_k[(long long)b * p.Sk + j] : 0;
        ck[e] = j < p.Sk && p.chain_k ? p.chain_k[(long long)b * p.Sk + j] : 0;
    }
    for (int i = blockIdx.y * p.ti + ty; i < i_end; i += blockDim.x >> p.lane_cols) {
        const int pq = p.pos_q[(long long)b * p.Sq + i];
        const int cq = p.chain_q ? p.chain_q[(long long)b * p.Sq + i] : 0;
#pragma unroll
        for (int e = 0; e < kRelCols; ++e) {
            const int j = j0 + e * lanes;
            if (j >= p.Sk) continue;
            const int r = cq == ck[e] ? L.row(rel_distance(pq, pk[e])) : p.nb + 1;
            for (int h = 0; h < p.H; ++h) {
                const long long at = (((long long)b * p.H + h) * p.Sq + i) * p.Sk + j;
                const T t = p.table[(long long)r * p.H + h];
                p.pair[at] = p.base ? rel_from<T>(rel_f32(t) + rel_f32(p.base[at])) : t;
            }
        }
    }
}

// One block: `ti` query rows x 128 threads' key columns of one head, table rows
// [bin0, bin0 + kRelBins).  Each thread sums into its own column of shared
// memory, [bin][thread], so no two threads meet and the order of the additions
// is fixed; while a key column stays in one bucket its sum stays in a register.
template <typename T>
__global__ void __launch_bounds__(kRelBwdThreads) evo_relpos_bwd_kernel(const RelParams<T> p) {
    extern __shared__ float bins[];  // [min(rows - bin0, kRelBins)][128]
    __shared__ int sborders[kRelMaxBorders];
    __shared__ uint16_t lut[kRelLut];
    const int jt = blockIdx.x, itile = blockIdx.y;
    const int chunks = (p.rows + kRelBins - 1) / kRelBins;
    const int bin0 = (blockIdx.z % chunks) * kRelBins, nbins = min(kRelBins, p.rows - bin0);
    const int bh = blockIdx.z / chunks, b = bh / p.H, h = bh % p.H;
    for (int i = threadIdx.x; i < nbins * kRelBwdThreads; i += kRelBwdThreads) bins[i] = 0.0f;
    const RelLookup L = rel_setup(p.borders, p.nb, sborders, lut);
    const int lanes = 1 << p.lane_cols, tx = threadIdx.x & (lanes - 1), ty = threadIdx.x >> p.lane_cols;
    const int j0 = jt * lanes * kRelCols + tx, i_end = min(p.Sq, (itile + 1) * p.ti);
    int pk[kRelCols], ck[kRelCols], cur[kRelCols];
    float sum[kRelCols];
#pragma unroll
    for (int e = 0; e < kRelCols; ++e) {
        const int j = j0 + e * lanes;
        pk[e] = j < p.Sk ? p.pos_k[(long long)b * p.Sk + j] : 0;
        ck[e] = j < p.Sk && p.chain_k ? p.chain_k[(long long)b * p.Sk + j] : 0;
        cur[e] = -1;
        sum[e] = 0.0f;
    }
    auto flush = [&](int r, float s) {
        if (r >= bin0 && r < bin0 + nbins) bins[(r - bin0) * kRelBwdThreads + threadIdx.x] += s;
    };
    for (int i = itile * p.ti + ty; i < i_end; i += kRelBwdThreads >> p.lane_cols) {
        const int pq = p.pos_q[(long long)b * p.Sq + i];
        const int cq = p.chain_q ? p.chain_q[(long long)b * p.Sq + i] : 0;
        const T* row = p.dpair + ((long long)bh * p.Sq + i) * p.Sk;
        float v[kRelCols];
#pragma unroll
        for (int e = 0; e < kRelCols; ++e) v[e] = j0 + e * lanes < p.Sk ? rel_f32(row[j0 + e * lanes]) : 0.0f;
#pragma unroll
        for (int e = 0; e < kRelCols; ++e) {
            const int r = cq == ck[e] ? L.row(rel_distance(pq, pk[e])) : p.nb + 1;
            if (r != cur[e]) {
                flush(cur[e], sum[e]);
                cur[e] = r;
                sum[e] = 0.0f;
            }
            sum[e] += v[e];
        }
    }
#pragma unroll
    for (int e = 0; e < kRelCols; ++e) flush(cur[e], sum[e]);
    __syncthreads();
    // the 128 columns of each bin, a warp a bin, in a fixed order
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long tile = ((long long)b * gridDim.y + itile) * gridDim.x + jt;
    for (int r = warp; r < nbins; r += kRelBwdThreads / 32) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kRelBwdThreads / 32; ++k) s += bins[r * kRelBwdThreads + 32 * k + lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) p.part[(tile * p.H + h) * p.rows + bin0 + r] = s;
    }
}

// dtable[r, h] = the sum over the tiles, a warp an element, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256) evo_relpos_bwd_sum_kernel(const float* __restrict__ part, long long tiles, int H,
                                                                 int rows, T* __restrict__ dtable) {
    const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (w >= (long long)H * rows) return;
    const int h = int(w / rows), r = int(w % rows);
    float s = 0.0f;
    for (long long t = lane; t < tiles; t += 32) s += part[(t * H + h) * rows + r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) dtable[(long long)r * H + h] = rel_from<T>(s);
}

}  // namespace evo
