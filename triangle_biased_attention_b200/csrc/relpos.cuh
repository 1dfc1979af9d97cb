// The learned relative-position bias: a pair bias looked up in a table by the
// bucket of the residue distance, and the table's gradient.
//
//     P[b, 0, h, i, j]  = table[r(b, i, j), h]  (+ base[b, 0, h, i, j])
//     dtable[r, h]      = sum of dP[b, 0, h, i, j] over the (b, i, j) with r(b, i, j) = r
//     r(b, i, j)        = the number of borders <= pos_q[b, i] - pos_k[b, j],
//                         or num_borders + 1 where the chains of i and j differ
//
// A thread owns a few key columns j and walks the query rows i, so the key
// positions stay in registers.  A distance finds its row in one shared-memory
// read when the borders span at most kRelLut - 2 distances (every distance
// between the first and the last border has an entry), else by a binary search
// in the borders.  What they cannot do without is memory traffic: the forward
// writes P (and reads the base), the backward reads dP once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "common.cuh"

namespace evo {

constexpr int kRelThreads = 256;      // forward
constexpr int kRelCols = 8;           // key columns of a forward thread
constexpr int kRelBwdThreads = 128;   // backward
constexpr int kRelBwdCols = 8;        // key columns of a backward thread
constexpr int kRelBwdRows = 480;      // most query rows of a backward thread
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
    int jt, it;           // backward: tiles along j and along i
    int groups;           // forward: groups of heads
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
__device__ __forceinline__ RelLookup rel_setup(const int* borders, int nb, int* sborders, uint16_t* lut) {
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

// Shared memory of a block, in this order: the table rows or the sums, the
// borders, the distance table.
__host__ __device__ inline int rel_smem(int head_bytes, int nb) { return head_bytes + (nb + 3) / 4 * 16 + kRelLut * 2; }

// The pair (a, b) of 16-bit values at half `hi` of two words, as one word.
__device__ __forceinline__ uint32_t rel_halves(uint32_t a, uint32_t b, int hi) {
    return __byte_perm(a, b, hi ? 0x7632 : 0x5410);
}

// sum of two packed pairs (or two floats) in fp32, rounded to the type
template <typename T>
__device__ __forceinline__ uint32_t rel_add(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    } else if constexpr (std::is_same<T, __half>::value) {
        const float2 x = __half22float2(reinterpret_cast<const __half2&>(a));
        const float2 y = __half22float2(reinterpret_cast<const __half2&>(b));
        return ptx::pack_f16x2(x.x + y.x, x.y + y.y);
    } else {
        return ptx::pack_bf16x2(ptx::bf16lo_to_f32(a) + ptx::bf16lo_to_f32(b), ptx::bf16hi_to_f32(a) + ptx::bf16hi_to_f32(b));
    }
}

// One block: `ti` query rows x the key columns of its threads x a group of heads.
// The group's part of the table lies in shared memory, NW words a row (NW * 4 /
// sizeof(T) heads), so one read fetches a pair's value for every head of the
// group.  VEC: a thread's columns are 16 whole bytes of each head's row of P,
// written at once (the values of its columns are transposed in registers); else
// its columns lie the block's width apart and are written one by one.
// 2048 x 2048 x 8 heads, bf16, with a base: 30.9 us, 134 MB, 4.35 TB/s (L2 takes part of
// the writes); one shared-memory read for all heads instead of one each, and 16-byte
// writes, brought it from 254 us.  Its 683 blocks of 3 rows take 2.3 rounds, each with
// the tables to fill first (issue 39 %).
template <typename T, int NW, bool VEC>
__global__ void __launch_bounds__(kRelThreads, 2) evo_relpos_fwd_kernel(const RelParams<T> p) {
    constexpr int HEADS = NW * 4 / int(sizeof(T));
    constexpr int COLS = VEC ? 16 / int(sizeof(T)) : kRelCols;
    extern __shared__ __align__(16) uint8_t rel_sm[];
    ptx::pdl_launch();
    ptx::pdl_wait();
    T* stable = reinterpret_cast<T*>(rel_sm);
    int* sborders = reinterpret_cast<int*>(rel_sm + (p.rows * NW * 4 + 15) / 16 * 16);
    uint16_t* lut = reinterpret_cast<uint16_t*>(sborders + (p.nb + 3) / 4 * 4);
    const int b = blockIdx.z / p.groups, h0 = (blockIdx.z % p.groups) * HEADS, nh = min(HEADS, p.H - h0);
    for (int i = threadIdx.x; i < p.rows * HEADS; i += kRelThreads) {
        const int r = i / HEADS, h = i % HEADS;
        stable[i] = h < nh ? p.table[(long long)r * p.H + h0 + h] : rel_from<T>(0.0f);
    }
    const RelLookup L = rel_setup(p.borders, p.nb, sborders, lut);
    const int lanes = 1 << p.lane_cols, tx = threadIdx.x & (lanes - 1), ty = threadIdx.x >> p.lane_cols;
    const int j0 = blockIdx.x * lanes * COLS + (VEC ? tx * COLS : tx), step = VEC ? 1 : lanes;
    const int i_end = min(p.Sq, int(blockIdx.y + 1) * p.ti);
    int pk[COLS], ck[COLS];
#pragma unroll
    for (int e = 0; e < COLS; ++e) {
        const int j = j0 + e * step;
        pk[e] = j < p.Sk ? p.pos_k[(long long)b * p.Sk + j] : 0;
        ck[e] = j < p.Sk && p.chain_k ? p.chain_k[(long long)b * p.Sk + j] : 0;
    }
    if (j0 >= p.Sk) return;
    const long long plane = (long long)p.Sq * p.Sk;
    for (int i = blockIdx.y * p.ti + ty; i < i_end; i += kRelThreads >> p.lane_cols) {
        const int pq = p.pos_q[(long long)b * p.Sq + i];
        const int cq = p.chain_q ? p.chain_q[(long long)b * p.Sq + i] : 0;
        const long long at = ((long long)b * p.H + h0) * plane + (long long)i * p.Sk + j0;
        uint4 base[VEC ? HEADS : 1];
        if (VEC && p.base) {  // in flight while the rows are looked up
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h < nh) base[h] = *reinterpret_cast<const uint4*>(p.base + at + h * plane);
        }
        uint32_t v[COLS][NW];  // a column's values, HEADS of them
#pragma unroll
        for (int e = 0; e < COLS; ++e) {
            const int r = cq == ck[e] ? L.row(rel_distance(pq, pk[e])) : p.nb + 1;
            if constexpr (NW == 4) {
                const uint4 w = *reinterpret_cast<const uint4*>(rel_sm + r * 16);
                v[e][0] = w.x, v[e][1] = w.y, v[e][2] = w.z, v[e][3] = w.w;
            } else if constexpr (NW == 2) {
                const uint2 w = *reinterpret_cast<const uint2*>(rel_sm + r * 8);
                v[e][0] = w.x, v[e][1] = w.y;
            } else {
                v[e][0] = *reinterpret_cast<const uint32_t*>(rel_sm + r * 4);
            }
        }
        if constexpr (VEC) {
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                if (h >= nh) break;
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = sizeof(T) == 4 ? v[k][h % NW] : rel_halves(v[(2 * k) % COLS][(h / 2) % NW], v[(2 * k + 1) % COLS][(h / 2) % NW], h & 1);
                if (p.base) {
                    w[0] = rel_add<T>(w[0], base[h].x);
                    w[1] = rel_add<T>(w[1], base[h].y);
                    w[2] = rel_add<T>(w[2], base[h].z);
                    w[3] = rel_add<T>(w[3], base[h].w);
                }
                *reinterpret_cast<uint4*>(p.pair + at + h * plane) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < COLS; ++e) {
                if (j0 + e * step >= p.Sk) break;
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    if (h >= nh) break;
                    const T t = reinterpret_cast<const T*>(v[e])[h];
                    const long long o = at + h * plane + (long long)e * step;
                    p.pair[o] = p.base ? rel_from<T>(rel_f32(t) + rel_f32(p.base[o])) : t;
                }
            }
        }
    }
}

// One block: `ti` query rows x 128 threads' key columns of one head, table rows
// [bin0, bin0 + kRelBins).  Each thread sums into its own column of shared
// memory, [bin][thread], so no two threads meet and the order of the additions
// is fixed.  A bin takes up to one addition for each of a thread's columns and rows,
// 8 x kRelBwdRows = 3840, and 9 more across threads and tiles: the fp32 sums are less than
// 4096 additions deep at every size.  While no column of a warp leaves its bucket the sums stay in
// registers; when one does, the warp adds all of them to their bins, without a
// branch for each (branches for each column, or taking only the columns that
// moved, took 5 times as long: near the diagonal most rows move some column).
// The next two rows' values are in flight meanwhile.  The issue rate is the limit
// beside the memory, so the distance table holds the bins' byte offsets (a row of
// another range of bins: the one behind the last, which nobody reads) and the
// positions are kept as byte offsets into it: an element costs a subtraction, a
// clamp, a read and an addition.  1733 x 1733 x 16 heads, fp32: 67.6 us, 192 MB, 2.84 TB/s, the
// issue slots 66 % busy (an odd row length allows 4-byte loads only, and log-spaced
// buckets move some column of a warp in most rows).  That needs positions below 2^27 in size and
// borders within the table's span; other blocks search the borders.
// VEC: a thread's columns are runs of 16 whole bytes; else they lie the block's
// width apart.
__host__ __device__ inline int rel_bwd_smem(int bins, int nb) {
    return (bins + 1) * kRelBwdThreads * 4 + (nb + 3) / 4 * 16 + kRelLut * 4;
}

template <typename T, bool VEC, bool CHAINS>
__global__ void __launch_bounds__(kRelBwdThreads, 5) evo_relpos_bwd_kernel(const RelParams<T> p) {
    constexpr int RUN = VEC ? 16 / int(sizeof(T)) : 1;  // adjacent columns
    constexpr int COLS = kRelBwdCols;
    constexpr int ROW = kRelBwdThreads * 4;  // bytes of a bin
    extern __shared__ __align__(16) uint8_t rel_sm[];
    const int jt = blockIdx.x % p.jt, itile = blockIdx.x / p.jt;
    const int chunks = (p.rows + kRelBins - 1) / kRelBins;
    const int bin0 = (blockIdx.y % chunks) * kRelBins, nbins = min(kRelBins, p.rows - bin0);
    const int bh = blockIdx.y / chunks, b = bh / p.H, h = bh % p.H;
    float* bins = reinterpret_cast<float*>(rel_sm);  // [nbins + 1][128]
    int* sborders = reinterpret_cast<int*>(bins + (min(p.rows, kRelBins) + 1) * kRelBwdThreads);
    uint32_t* lut = reinterpret_cast<uint32_t*>(sborders + (p.nb + 3) / 4 * 4);
    for (int i = threadIdx.x; i < (nbins + 1) * (kRelBwdThreads / 4); i += kRelBwdThreads)
        reinterpret_cast<float4*>(bins)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    ptx::pdl_launch();
    for (int i = threadIdx.x; i < p.nb; i += kRelBwdThreads) sborders[i] = p.borders[i];

    const int lanes = 1 << p.lane_cols, tx = threadIdx.x & (lanes - 1), ty = threadIdx.x >> p.lane_cols;
    const int i0 = itile * p.ti, rows = min(p.Sq - i0, p.ti), di = kRelBwdThreads >> p.lane_cols;
    const int j0 = jt * lanes * COLS + tx * RUN;
    auto col = [&](int e) -> int { return j0 + (e / RUN) * lanes * RUN + e % RUN; };
    const T* tile = p.dpair + ((long long)bh * p.Sq + i0) * p.Sk;  // row i of the tile: 32-bit offsets (ti * Sk < 2^31)
    const int *posq = p.pos_q + (long long)b * p.Sq + i0, *chainq = CHAINS ? p.chain_q + (long long)b * p.Sq + i0 : nullptr;
    constexpr int WORDS = VEC ? COLS * int(sizeof(T)) / 4 : COLS;  // a row's values as loaded
    auto fetch = [&](int i, uint32_t (&w)[WORDS]) {  // row i, or the last one once more
        const uint32_t at = uint32_t(min(i, rows - 1)) * uint32_t(p.Sk);
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) {
                const int j = col(k * RUN);
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (j < p.Sk) x = *reinterpret_cast<const uint4*>(tile + (at + uint32_t(j)));
                w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < COLS; ++e) {
                const int j = col(e);
                if constexpr (sizeof(T) == 4) w[e] = j < p.Sk ? __float_as_uint(tile[at + uint32_t(j)]) : 0u;
                else w[e] = j < p.Sk ? reinterpret_cast<const uint16_t*>(tile)[at + uint32_t(j)] : 0u;
            }
        }
    };
    auto value = [&](const uint32_t (&w)[WORDS], int e) -> float {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        else if constexpr (!VEC && std::is_same<T, __half>::value) return __half2float(__ushort_as_half(uint16_t(w[e])));
        else if constexpr (!VEC) return ptx::bf16lo_to_f32(w[e]);
        else if constexpr (std::is_same<T, __half>::value) return __half2float(reinterpret_cast<const __half*>(w)[e]);
        else return e & 1 ? ptx::bf16hi_to_f32(w[e / 2]) : ptx::bf16lo_to_f32(w[e / 2]);
    };
    uint32_t w[WORDS], next[WORDS], after[WORDS];
    fetch(ty, w);
    fetch(ty + di, next);
    int pk[COLS], ck[COLS];
    bool near = true;
    auto small = [](int v) { return v > -(1 << 27) && v < (1 << 27); };
#pragma unroll
    for (int e = 0; e < COLS; ++e) {
        const int j = col(e);
        pk[e] = j < p.Sk ? p.pos_k[(long long)b * p.Sk + j] : 0;
        ck[e] = CHAINS && j < p.Sk ? p.chain_k[(long long)b * p.Sk + j] : 0;
        near = near && small(pk[e]);
    }
    for (int i = threadIdx.x; i < rows; i += kRelBwdThreads) near = near && small(posq[i]);
    near = __syncthreads_and(near);  // also: the borders are in place

    RelLookup L;
    L.borders = sborders;
    L.nb = p.nb;
    auto offset = [&](int r) -> uint32_t { return min(uint32_t(r - bin0), uint32_t(nbins)) * ROW; };
    // one entry below the first border, one for each distance up to the last
    const long long first = p.nb > 0 ? sborders[0] : 0, last = p.nb > 0 ? sborders[p.nb - 1] : 0;
    const long long span = last - first + 2;
    const bool direct = near && span >= 2 && span <= kRelLut && small(int(first)) && small(int(last));
    if (direct)
        for (int e = threadIdx.x; e < int(span); e += kRelBwdThreads) lut[e] = offset(L.search(int(first) - 1 + e));
    __syncthreads();
    const int limit = 4 * int(span) - 4;  // byte offset of the last entry
    if (direct) {
#pragma unroll
        for (int e = 0; e < COLS; ++e) pk[e] = 4 * (pk[e] + int(first) - 1);
    }

    char* mine = reinterpret_cast<char*>(bins + threadIdx.x);
    auto flush = [&](uint32_t at, float s) { *reinterpret_cast<float*>(mine + at) += s; };
    uint32_t cur[COLS];
    float sum[COLS];
#pragma unroll
    for (int e = 0; e < COLS; ++e) {
        cur[e] = uint32_t(nbins) * ROW;
        sum[e] = 0.0f;
    }
    const uint32_t apart = offset(p.nb + 1);
    int pq = ty < rows ? posq[ty] : 0, cq = CHAINS && ty < rows ? chainq[ty] : 0;
    auto step = [&](int i) {  // row i; all lanes of a warp take part
        fetch(i + 2 * di, after);
        const int pq_next = posq[min(i + di, rows - 1)], cq_next = CHAINS ? chainq[min(i + di, rows - 1)] : 0;
        uint32_t r[COLS], moved = 0;
        if (direct) {
#pragma unroll
            for (int e = 0; e < COLS; ++e)
                r[e] = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(lut) + __vimin_s32_relu(4 * pq - pk[e], limit));
        } else {
#pragma unroll
            for (int e = 0; e < COLS; ++e) r[e] = offset(L.search(rel_distance(pq, pk[e])));
        }
#pragma unroll
        for (int e = 0; e < COLS; ++e) {
            if (CHAINS && cq != ck[e]) r[e] = apart;
            moved |= r[e] ^ cur[e];
        }
        if (__any_sync(0xffffffffu, moved != 0)) {
#pragma unroll
            for (int e = 0; e < COLS; ++e) {
                flush(cur[e], sum[e]);
                cur[e] = r[e];
                sum[e] = value(w, e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < COLS; ++e) sum[e] += value(w, e);
        }
#pragma unroll
        for (int k = 0; k < WORDS; ++k) w[k] = next[k], next[k] = after[k];
        pq = pq_next;
        cq = cq_next;
    };
    int first_row = 0;  // of those that the block's threads take at once
    for (; first_row + di <= rows; first_row += di) step(first_row + ty);
    if (first_row < rows) {  // some lanes have no row left: they add zeros
        if (first_row + ty >= rows) {
#pragma unroll
            for (int k = 0; k < WORDS; ++k) w[k] = 0u;
        }
        step(first_row + ty);
    }
#pragma unroll
    for (int e = 0; e < COLS; ++e) flush(cur[e], sum[e]);
    __syncthreads();
    // the 128 columns of each bin, a warp a bin, in a fixed order
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long slot = ((long long)b * p.it + itile) * p.jt + jt;
#pragma unroll 4
    for (int r = warp; r < nbins; r += kRelBwdThreads / 32) {
        const float4 x = reinterpret_cast<const float4*>(bins + r * kRelBwdThreads)[lane];
        float s = (x.x + x.y) + (x.z + x.w);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) p.part[(slot * p.H + h) * p.rows + bin0 + r] = s;
    }
}

// dtable[r, h] = the sum over the tiles, a warp an element, in a fixed order: four at a
// time in fp32, then in fp64, because there may be any number of tiles.  (No restrict
// pointers where a kernel waits for the one before: a read could move ahead of the wait.)
template <typename T>
__global__ void __launch_bounds__(256) evo_relpos_bwd_sum_kernel(const float* part, long long tiles, int H,
                                                                 int rows, T* dtable) {
    ptx::pdl_launch();
    ptx::pdl_wait();
    const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (w >= (long long)H * rows) return;
    const int h = int(w / rows), r = int(w % rows);
    double s = 0.0;
    for (long long t = lane; t < tiles; t += 128) {  // four on their way at a time, added in pairs first
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = t + 32 * k < tiles ? part[((t + 32 * k) * H + h) * rows + r] : 0.0f;
        s += (v[0] + v[1]) + (v[2] + v[3]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) dtable[(long long)r * H + h] = rel_from<T>(float(s));
}

}  // namespace evo
