// The fp32 transition: products on the FMA units, sums in registers (1e-5 relative
// accuracy rules out TF32).
//
// One tile routine serves every product: 256 threads hold a 128 x 128 tile of
// fp32 sums, 8 x 8 a thread as two groups of four rows and of four columns 64
// apart, so that a thread's operand reads from shared memory are 16-byte and
// conflict-free.  K advances in slabs of 16, double-buffered: the next slab's
// global loads are in flight while the current one is multiplied.  The products
// use the packed two-lane FMA, which halves the FMA instructions issued.
// Bound by the FMA pipes: 16384 rows, C = 128, F = 512: 175 us forward, 36.8 TFLOP/s, half
// of the pipes' 74 TFLOP/s at the highest clock; what is lost is the issue slots
// of the shared-memory reads and of the slabs' stores, and the gate kernel's spills
// (288 bytes stored, 152 loaded a thread).  Two blocks an SM measured
// 177 us against 182 for one, plain FMAs 187 us.
// The B operand is two groups of 64 rows with pointers of their own: the gate
// and the up projection of the same 64 features come out in the same thread, so
// act(G) * U needs no exchange.
#pragma once

#include "transition_common.cuh"

namespace evo {

constexpr int kTrThreads = 256;
constexpr int kTrK = 16;        // K slab
constexpr int kTrLd = 128 + 4;  // shared row of one k

// One operand of a tile: element (row, k) of group h is p[h][row * ld + k] when
// k is contiguous, p[h][k * ld + row] otherwise; rows >= lim[h] read as zero.
struct TrOperand {
    const float* p[2];
    int lim[2];
    long long ld;
};

__device__ __forceinline__ TrOperand tr_rows(const float* p, long long row_stride, long long ld, int row0, int rows) {
    TrOperand o;
    o.ld = ld;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        o.lim[h] = max(0, min(64, rows - row0 - 64 * h));
        o.p[h] = p + (long long)(o.lim[h] > 0 ? row0 + 64 * h : 0) * row_stride;
    }
    return o;
}

// This thread's share of an operand's 128 x 16 slabs.  K-contiguous: 8 k of one
// row; else 8 rows of one k.
template <bool KC>
struct TrFetch {
    const float* p;  // its first element of the next slab
    long long step;  // to the next slab
    int k, rows;     // that slab's k; rows in range from its own on

    __device__ __forceinline__ TrFetch(const TrOperand& o, int kbeg) {
        const int t = threadIdx.x, row = KC ? (t >> 1) : (t & 15) * 8, r = row & 63;
        const bool second = row >= 64;
        const float* base = second ? o.p[1] : o.p[0];
        k = kbeg + (KC ? (t & 1) * 8 : (t >> 4));
        rows = (second ? o.lim[1] : o.lim[0]) - r;
        p = KC ? base + r * o.ld + k : base + (long long)k * o.ld + r;
        step = KC ? kTrK : kTrK * o.ld;
    }

    __device__ __forceinline__ void load(float (&v)[8], int kend, bool vec) {
        const int n = KC ? (rows > 0 ? kend - k : 0) : (k < kend ? rows : 0);  // elements in range
        if (vec && n >= 8) {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.0f;
        }
        p += step;
        k += kTrK;
    }
};

template <bool KC>
__device__ __forceinline__ void tr_put(float* s, const float (&v)[8]) {
    const int t = threadIdx.x;
    if constexpr (KC) {
        const int row = t >> 1, k = (t & 1) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[(k + e) * kTrLd + row] = v[e];
    } else {
        float* d = s + (t >> 4) * kTrLd + (t & 15) * 8;
        *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
}

__device__ __forceinline__ void tr_fma2(float2& c, float2 a, float2 b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<unsigned long long&>(c))
        : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
}

// acc += A B^T over k in [kbeg, kend).  COLS: column groups computed (2, or 1
// for a 64-column tile).  veca, vecb: 16-byte loads allowed.  `smem` holds 4 slabs.
template <bool AKC, bool BKC, int COLS>
__device__ __forceinline__ void tr_tile(float2 (&acc)[8][2 * COLS], const TrOperand& A, const TrOperand& B,
                                        int kbeg, int kend, bool veca, bool vecb, float* smem) {
    constexpr int SLAB = kTrK * kTrLd;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float va[8], vb[8];
    TrFetch<AKC> fa(A, kbeg);
    TrFetch<BKC> fb(B, kbeg);
    __syncthreads();  // an earlier product's slabs are no longer read
    if (kbeg < kend) {
        fa.load(va, kend, veca);
        fb.load(vb, kend, vecb);
        tr_put<AKC>(smem, va);
        tr_put<BKC>(smem + SLAB, vb);
    }
    __syncthreads();
    int cur = 0;
    for (int k0 = kbeg; k0 < kend; k0 += kTrK) {
        const bool more = k0 + kTrK < kend;
        if (more) {
            fa.load(va, kend, veca);
            fb.load(vb, kend, vecb);
        }
        const float* sa = smem + 2 * cur * SLAB;
        const float* sb = sa + SLAB;
#pragma unroll
        for (int k = 0; k < kTrK; ++k) {
            float a[8];
            float4 b[COLS];
            *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(sa + k * kTrLd + 4 * ty);
            *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(sa + k * kTrLd + 64 + 4 * ty);
#pragma unroll
            for (int c = 0; c < COLS; ++c)
                b[c] = *reinterpret_cast<const float4*>(sb + k * kTrLd + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 ai = make_float2(a[i], a[i]);
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    tr_fma2(acc[i][2 * c], ai, make_float2(b[c].x, b[c].y));
                    tr_fma2(acc[i][2 * c + 1], ai, make_float2(b[c].z, b[c].w));
                }
            }
        }
        if (more) {
            cur ^= 1;
            tr_put<AKC>(smem + 2 * cur * SLAB, va);
            tr_put<BKC>(smem + 2 * cur * SLAB + SLAB, vb);
            __syncthreads();
        }
    }
}

__device__ __forceinline__ int tr_row(int i) {
    return (i < 4 ? 0 : 60) + 4 * int(threadIdx.x >> 4) + i;
}
// column of element e (0..3) of a thread's column group c
__device__ __forceinline__ int tr_col(int c, int e) { return 64 * c + 4 * int(threadIdx.x & 15) + e; }

// Writes four consecutive columns of a row (n in range), 16 bytes at once where it may.
__device__ __forceinline__ void tr_store4(float* p, const float (&v)[4], int n, bool vec) {
    if (vec && n >= 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n) p[e] = v[e];
}

struct TrSimtParams {
    const float *x, *wg, *wu, *wd, *dy;
    float *h, *dg, *du;    // [rows, ldf]
    float* out;                // Y or dX, [rows, C]
    float* part;           // [splits][3][F * C] partial weight gradients
    int rows, C, F, ldf;   // ldf: F up to 4
    int splits, split_rows;
    bool vc, vd, vo;       // float4 accesses allowed: x, dy, wg and wu; wd; out
    int first;             // the first chunk of rows: the partial sums start here
    int dw_mask;           // which weight gradients (bit 0 dWg, 1 dWu, 2 dWd)
};

// H = act(X Wg^T) * (X Wu^T): 128 rows x 64 features a block.
template <int ACT>
__global__ void __launch_bounds__(kTrThreads, 2) evo_tr_simt_gate_kernel(const TrSimtParams p) {
    extern __shared__ __align__(16) float tr_smem[];
    const int f0 = blockIdx.x * 64, m0 = blockIdx.y * 128;
    const TrOperand A = tr_rows(p.x, p.C, p.C, m0, p.rows);
    TrOperand B;
    B.ld = p.C;
    B.p[0] = p.wg + (long long)f0 * p.C;
    B.p[1] = p.wu + (long long)f0 * p.C;
    B.lim[0] = B.lim[1] = min(64, p.F - f0);
    float2 acc[8][4] = {};
    tr_tile<true, true, 2>(acc, A, B, 0, p.C, p.vc, p.vc, tr_smem);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = m0 + tr_row(i), f = f0 + tr_col(0, 0);
        if (m >= p.rows) continue;
        const float g[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
        const float u[4] = {acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y};
        float h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = tr_act<ACT>(g[e]) * u[e];
        tr_store4(p.h + (long long)m * p.ldf + f, h, p.ldf - f, true);
    }
}

// Y = H Wd^T (BWD false), or dX = dG Wg + dU Wu: 128 rows x 64 * COLS channels a
// block (64 where 128 would leave SMs without two blocks).
template <bool BWD, int COLS>
__global__ void __launch_bounds__(kTrThreads, 2) evo_tr_simt_out_kernel(const TrSimtParams p) {
    extern __shared__ __align__(16) float tr_smem[];
    const int c0 = blockIdx.x * 64 * COLS, m0 = blockIdx.y * 128;
    float2 acc[8][2 * COLS] = {};
    const int c_end = min(p.C, c0 + 64 * COLS);
    if constexpr (BWD) {
        tr_tile<true, false, COLS>(acc, tr_rows(p.dg, p.ldf, p.ldf, m0, p.rows), tr_rows(p.wg, 1, p.C, c0, c_end), 0, p.F, true, p.vc,
                                   tr_smem);
        tr_tile<true, false, COLS>(acc, tr_rows(p.du, p.ldf, p.ldf, m0, p.rows), tr_rows(p.wu, 1, p.C, c0, c_end), 0, p.F, true, p.vc,
                                   tr_smem);
    } else {
        tr_tile<true, true, COLS>(acc, tr_rows(p.h, p.ldf, p.ldf, m0, p.rows), tr_rows(p.wd, p.F, p.F, c0, c_end), 0, p.F, true, p.vd,
                                  tr_smem);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = m0 + tr_row(i);
        if (m >= p.rows) continue;
#pragma unroll
        for (int g = 0; g < COLS; ++g) {
            const int c = c0 + tr_col(g, 0);
            const float v[4] = {acc[i][2 * g].x, acc[i][2 * g].y, acc[i][2 * g + 1].x, acc[i][2 * g + 1].y};
            tr_store4(p.out + (long long)m * p.C + c, v, p.C - c, p.vo);
        }
    }
}

// H, dG and dU from X and dY: the gate and up products are recomputed (no
// [M, F] array of the forward is kept), then dH = dY Wd of the same 128 x 64 tile.
template <int ACT>
__global__ void __launch_bounds__(kTrThreads) evo_tr_simt_grad_kernel(const TrSimtParams p) {
    extern __shared__ __align__(16) float tr_smem[];
    const int f0 = blockIdx.x * 64, m0 = blockIdx.y * 128;
    TrOperand B;
    B.ld = p.C;
    B.p[0] = p.wg + (long long)f0 * p.C;
    B.p[1] = p.wu + (long long)f0 * p.C;
    B.lim[0] = B.lim[1] = min(64, p.F - f0);
    float2 acc[8][4] = {};
    tr_tile<true, true, 2>(acc, tr_rows(p.x, p.C, p.C, m0, p.rows), B, 0, p.C, p.vc, p.vc, tr_smem);
    float2 dh[8][2] = {};
    TrOperand D = tr_rows(p.wd, 1, p.F, f0, p.F);
    D.lim[1] = 0;
    tr_tile<true, false, 1>(dh, tr_rows(p.dy, p.C, p.C, m0, p.rows), D, 0, p.C, p.vc, p.vd, tr_smem);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = m0 + tr_row(i), f = f0 + tr_col(0, 0);
        if (m >= p.rows) continue;
        const float g[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
        const float u[4] = {acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y};
        const float d[4] = {dh[i][0].x, dh[i][0].y, dh[i][1].x, dh[i][1].y};
        float h[4], dg[4], du[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, da;
            tr_act_grad<ACT>(g[e], a, da);
            h[e] = a * u[e];
            dg[e] = u[e] * da * d[e];  // (d u may overflow where act' is 0)
            du[e] = d[e] * a;
        }
        const long long at = (long long)m * p.ldf + f;
        tr_store4(p.h + at, h, p.ldf - f, true);
        tr_store4(p.dg + at, dg, p.ldf - f, true);
        tr_store4(p.du + at, du, p.ldf - f, true);
    }
}

// Partial weight gradients of one range of rows: dG^T X, dU^T X [F, C] and
// dY^T H [C, F], summed into this range's own slot (chunks of rows run one after
// another, so each slot is added to in a fixed order: no atomics).
static __global__ void __launch_bounds__(kTrThreads, 2) evo_tr_simt_dw_kernel(const TrSimtParams p) {
    extern __shared__ __align__(16) float tr_smem[];
    const int which = blockIdx.z % 3, split = blockIdx.z / 3;
    if (!((p.dw_mask >> which) & 1)) return;
    const int R = which == 2 ? p.C : p.F, N = which == 2 ? p.F : p.C;
    const int r0 = blockIdx.y * 128, n0 = blockIdx.x * 128;
    if (r0 >= R || n0 >= N) return;
    const int m_beg = split * p.split_rows, m_end = min(p.rows, m_beg + p.split_rows);
    const float* a = which == 0 ? p.dg : which == 1 ? p.du : p.dy;
    const float* b = which == 2 ? p.h : p.x;
    float2 acc[8][4] = {};
    tr_tile<false, false, 2>(acc, tr_rows(a, 1, which == 2 ? p.C : p.ldf, r0, R), tr_rows(b, 1, which == 2 ? p.ldf : p.C, n0, N),
                             m_beg, m_end, which != 2 || p.vc, which == 2 || p.vc, tr_smem);
    float* out = p.part + ((long long)split * 3 + which) * p.F * p.C;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + tr_row(i);
        if (r >= R) continue;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int n = n0 + tr_col(g, 0);
            float v[4] = {acc[i][2 * g].x, acc[i][2 * g].y, acc[i][2 * g + 1].x, acc[i][2 * g + 1].y};
            float* o = out + (long long)r * N + n;
            if (!p.first) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < N) v[e] += o[e];
            }
            tr_store4(o, v, N - n, N % 4 == 0);
        }
    }
}

// dW = the sum of its slots in order.
static __global__ void __launch_bounds__(256) evo_tr_dw_reduce_kernel(const float* __restrict__ part, int splits,
                                                                      long long n, float* dwg, float* dwu, float* dwd) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float* const out[3] = {dwg, dwu, dwd};
#pragma unroll
    for (int w = 0; w < 3; ++w) {
        if (out[w] == nullptr) continue;
        float s = 0.0f;
        for (int k = 0; k < splits; ++k) s += part[((long long)k * 3 + w) * n + i];
        out[w][i] = s;
    }
}

// ---------------------------------------------------------- products in parts

// Few row tiles leave most of the SMs without a block, and a block walks all of K, one
// slab after another.  Then the products are taken in parts: ranges of K with a
// slot of their own, which a second kernel adds in order (and, for G, U and dH, turns into
// H, dG and dU), in tiles of 128 or 32 rows.  Which tile and how many ranges:
// tr_parts in evo_blocks.cu.  Still bound by the tiles' walk over K, now shorter; whole
// calls with and without parts, us: backward 2 x 752 x 3008 75 / 523, 64 x 384 x 1536 62 / 286, 165 x 656 x
// 2558 203 / 731; forward 192 x 384 x 1536 41 / 159, 96 x 1024 x 4096 98 / 404, 411 x 602 x 2408 142 / 382
// (the products by PyTorch and plain operators: 187, 184, 270; 100, 193, 156).

// 32 rows x 128 columns: 4 rows of a warp's own by 4 columns a thread.  acc += A B^T
// over k in [kbeg, kend).
template <bool BKC>
__device__ __forceinline__ void tr_tile32(float2 (&acc)[4][2], const TrOperand& A, const TrOperand& B, int kbeg, int kend,
                                          bool veca, bool vecb, float* smem) {
    constexpr int SLAB = kTrK * kTrLd;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const bool mine = threadIdx.x < 64;  // 32 rows x 16 k, 8 k of a row each
    float va[8], vb[8];
    TrFetch<true> fa(A, kbeg);
    TrFetch<BKC> fb(B, kbeg);
    if (kbeg < kend) {
        if (mine) fa.load(va, kend, veca);
        fb.load(vb, kend, vecb);
        if (mine) tr_put<true>(smem, va);
        tr_put<BKC>(smem + SLAB, vb);
    }
    __syncthreads();
    int cur = 0;
    for (int k0 = kbeg; k0 < kend; k0 += kTrK) {
        const bool more = k0 + kTrK < kend;
        if (more) {
            if (mine) fa.load(va, kend, veca);
            fb.load(vb, kend, vecb);
        }
        const float* sa = smem + 2 * cur * SLAB;
        const float* sb = sa + SLAB;
#pragma unroll
        for (int k = 0; k < kTrK; ++k) {
            const float4 a = *reinterpret_cast<const float4*>(sa + k * kTrLd + 4 * ty);
            const float4 b = *reinterpret_cast<const float4*>(sb + k * kTrLd + 4 * tx);
            const float r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 ai = make_float2(r[i], r[i]);
                tr_fma2(acc[i][0], ai, make_float2(b.x, b.y));
                tr_fma2(acc[i][1], ai, make_float2(b.z, b.w));
            }
        }
        if (more) {
            cur ^= 1;
            if (mine) tr_put<true>(smem + 2 * cur * SLAB, va);
            tr_put<BKC>(smem + 2 * cur * SLAB + SLAB, vb);
            __syncthreads();
        }
    }
}

// out = A B^T, A [rows, K] with k contiguous; B [N, K] with k contiguous (kc), else [K, N].
struct TrJob {
    const float *a, *b;
    int lda;
    bool kc, veca, vecb;
};
enum TrLayoutOfB { TR_B_K, TR_B_N, TR_B_MIXED };  // contiguous along k in every job, in none, in some

struct TrPartParams {
    TrJob job[3];
    int jobs, splits;
    int rows, N, K;
    int ld;             // of a slot's rows: N up to 4
    float* slots;       // [splits][jobs][rows][ld]
};

// ROWS x 64 * COLS (128 columns with 32 rows) of one job over one range of K a block.
template <int ROWS, int COLS, int B_LAYOUT>
__global__ void __launch_bounds__(kTrThreads, ROWS == 32 ? 4 : 2) evo_tr_simt_part_kernel(const __grid_constant__ TrPartParams p) {
    extern __shared__ __align__(16) float tr_smem[];
    const int j = blockIdx.z % p.jobs, split = blockIdx.z / p.jobs;
    const int n0 = blockIdx.x * 64 * COLS, m0 = blockIdx.y * ROWS;
    const int per = ((p.K + kTrK - 1) / kTrK + p.splits - 1) / p.splits * kTrK;
    const int kbeg = split * per, kend = min(p.K, kbeg + per);
    const bool kc = B_LAYOUT == TR_B_K || (B_LAYOUT == TR_B_MIXED && p.job[j].kc);
    const bool veca = p.job[j].veca, vecb = p.job[j].vecb;
    const TrOperand A = tr_rows(p.job[j].a, p.job[j].lda, p.job[j].lda, m0, min(p.rows, m0 + ROWS));
    const TrOperand B = tr_rows(p.job[j].b, kc ? p.K : 1, kc ? p.K : p.N, n0, min(p.N, n0 + 64 * COLS));
    float* out = p.slots + (long long)blockIdx.z * p.rows * p.ld;
    if constexpr (ROWS == 32) {
        float2 acc[4][2] = {};
        if (kc) tr_tile32<true>(acc, A, B, kbeg, kend, veca, vecb, tr_smem);
        else tr_tile32<false>(acc, A, B, kbeg, kend, veca, vecb, tr_smem);
        const int n = n0 + 4 * int(threadIdx.x & 31);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + 4 * int(threadIdx.x >> 5) + i;
            const float v[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
            if (m < p.rows) tr_store4(out + (long long)m * p.ld + n, v, p.ld - n, true);
        }
    } else {
        float2 acc[8][2 * COLS] = {};
        if (kc) tr_tile<true, true, COLS>(acc, A, B, kbeg, kend, veca, vecb, tr_smem);
        else tr_tile<true, false, COLS>(acc, A, B, kbeg, kend, veca, vecb, tr_smem);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = m0 + tr_row(i);
            if (m >= p.rows) continue;
#pragma unroll
            for (int g = 0; g < COLS; ++g) {
                const int n = n0 + tr_col(g, 0);
                const float v[4] = {acc[i][2 * g].x, acc[i][2 * g].y, acc[i][2 * g + 1].x, acc[i][2 * g + 1].y};
                tr_store4(out + (long long)m * p.ld + n, v, p.ld - n, true);
            }
        }
    }
}

// four elements at `at` of slots `first`, `first + step`, .., added in order
__device__ __forceinline__ float4 tr_slots(const float* slots, long long slot, int first, int step, int count, long long at) {
    float4 s = *reinterpret_cast<const float4*>(slots + first * slot + at);
    for (int k = 1; k < count; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(slots + (first + (long long)k * step) * slot + at);
        s.x += y.x, s.y += y.y, s.z += y.z, s.w += y.w;
    }
    return s;
}

// H (and dG, dU) of four features a thread from the slots of G, U (and dH).
template <int ACT, bool BWD>
__global__ void __launch_bounds__(256) evo_tr_join_act_kernel(const float* slots, int splits, int rows, int ld,
                                                              float* h, float* dg, float* du) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, slot = (long long)rows * ld;
    if (4 * i >= slot) return;
    constexpr int jobs = BWD ? 3 : 2;
    const float4 gs = tr_slots(slots, slot, 0, jobs, splits, 4 * i), us = tr_slots(slots, slot, 1, jobs, splits, 4 * i);
    const float g[4] = {gs.x, gs.y, gs.z, gs.w}, u[4] = {us.x, us.y, us.z, us.w};
    const long long at = 4 * i;  // H's rows are as long as the slots'
    float hv[4];
    if constexpr (BWD) {
        const float4 ds = tr_slots(slots, slot, 2, jobs, splits, 4 * i);
        const float d[4] = {ds.x, ds.y, ds.z, ds.w};
        float dgv[4], duv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, da;
            tr_act_grad<ACT>(g[e], a, da);
            hv[e] = a * u[e];
            dgv[e] = u[e] * da * d[e];
            duv[e] = d[e] * a;
        }
        *reinterpret_cast<float4*>(dg + at) = make_float4(dgv[0], dgv[1], dgv[2], dgv[3]);
        *reinterpret_cast<float4*>(du + at) = make_float4(duv[0], duv[1], duv[2], duv[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) hv[e] = tr_act<ACT>(g[e]) * u[e];
    }
    *reinterpret_cast<float4*>(h + at) = make_float4(hv[0], hv[1], hv[2], hv[3]);
}

// Y or dX, four channels a thread, from all of its slots.
static __global__ void __launch_bounds__(256) evo_tr_join_out_kernel(const float* slots, int count, int rows, int C, int ld,
                                                                     float* out, int vec) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, slot = (long long)rows * ld;
    if (4 * i >= slot) return;
    const int m = int(4 * i / ld), c = int(4 * i - (long long)m * ld);
    const float4 s = tr_slots(slots, slot, 0, 1, count, 4 * i);
    const float v[4] = {s.x, s.y, s.z, s.w};
    tr_store4(out + (long long)m * C + c, v, C - c, vec);
}

}  // namespace evo
