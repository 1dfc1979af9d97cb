// The transition's products on the tensor cores (bf16 / fp16 operands, fp32
// accumulation in tensor memory), for sm_100a.
//
// Rows are taken in chunks whose [rows, F] intermediates stay in L2.  Five
// products, one persistent kernel template (a CTA per SM, tiles with a stride of
// the grid):
//   GATE  H = act(X Wg^T) * (X Wu^T)     128 rows x 128 features: the rows of Wg
//         and Wu for the same features are one 256-row operand, so both
//         projections are one N = 256 MMA per 16-deep step, and a thread of the
//         epilogue finds G and U of its elements in the same tensor-memory lane.
//   OUT   Y = H Wd^T                     128 rows x BN channels
//   GRAD  dH = dY Wd beside G and U; writes H, dG, dU.  Tensor memory holds G and
//         U once (256 columns) and dH twice, so that the next tile's dH product
//         runs during this tile's epilogue.
//   DX    dX = dG Wg + dU Wu             128 rows x BN channels, both products
//         into one accumulator
//   DW    dG^T X, dU^T X [F, C] and dY^T H [C, F]: 128 x 256 (or 128 x 128) of one
//         range of rows, written as the gradient itself where one range takes all
//         rows, else added into the range's own fp32 slot.
// Operands that are contiguous along k are read K-major, the others (Wd in GRAD,
// the weights in DX, both in DW) MN-major: the same swizzled TMA boxes of 128-byte
// rows serve both, so nothing is transposed in memory.
//
// Warp roles (384 threads): warp 0 loads (TMA ring), warp 1 issues the MMAs,
// warps 4-11 drain the accumulators: warp w reads the 32 tensor-memory lanes of
// its place in its warpgroup, the two warpgroups half the columns each.  Results
// leave through 32-column boxes of shared memory, a warp's own, and TMA stores:
// stored from registers a warp writes 32 rows 16 or 32 bytes at a time, which took
// longer than the products (GRAD at C = 128: 22 us for 18944 rows x 512 features).
//
// 8192 rows, C = 1024, F = 4096, fp16, GELU (backward 575 us): GRAD 200 us (1.03 PFLOP/s),
// DX 93 us (1.48), DW 163 us (1.26: 384 tiles on 148 SMs are 2.6 rounds).  GRAD is
// held by its 128-column dH MMAs, which keep their issuer about as long as
// 256-column ones (120 cycles against 128), and by a tile's G and U products waiting
// for the epilogue before (tensor memory is full).  Sixteen epilogue warps there: 225 us; the next
// stage's barrier tested between the MMAs: no change.
// Every wait is bounded (2 s); on expiry the CTA records EVO_ERR_TIMEOUT, drains
// its own copies and MMAs, frees tensor memory and exits.
#pragma once

#include <cuda.h>
#include <cstdint>
#include <type_traits>

#include "tile_sm100.cuh"
#include "transition_common.cuh"

namespace evo {

enum TrKind { TR_GATE, TR_OUT, TR_GRAD, TR_DX, TR_DW };

// Operands, then results (0-based): GATE: X, Wg, Wu, H.  OUT: H, Wd, Y.
// GRAD: X, Wg, Wu, dY, Wd, H, dG, dU.  DX: dG, Wg, dU, Wu, dX.
// DW: X, dY, dG, dU, H, and the three gradients (or their slots).
struct TrMaps {
    CUtensorMap m[8];
};

struct TrMmaParams {
    uint16_t* out;    // Y or dX, [rows, C]
    int rows, C, F;
    int tiles_m, tiles_n, num_tiles;
    int kb;           // 64-deep K blocks of one product
    int tma_out;      // OUT, DX: rows of whole 16-byte units (else element by element)
    // DW
    int split_rows;   // rows of a range, a multiple of 64
    int which[3], num_which;  // the gradients asked for
    int tn01, tn2;    // column tiles of dWg and dWu, and of dWd
    int tiles01, tiles2;      // tiles of one of dWg, dWu, and of dWd
    int bn01;         // columns of a tile of dWg, dWu: 256 or 128
    int direct;       // one range and one chunk: the tiles are the gradients
    int first;        // the slots start here
};

template <int KIND, int BN, bool F16>
struct TrCfg {
    static constexpr int THREADS = 384;
    static constexpr int STAGES = KIND == TR_GRAD ? 3 : BN == 64 ? 6 : 4;
    static constexpr int BOXES = KIND == TR_GRAD ? 6144 : 4096;  // a warp's boxes for its results
    static constexpr int OPER_A = 128 * 128;   // 128 rows x 64 k, or 64 k x 128 columns
    static constexpr int OPER_B = BN * 128;
    static constexpr int STAGE_BYTES = OPER_A + OPER_B;
    static constexpr int OFF_BOX = STAGES * STAGE_BYTES;
    static constexpr int OFF_BAR = OFF_BOX + 8 * BOXES;
    static constexpr int BAR_FULL = 0, BAR_EMPTY = STAGES, BAR_AF = 2 * STAGES, BAR_AE = 2 * STAGES + 2,
                         BAR_DRAIN = 2 * STAGES + 4, NUM_BARS = 2 * STAGES + 5;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static constexpr uint32_t TMEM_COLS = KIND == TR_GRAD ? 512 : 2 * BN;
    static constexpr uint32_t AB = F16 ? 0u : ((1u << 7) | (1u << 10));
    __host__ __device__ static constexpr uint32_t idesc(bool a_mn, bool b_mn, int n) {
        return (1u << 4) | AB | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t(n) >> 3) << 17) |
               ((128u >> 4) << 24);
    }
};

__device__ __forceinline__ float2 tr_mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 tr_add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
    return d;
}

__device__ __forceinline__ float2 tr_mad2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
          "l"(reinterpret_cast<const unsigned long long&>(c)));
    return d;
}
__device__ __forceinline__ float2 tr_both(float v) { return make_float2(v, v); }

// 1 / a of two elements with one reciprocal; a.x * a.y must be finite
__device__ __forceinline__ float2 tr_rcp2(float2 a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a.x * a.y));
    return tr_mul2(tr_both(r), make_float2(a.y, a.x));
}

// sigmoid of two elements.  One reciprocal serves both: 1/a = b / (a b), which
// leaves the special-function unit 1.5 instructions an element instead of 2.
// FAR false: |g| <= kTrNear, so that a b is finite.  FAR true, any g: from
// e^-|g| <= 1, as 1 / (1 + e^-|g|) on the positive side and e^-|g| times that on
// the negative one, which goes to 0 with e^g (below g = -87 it is 0).
template <bool FAR>
__device__ __forceinline__ float2 tr_sigmoid2(float2 g) {
    float2 x = tr_mul2(g, make_float2(-kLog2e, -kLog2e));
    if constexpr (FAR) x = make_float2(fminf(-fabsf(x.x), 0.0f), fminf(-fabsf(x.y), 0.0f));  // (NaN: 0, so that it stays its own)
    const float2 e = make_float2(ptx::ex2_approx(x.x), ptx::ex2_approx(x.y));
    const float2 s = tr_rcp2(tr_add2(e, tr_both(1.0f)));
    return FAR ? tr_mul2(s, make_float2(g.x < 0.0f ? e.x : 1.0f, g.y < 0.0f ? e.y : 1.0f)) : s;
}

// Gates up to this size on either side take the short forms: (1 + e^43)^2 < 2^126,
// within the range of the reciprocal that serves two elements.
constexpr float kTrNear = 43.0f;

// Whether all of a lane's gates are near (false with a NaN among them).  One
// comparison a gate, as holding each exponent back by itself would cost.
template <int N>
__device__ __forceinline__ bool tr_near(const float (&g)[N]) {
    float m[4] = {};
#pragma unroll
    for (int e = 0; e < N; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m[e & 3]) : "f"(fabsf(g[e])));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m[0]) : "f"(m[1]));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m[2]) : "f"(m[3]));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m[0]) : "f"(m[2]));
    return m[0] <= kTrNear;
}

__device__ __forceinline__ float2 tr_above2(float2 g) { return make_float2(tr_above(g.x), tr_above(g.y)); }
__device__ __forceinline__ float2 tr_finite2(float2 g) { return make_float2(tr_finite(g.x), tr_finite(g.y)); }

// Phi(-|g|) e^(g^2/2) = t (c0 + c1 t + .. + c6 t^6), t = 1 / (1 + kPhiT |g|): fitted for the
// smallest relative error on |g| <= 13.3, where e^(-g^2/2) leaves fp32's normal numbers
// (weighted least squares, the weights raised where the error is largest, until it is
// level): at most 6.3e-7, 9.4e-7 in fp32.
constexpr float kPhiT = 0.265f;
constexpr float kPhiC0 = 0.1055998355f;
constexpr float kPhiC1 = 0.1078367457f;
constexpr float kPhiC2 = 0.08294672519f;
constexpr float kPhiC3 = 0.1424930245f;
constexpr float kPhiC4 = -0.06636252999f;
constexpr float kPhiC5 = 0.1952728629f;
constexpr float kPhiC6 = -0.06778696924f;

// Phi(g) and e^(-g^2/2) of two elements.  The error is relative to Phi on the
// negative side too, where g Phi(g) is small: a formula with an absolute error of 1.5e-7
// is 0.2 % off at g = -4, which is more than the rounding of a 16-bit H.
// FAR (not all gates near): |g| is held at 2^40, where the exponential has long
// been 0 and the reciprocals' product is still finite.
template <bool FAR>
__device__ __forceinline__ float2 tr_phi2(float2 g, float2& e) {
    float2 a = make_float2(fabsf(g.x), fabsf(g.y));
    if (FAR) a = make_float2(fminf(a.x, 0x1p40f), fminf(a.y, 0x1p40f));
    const float2 t = tr_rcp2(tr_mad2(tr_both(kPhiT), a, tr_both(1.0f)));
    float2 p = tr_mad2(tr_both(kPhiC6), t, tr_both(kPhiC5));
    p = tr_mad2(p, t, tr_both(kPhiC4));
    p = tr_mad2(p, t, tr_both(kPhiC3));
    p = tr_mad2(p, t, tr_both(kPhiC2));
    p = tr_mad2(p, t, tr_both(kPhiC1));
    p = tr_mad2(p, t, tr_both(kPhiC0));
    const float2 y = tr_mul2(tr_mul2(a, tr_both(-0.5f * kLog2e)), a);
    e = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
    const float2 low = tr_mul2(tr_mul2(p, t), e);  // Phi(-|g|)
    // 1 - Phi(-|g|) on the positive side
    return make_float2(g.x >= 0.0f ? 1.0f - low.x : low.x, g.y >= 0.0f ? 1.0f - low.y : low.y);
}

// h = act(g) * u of a pair.  (act(g) first: g u may overflow where act(g) is 0.)
template <int ACT, bool FAR>
__device__ __forceinline__ float2 tr_gate2(float2 g, float2 u) {
    float2 p, e;
    if constexpr (ACT == EVO_ACT_SILU) p = tr_sigmoid2<FAR>(g);
    else p = tr_phi2<FAR>(g, e);
    return tr_mul2(tr_mul2(FAR ? tr_above2(g) : g, p), u);
}

// h, dg and du of a pair from g, u and d = dH
template <int ACT, bool FAR>
__device__ __forceinline__ void tr_grad2(float2 g, float2 u, float2 d, float2& h, float2& dg, float2& du) {
    float2 p, e, da;
    if constexpr (ACT == EVO_ACT_SILU) p = tr_sigmoid2<FAR>(g);
    else p = tr_phi2<FAR>(g, e);
    const float2 a = tr_mul2(FAR ? tr_above2(g) : g, p);
    if (FAR) g = tr_finite2(g);
    if constexpr (ACT == EVO_ACT_SILU) da = tr_mad2(FAR ? tr_mul2(g, p) : a, tr_mad2(p, tr_both(-1.0f), tr_both(1.0f)), p);
    else da = tr_mad2(tr_mul2(g, tr_both(0.3989422804014327f)), e, p);
    h = tr_mul2(a, u);
    du = tr_mul2(d, a);
    dg = tr_mul2(tr_mul2(u, da), d);
}

// N gates and ups of a lane: h in place of g.  A lane with a gate that is not
// near takes the longer form for all of its own.
template <int ACT, int N>
__device__ __forceinline__ void tr_gate_all(float (&g)[N], const float (&u)[N]) {
    auto all = [&](auto far) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 h = tr_gate2<ACT, decltype(far)::value>(make_float2(g[e], g[e + 1]), make_float2(u[e], u[e + 1]));
            g[e] = h.x, g[e + 1] = h.y;
        }
    };
    if (tr_near(g)) all(std::false_type{});
    else all(std::true_type{});
}

// dg, du and h in place of g, u and d
template <int ACT, int N>
__device__ __forceinline__ void tr_grad_all(float (&g)[N], float (&u)[N], float (&d)[N]) {
    auto all = [&](auto far) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            float2 h, dg, du;
            tr_grad2<ACT, decltype(far)::value>(make_float2(g[e], g[e + 1]), make_float2(u[e], u[e + 1]),
                                                make_float2(d[e], d[e + 1]), h, dg, du);
            d[e] = h.x, d[e + 1] = h.y;
            g[e] = dg.x, g[e + 1] = dg.y;
            u[e] = du.x, u[e + 1] = du.y;
        }
    };
    if (tr_near(g)) all(std::false_type{});
    else all(std::true_type{});
}

template <bool F16>
__device__ __forceinline__ uint32_t tr_pack(float lo, float hi) {
    return F16 ? ptx::pack_f16x2(lo, hi) : ptx::pack_bf16x2(lo, hi);
}

// 32 columns of this lane's row, packed, as 4 16-byte pieces `first` .. of a box
// row: 32 rows of 64 bytes, 64 B swizzle.
template <bool F16, int PIECES>
__device__ __forceinline__ void tr_box16(uint32_t box, int lane, int first, const float* v) {
#pragma unroll
    for (int e = 0; e < PIECES; ++e)
        ptx::st_shared_v4(box + swz_chunk<64>(lane, first + e),
                          make_uint4(tr_pack<F16>(v[8 * e], v[8 * e + 1]), tr_pack<F16>(v[8 * e + 2], v[8 * e + 3]),
                                     tr_pack<F16>(v[8 * e + 4], v[8 * e + 5]), tr_pack<F16>(v[8 * e + 6], v[8 * e + 7])));
}

// 32 columns c0 .. of 32 rows m0 .. of an output whose rows TMA cannot store (no
// whole 16-byte units): turned in a warp's 2 KB of shared memory, so that a store
// covers 64 adjacent bytes of one row.  Word e of row r lies at r * 16 + (e ^ r % 16):
// no bank is asked twice, either way.
template <bool F16>
__device__ __forceinline__ void tr_store_rows(uint32_t box, int lane, const float* v, uint16_t* out, int C, int c0, int m0,
                                              int rows) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(box + uint32_t(lane * 64 + ((e ^ (lane & 15)) << 2))),
                     "r"(tr_pack<F16>(v[2 * e], v[2 * e + 1]))
                     : "memory");
    __syncwarp();
    const int n = min(32, rows - m0);
    if (c0 + lane < C) {
        uint16_t* o = out + size_t(m0) * C + c0 + lane;
#pragma unroll 8
        for (int r = 0; r < n; ++r, o += C) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(h)
                         : "r"(box + uint32_t(r * 64 + (((lane >> 1) ^ (r & 15)) << 2) + 2 * (lane & 1))));
            *o = h;
        }
    }
    __syncwarp();
}

template <int KIND, int ACT, bool F16, int BN>
__global__ void __launch_bounds__(384, 1)
evo_tr_mma_kernel(const __grid_constant__ TrMaps maps, const TrMmaParams p) {
    using C = TrCfg<KIND, BN, F16>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = ptx::smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int G = gridDim.x;
    auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8u * uint32_t(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

    // K blocks of one tile; GRAD runs dH's product first, then G and U; DX dG's, then dU's
    constexpr int PRODUCTS = (KIND == TR_GRAD || KIND == TR_DX) ? 2 : 1;
    // tile L: column block fastest, then row block.  DW: every tile of a range of
    // rows (gradient by gradient), then the next range
    auto tile = [&](int L, int& tn, int& tm, int& which, int& split) {
        which = split = 0;
        if constexpr (KIND == TR_DW) {
            const int per = p.num_tiles;  // of a range
            split = L / per;
            L -= split * per;
            for (int w = 0; w < p.num_which; ++w) {
                which = p.which[w];
                const int n = which == 2 ? p.tiles2 : p.tiles01;
                if (L < n) break;
                L -= n;
            }
            const int cols = which == 2 ? p.tn2 : p.tn01;
            tn = L % cols;
            tm = L / cols;
        } else {
            tn = L % p.tiles_n;
            tm = L / p.tiles_n;
        }
    };
    const int all_tiles = KIND == TR_DW ? p.num_tiles * p.tiles_n : p.num_tiles;  // DW: tiles_n ranges
    auto blocks = [&](int split) -> int {
        if constexpr (KIND == TR_DW) {
            const int n = min(p.split_rows, p.rows - split * p.split_rows);
            return n > 0 ? (n + 63) / 64 : 0;
        }
        return p.kb;
    };
    auto dw_cols = [&](int which) -> int { return which == 2 ? 256 : p.bn01; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(bar(C::BAR_FULL + s), 1);
            ptx::mbar_init(bar(C::BAR_EMPTY + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(bar(C::BAR_AF + a), 1);
            ptx::mbar_init(bar(C::BAR_AE + a), 8);
        }
        ptx::mbar_init(bar(C::BAR_DRAIN), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::pdl_launch();
    ptx::pdl_wait();

    if (warp == 0) {
        // -------------------------------------------------------------- loads
        int n = 0;
        bool ok = true;
        for (int L = blockIdx.x; L < all_tiles && ok; L += G) {
            int tn, tm, which, split;
            tile(L, tn, tm, which, split);
            const int kbs = blocks(split);
#pragma unroll 1
            for (int kt = 0; kt < PRODUCTS * kbs; ++kt, ++n) {
                const int s = n % C::STAGES;
                ok = wait_warp(bar(C::BAR_EMPTY + s), ((n / C::STAGES) & 1) ^ 1, abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t a = sb + uint32_t(s * C::STAGE_BYTES), b = a + C::OPER_A;
                    const uint32_t f = bar(C::BAR_FULL + s);
                    const bool second = PRODUCTS == 2 && kt >= kbs;
                    const int k = 64 * (second ? kt - kbs : kt);
                    if constexpr (KIND == TR_GATE) {
                        ptx::mbar_arrive_expect_tx(f, C::STAGE_BYTES);
                        ptx::tma_load_2d(a, &maps.m[0], f, k, 128 * tm);
                        ptx::tma_load_2d(b, &maps.m[1], f, k, 128 * tn);
                        ptx::tma_load_2d(b + 16384, &maps.m[2], f, k, 128 * tn);
                    } else if constexpr (KIND == TR_GRAD) {
                        if (!second) {
                            ptx::mbar_arrive_expect_tx(f, C::OPER_A + 16384);
                            ptx::tma_load_2d(a, &maps.m[3], f, k, 128 * tm);
                            ptx::tma_load_2d(b, &maps.m[4], f, 128 * tn, k);
                            ptx::tma_load_2d(b + 8192, &maps.m[4], f, 128 * tn + 64, k);
                        } else {
                            ptx::mbar_arrive_expect_tx(f, C::STAGE_BYTES);
                            ptx::tma_load_2d(a, &maps.m[0], f, k, 128 * tm);
                            ptx::tma_load_2d(b, &maps.m[1], f, k, 128 * tn);
                            ptx::tma_load_2d(b + 16384, &maps.m[2], f, k, 128 * tn);
                        }
                    } else if constexpr (KIND == TR_OUT) {
                        ptx::mbar_arrive_expect_tx(f, C::STAGE_BYTES);
                        ptx::tma_load_2d(a, &maps.m[0], f, k, 128 * tm);
                        constexpr int R = BN < 128 ? 64 : 128;  // rows of Wd's box
#pragma unroll
                        for (int x = 0; x < BN / R; ++x)
                            ptx::tma_load_2d(b + R * 128 * x, &maps.m[1], f, k, BN * tn + R * x);
                    } else if constexpr (KIND == TR_DX) {
                        ptx::mbar_arrive_expect_tx(f, C::STAGE_BYTES);
                        ptx::tma_load_2d(a, &maps.m[second ? 2 : 0], f, k, 128 * tm);
#pragma unroll
                        for (int x = 0; x < BN / 64; ++x)
                            ptx::tma_load_2d(b + 8192 * x, &maps.m[second ? 3 : 1], f, BN * tn + 64 * x, k);
                    } else {
                        const int m = split * p.split_rows + k, bn = dw_cols(which);
                        ptx::mbar_arrive_expect_tx(f, uint32_t(C::OPER_A + bn * 128));
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            ptx::tma_load_2d(a + 8192 * x, &maps.m[which == 2 ? 1 : 2 + which], f, 128 * tm + 64 * x, m);
                        for (int x = 0; x < bn / 64; ++x)
                            ptx::tma_load_2d(b + 8192 * x, &maps.m[which == 2 ? 4 : 0], f, bn * tn + 64 * x, m);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) {
            // the last load of each stage lands before the CTA exits
            for (int s = 0; s < C::STAGES; ++s)
                if (n - 1 >= s) {
                    const int last = s + C::STAGES * ((n - 1 - s) / C::STAGES);
                    wait_bounded(bar(C::BAR_FULL + s), uint32_t(last / C::STAGES) & 1u, nullptr);
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMAs
        int n = 0, t = 0;
        bool ok = true, issued = false;
        for (int L = blockIdx.x; L < all_tiles && ok; L += G, ++t) {
            int tn, tm, which, split;
            tile(L, tn, tm, which, split);
            const int kbs = blocks(split), acc = t & 1;
            // the epilogue has drained this accumulator's previous tile
            ok = wait_warp(bar(C::BAR_AE + acc), ((t >> 1) & 1) ^ 1, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int kt = 0; kt < PRODUCTS * kbs; ++kt, ++n) {
                const int s = n % C::STAGES;
                const bool second = PRODUCTS == 2 && kt >= kbs;
                if (KIND == TR_GRAD && kt == kbs && t > 0) {
                    // G and U share one place: the previous tile's epilogue is done with them
                    ok = wait_warp(bar(C::BAR_AE + (acc ^ 1)), uint32_t((t - 1) >> 1) & 1u, abort_flag);
                    if (!ok) break;
                    ptx::tc_fence_after();
                }
                ok = wait_warp(bar(C::BAR_FULL + s), uint32_t(n / C::STAGES) & 1u, abort_flag);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t a = sb + uint32_t(s * C::STAGE_BYTES), b = a + C::OPER_A;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if constexpr (KIND == TR_GRAD) {
                        const uint32_t add = ((second ? kt - kbs : kt) > 0 || kk > 0) ? 1u : 0u;
                        if (!second)
                            ptx::mma_ss_elect(tmem + uint32_t(256 + 128 * acc), desc_k_major<128>(a + 32 * kk),
                                              desc_mn_major<128>(b + 2048 * kk, 8192), C::idesc(false, true, 128), add);
                        else
                            ptx::mma_ss_elect(tmem, desc_k_major<128>(a + 32 * kk), desc_k_major<128>(b + 32 * kk),
                                              C::idesc(false, false, 256), add);
                    } else {
                        constexpr bool A_MN = KIND == TR_DW, B_MN = KIND == TR_DW || KIND == TR_DX;
                        const uint64_t da = A_MN ? desc_mn_major<128>(a + 2048 * kk, 8192) : desc_k_major<128>(a + 32 * kk);
                        const uint64_t db = B_MN ? desc_mn_major<128>(b + 2048 * kk, 8192) : desc_k_major<128>(b + 32 * kk);
                        const uint32_t id = KIND == TR_DW && dw_cols(which) == 128 ? C::idesc(A_MN, B_MN, 128)
                                                                                   : C::idesc(A_MN, B_MN, BN);
                        ptx::mma_ss_elect(tmem + uint32_t(BN * acc), da, db, id, (kt > 0 || kk > 0) ? 1u : 0u);
                    }
                }
                issued = true;
                ptx::mma_commit_elect(bar(C::BAR_EMPTY + s));
            }
            if (!ok) break;
            ptx::mma_commit_elect(bar(C::BAR_AF + acc));
        }
        if (!ok && issued) {
            ptx::mma_commit_elect(bar(C::BAR_DRAIN));
            wait_bounded(bar(C::BAR_DRAIN), 0, nullptr);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ----------------------------------------------------------- epilogue
        const int wq = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tl = tmem + (uint32_t(32 * wq) << 16);
        const uint32_t box = sb + uint32_t(C::OFF_BOX + C::BOXES * (warp - 4));
        int t = 0;
        uint32_t turn = 0;  // which of two boxes
        bool ok = true;
        for (int L = blockIdx.x; L < all_tiles && ok; L += G, ++t) {
            int tn, tm, which, split;
            tile(L, tn, tm, which, split);
            const int acc = t & 1, m0 = 128 * tm + 32 * wq;
            ok = wait_warp(bar(C::BAR_AF + acc), uint32_t(t >> 1) & 1u, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            auto release = [&]() {
                ptx::tc_fence_before();
                ptx::mbar_arrive_elect(bar(C::BAR_AE + acc));
            };
            // 32 columns c0 .. of this warp's rows of a 16-bit result through one of two boxes
            auto put16 = [&](const CUtensorMap* map, int c0, int r0, const float* v) {
                const uint32_t bx = box + 2048u * (turn & 1u);
                ++turn;
                ptx::bulk_wait_read<1>();  // the store before the last has read its box
                __syncwarp();
                tr_box16<F16, 4>(bx, lane, 0, v);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::tma_store_2d(map, bx, c0, r0);
                __syncwarp();
            };
            if constexpr (KIND == TR_GATE) {
                // rows past `rows` and features past F are zero (their operands read as zero)
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    float g[32], u[32];
                    ptx::tmem_ld_x32(tl + uint32_t(256 * acc + 64 * half + 32 * c), reinterpret_cast<uint32_t*>(g));
                    ptx::tmem_ld_x32(tl + uint32_t(256 * acc + 128 + 64 * half + 32 * c), reinterpret_cast<uint32_t*>(u));
                    ptx::tmem_ld_wait_x32(reinterpret_cast<uint32_t*>(g));
                    ptx::reg_fence_x32(reinterpret_cast<uint32_t*>(u));
                    if (c == 1) release();
                    tr_gate_all<ACT>(g, u);
                    __syncwarp();
                    put16(&maps.m[3], 128 * tn + 64 * half + 32 * c, m0, g);
                }
            } else if constexpr (KIND == TR_GRAD) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float g[16], u[16], d[16];
                    ptx::tmem_ld_x16(tl + uint32_t(64 * half + 16 * c), reinterpret_cast<uint32_t*>(g));
                    ptx::tmem_ld_x16(tl + uint32_t(128 + 64 * half + 16 * c), reinterpret_cast<uint32_t*>(u));
                    ptx::tmem_ld_x16(tl + uint32_t(256 + 128 * acc + 64 * half + 16 * c), reinterpret_cast<uint32_t*>(d));
                    ptx::tmem_ld_wait_x16(reinterpret_cast<uint32_t*>(g));
                    ptx::reg_fence_x8(reinterpret_cast<uint32_t*>(u));
                    ptx::reg_fence_x8(reinterpret_cast<uint32_t*>(u) + 8);
                    ptx::reg_fence_x8(reinterpret_cast<uint32_t*>(d));
                    ptx::reg_fence_x8(reinterpret_cast<uint32_t*>(d) + 8);
                    if (c == 3) release();
                    tr_grad_all<ACT>(g, u, d);
                    __syncwarp();
                    if ((c & 1) == 0) {  // the boxes of the 32 features before have been read
                        ptx::bulk_wait_read<0>();
                        __syncwarp();
                    }
                    tr_box16<F16, 2>(box, lane, 2 * (c & 1), d);
                    tr_box16<F16, 2>(box + 2048, lane, 2 * (c & 1), g);
                    tr_box16<F16, 2>(box + 4096, lane, 2 * (c & 1), u);
                    if (c & 1) {
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            const int c0 = 128 * tn + 64 * half + 32 * (c >> 1);
#pragma unroll
                            for (int o = 0; o < 3; ++o) ptx::tma_store_2d(&maps.m[5 + o], box + 2048u * o, c0, m0);
                        }
                        __syncwarp();
                    }
                }
            } else if constexpr (KIND == TR_DW) {
                const int cols = dw_cols(which) / 2, R = which == 2 ? p.C : p.F, N = which == 2 ? p.F : p.C;
                const bool empty = blocks(split) == 0;  // a range past the chunk's rows adds nothing
#pragma unroll 1
                for (int c = 0; c < cols / 32; ++c) {
                    float v[32];
                    ptx::tmem_ld_x32(tl + uint32_t(BN * acc + cols * half + 32 * c), reinterpret_cast<uint32_t*>(v));
                    ptx::tmem_ld_wait_x32(reinterpret_cast<uint32_t*>(v));
                    if (c == cols / 32 - 1) release();
                    const int c0 = dw_cols(which) * tn + cols * half + 32 * c;
                    const bool in = c0 < N && m0 < R && !(empty && !p.first);
                    if (in && p.direct) put16(&maps.m[5 + which], c0, m0, v);
                    if (in && !p.direct) {
                        ptx::bulk_wait_read<0>();
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            ptx::st_shared_v4(box + swz_chunk<128>(lane, e),
                                              empty ? make_uint4(0u, 0u, 0u, 0u)
                                                    : make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]),
                                                                 __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3])));
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (p.first) ptx::tma_store_3d(&maps.m[5 + which], box, c0, m0, split);
                            else ptx::tma_add_3d(&maps.m[5 + which], box, c0, m0, split);
                        }
                        __syncwarp();
                    }
                }
            } else {
                const int cols = BN / 2;
#pragma unroll 1
                for (int c = 0; c < cols / 32; ++c) {
                    float v[32];
                    ptx::tmem_ld_x32(tl + uint32_t(BN * acc + cols * half + 32 * c), reinterpret_cast<uint32_t*>(v));
                    ptx::tmem_ld_wait_x32(reinterpret_cast<uint32_t*>(v));
                    if (c == cols / 32 - 1) release();
                    const int c0 = BN * tn + cols * half + 32 * c;
                    if (c0 < p.C && m0 < p.rows) {
                        if (p.tma_out) put16(&maps.m[KIND == TR_OUT ? 2 : 4], c0, m0, v);
                        else tr_store_rows<F16>(box, lane, v, p.out, p.C, c0, m0, p.rows);
                    }
                }
            }
        }
        ptx::bulk_wait_all();  // the stores have left shared memory and are done
        __syncwarp();
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
}

// ------------------------------------------------------- the whole block at once

// Y of 128 rows in one CTA, for C <= 256: the rows' X stays in shared memory, the
// weights stream through a ring (from L2, where they stay), H never leaves the
// SM.  Per chunk of 128 features: G and U (one N = 256 MMA a step) into 256
// columns of tensor memory; the epilogue warps turn them into a 128 x 128 tile
// of H; Y += H Wd^T accumulates in CN columns of tensor memory.  At CN = 128 H
// lies in tensor memory too, as the A operand of its product: the MMAs' operand
// reads and the weights' arrival already take most of the 128 bytes a cycle of
// shared memory, and H there would add a write and a read.  At CN = 256 tensor
// memory is full and H goes to shared memory, swizzled as the tensor core reads
// it.  One warp issues the products GU, another OUT (an issuing warp is busy for most of an MMA's time, so one would
// leave the tensor cores idle at its waits); GU(q + 1) runs beside the activation
// of chunk q, across tiles too, and a tile's Y is drained after the first
// activation of the next tile.  An activation holds its packed H in registers
// until OUT of the chunk before has read the one H tile.  Y goes through 32 x 32
// tiles a warp of shared memory and TMA stores: straight from registers, a warp's
// 32-byte pieces of 32 rows held up the H stores of the other warps (a drain took
// 2000 cycles of a tile's 12000 at C = 128).
//
// 131072 rows, C = 256, F = 1024: 163 us, 1.27 PFLOP/s, the tensor pipe 80 % busy at the
// 1.5 GHz that the power limit leaves.  589824 rows, C = 128, F = 512: 229 us, 1.0
// PFLOP/s: tensor pipe and special functions 63 % busy each, because a chunk's G and
// U have one place in tensor memory and the activation and GU wait for each other.
// (64-feature chunks in two places, two groups of warps in turn: 248 us; an N = 128
// MMA keeps its issuer as busy as an N = 256 one.)
struct TrFusedParams {
    uint16_t* out;  // Y [M, C]
    int M, C, F;
    int num_tiles;  // ceil(M / 128)
    int kc;         // 64-deep blocks of C
    int chunks;     // ceil(F / 128)
    int wide_store;  // Y through TMA (rows of whole 16-byte units), else element by element
};

template <bool F16, int CN>
struct TrFusedCfg {
    static constexpr int EPI_WARPS = 16;           // a warp: 32 rows x 32 features of a chunk
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int XSLOTS = 4;               // 128 rows x 64 k of X, 16 KB each
    static constexpr bool H_TMEM = CN == 128;
    static constexpr int STAGES = H_TMEM ? 4 : 3;  // weights: 32 KB each
    static constexpr int OUT_STAGES = CN / 128;    // ring stages of Wd for a chunk
    static constexpr int OFF_H = XSLOTS * 16384;   // 128 rows x 128 features
    static constexpr int OFF_Y = OFF_H + (H_TMEM ? 0 : 32768);    // 2 KB a warp: 32 rows x 32 channels of Y
    static constexpr int OFF_W = OFF_Y + EPI_WARPS * 2048;
    static constexpr int OFF_BAR = OFF_W + STAGES * 32768;
    static constexpr int XF = 0, XE = XF + XSLOTS, WF = XE + XSLOTS, WE = WF + STAGES, GF = WE + STAGES, GE = GF + 1,
                         HF = GE + 1, HE = HF + 1, OF = HE + 1, OE = OF + 1, GC = OE + 1, OC = GC + 1, DRAIN = OC + 1,
                         NUM_BARS = DRAIN + 2;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static constexpr uint32_t TMEM_COLS = 512;     // G, U: 0-255, Y: CN columns from 256, H: 64 columns from 384
    static constexpr uint32_t AB = F16 ? 0u : ((1u << 7) | (1u << 10));
    __host__ __device__ static constexpr uint32_t idesc(int n) {
        return (1u << 4) | AB | ((uint32_t(n) >> 3) << 17) | ((128u >> 4) << 24);
    }
};

// maps: X, Wg, Wu, Wd, Y
template <int ACT, bool F16, int CN>
__global__ void __launch_bounds__(640, 1)
evo_tr_fused_kernel(const __grid_constant__ TrMaps maps, const TrFusedParams p) {
    using C = TrFusedCfg<F16, CN>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = ptx::smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int G = gridDim.x;
    auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8u * uint32_t(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    const int my_tiles = (p.num_tiles - int(blockIdx.x) + G - 1) / G;
    const int total = my_tiles * p.chunks;  // this CTA's chunks, in order

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::XSLOTS; ++i) {
            ptx::mbar_init(bar(C::XF + i), 1);
            ptx::mbar_init(bar(C::XE + i), 1);
        }
        for (int i = 0; i < C::STAGES; ++i) {
            ptx::mbar_init(bar(C::WF + i), 1);
            ptx::mbar_init(bar(C::WE + i), 1);
        }
        ptx::mbar_init(bar(C::GF), 1);
        ptx::mbar_init(bar(C::GE), C::EPI_WARPS);
        ptx::mbar_init(bar(C::HF), C::EPI_WARPS);
        ptx::mbar_init(bar(C::HE), 1);
        ptx::mbar_init(bar(C::OF), 1);
        ptx::mbar_init(bar(C::OE), C::EPI_WARPS);
        ptx::mbar_init(bar(C::GC), 1);
        ptx::mbar_init(bar(C::OC), 1);
        ptx::mbar_init(bar(C::DRAIN), 1);
        ptx::mbar_init(bar(C::DRAIN + 1), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::pdl_launch();
    ptx::pdl_wait();
    // Fill n of the weight ring has landed.  Two warps take stages from the one
    // ring.  A parity cannot tell fill n of a stage from the one two fills before,
    // so a warp must know that the fill between, which may be the other warp's, has
    // landed: GU(q) starts when OUT(q - 2) has seen its stages land (barrier OC),
    // OUT(q) when GU(q + 1) has (GC).  Every stage before GU(q) and OUT(q) in the
    // ring's order is one of those, an earlier one or the warp's own.
    auto weights_full = [&](int n) -> bool {
        return wait_warp(bar(C::WF + n % C::STAGES), uint32_t(n / C::STAGES) & 1u, abort_flag);
    };

    if (warp == 0) {
        // -------------------------------------------------------------- loads
        int n = 0, xn = 0;  // weight stages and X slots filled so far
        bool ok = true;
        auto weights = [&](bool gate, int chunk, int k) -> bool {
            const int s = n % C::STAGES;
            if (!wait_warp(bar(C::WE + s), ((n / C::STAGES) & 1) ^ 1, abort_flag)) return false;
            if (lane == 0) {
                const uint32_t d = sb + uint32_t(C::OFF_W + 32768 * s), f = bar(C::WF + s);
                ptx::mbar_arrive_expect_tx(f, 32768);
                if (gate) {
                    ptx::tma_load_2d(d, &maps.m[1], f, 64 * k, 128 * chunk);
                    ptx::tma_load_2d(d + 16384, &maps.m[2], f, 64 * k, 128 * chunk);
                } else if (CN == 128) {  // 128 channels x both halves of the chunk's features
                    ptx::tma_load_2d(d, &maps.m[3], f, 128 * chunk, 0);
                    ptx::tma_load_2d(d + 16384, &maps.m[3], f, 128 * chunk + 64, 0);
                } else {                 // 256 channels x half k of the chunk's features
                    ptx::tma_load_2d(d, &maps.m[3], f, 128 * chunk + 64 * k, 0);
                    ptx::tma_load_2d(d + 16384, &maps.m[3], f, 128 * chunk + 64 * k, 128);
                }
            }
            __syncwarp();
            ++n;
            return true;
        };
        int tile = blockIdx.x, j = 0, prev = 0;
        for (int q = 0; q <= total && ok; ++q) {
            if (q < total) {
                if (j == 0) {
                    for (int k = 0; k < p.kc && ok; ++k, ++xn) {
                        const int s = xn % C::XSLOTS;
                        ok = wait_warp(bar(C::XE + s), ((xn / C::XSLOTS) & 1) ^ 1, abort_flag);
                        if (!ok) break;
                        if (lane == 0) {
                            ptx::mbar_arrive_expect_tx(bar(C::XF + s), 16384);
                            ptx::tma_load_2d(sb + uint32_t(16384 * s), &maps.m[0], bar(C::XF + s), 64 * k, 128 * tile);
                        }
                        __syncwarp();
                    }
                }
                for (int k = 0; k < p.kc && ok; ++k) ok = weights(true, j, k);
            }
            if (q > 0)
                for (int k = 0; k < C::OUT_STAGES && ok; ++k) ok = weights(false, prev, k);
            prev = j;
            if (++j == p.chunks) {
                j = 0;
                tile += G;
            }
        }
        if (!ok && lane == 0) {
            // the last load of each slot and stage lands before the CTA exits
            for (int s = 0; s < C::STAGES; ++s)
                if (n - 1 >= s) wait_bounded(bar(C::WF + s), uint32_t((n - 1 - s) / C::STAGES) & 1u, nullptr);
            for (int s = 0; s < C::XSLOTS; ++s)
                if (xn - 1 >= s) wait_bounded(bar(C::XF + s), uint32_t((xn - 1 - s) / C::XSLOTS) & 1u, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- GU products
        // weight stages come in the order GU(0), GU(1), OUT(0), GU(2), OUT(1), ...
        int j = 0, xn = 0;
        bool ok = true, issued = false;
        for (int q = 0; q < total && ok; ++q) {
            // the activation of chunk q - 1 has read its G and U
            ok = wait_warp(bar(C::GE), (q & 1) ^ 1, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            if (q >= 2) {
                ok = wait_warp(bar(C::OC), uint32_t(q) & 1u, abort_flag);  // OUT(q - 2)
                if (!ok) break;
            }
            const int n0 = q * p.kc + max(q - 1, 0) * C::OUT_STAGES;
            for (int k = 0; k < p.kc; ++k) {
                const int n = n0 + k, s = n % C::STAGES, x = (xn + k) % C::XSLOTS;
                if (j == 0) ok = wait_warp(bar(C::XF + x), uint32_t((xn + k) / C::XSLOTS) & 1u, abort_flag);
                if (!ok) break;
                ok = weights_full(n);
                if (!ok) break;
                if (k == p.kc - 1) ptx::mbar_arrive_elect(bar(C::GC));
                ptx::tc_fence_after();
                const uint32_t a = sb + uint32_t(16384 * x), b = sb + uint32_t(C::OFF_W + 32768 * s);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_ss_elect(tmem, desc_k_major<128>(a + 32 * kk), desc_k_major<128>(b + 32 * kk), C::idesc(256),
                                      (k > 0 || kk > 0) ? 1u : 0u);
                issued = true;
                ptx::mma_commit_elect(bar(C::WE + s));
                if (j == p.chunks - 1) ptx::mma_commit_elect(bar(C::XE + x));
            }
            if (!ok) break;
            ptx::mma_commit_elect(bar(C::GF));
            if (++j == p.chunks) {
                j = 0;
                xn += p.kc;
            }
        }
        if (!ok && issued) {
            ptx::mma_commit_elect(bar(C::DRAIN));
            wait_bounded(bar(C::DRAIN), 0, nullptr);
        }
        __syncwarp();
    } else if (warp == 2) {
        // --------------------------------------------------------- OUT products
        int j = 0, t = 0;  // chunk of the tile, tile
        bool ok = true, issued = false;
        for (int q = 0; q < total && ok; ++q) {
            // Y += H(q) Wd^T
            if (j == 0) {  // the tile before has been drained
                ok = wait_warp(bar(C::OE), (t & 1) ^ 1, abort_flag);
                if (!ok) break;
            }
            ok = wait_warp(bar(C::HF), uint32_t(q) & 1u, abort_flag);
            if (!ok) break;
            ok = wait_warp(bar(C::GC), uint32_t(min(q + 1, total - 1)) & 1u, abort_flag);  // GU(q + 1)
            if (!ok) break;
            const int n0 = min(q + 2, total) * p.kc + q * C::OUT_STAGES;
            for (int k = 0; k < C::OUT_STAGES; ++k) {
                const int n = n0 + k, s = n % C::STAGES;
                ok = weights_full(n);
                if (!ok) break;
                if (k == C::OUT_STAGES - 1) ptx::mbar_arrive_elect(bar(C::OC));
                ptx::tc_fence_after();
                const uint32_t b = sb + uint32_t(C::OFF_W + 32768 * s);
#pragma unroll
                for (int kk = 0; kk < 8 / C::OUT_STAGES; ++kk) {
                    const int f = kk + 4 * k;  // 16-feature step of the chunk
                    const uint64_t db = desc_k_major<128>(b + (CN == 128 ? 16384 * (f >> 2) : 0) + 32 * (f & 3));
                    const uint32_t add = (j > 0 || f > 0) ? 1u : 0u;
                    if constexpr (C::H_TMEM)
                        ptx::mma_ts_elect(tmem + 256u, tmem + uint32_t(384 + 8 * f), db, C::idesc(CN), add);
                    else
                        ptx::mma_ss_elect(tmem + 256u, desc_k_major<128>(sb + uint32_t(C::OFF_H + 16384 * (f >> 2) + 32 * (f & 3))),
                                          db, C::idesc(CN), add);
                }
                issued = true;
                ptx::mma_commit_elect(bar(C::WE + s));
            }
            if (!ok) break;
            ptx::mma_commit_elect(bar(C::HE));
            if (++j == p.chunks) {
                ptx::mma_commit_elect(bar(C::OF));
                j = 0;
                ++t;
            }
        }
        if (!ok && issued) {
            ptx::mma_commit_elect(bar(C::DRAIN + 1));
            wait_bounded(bar(C::DRAIN + 1), 0, nullptr);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ----------------------------------------------------------- epilogue
        const int wq = warp & 3, quarter = (warp - 4) >> 2;
        const int r = 32 * wq + lane;
        const uint32_t tl = tmem + (uint32_t(32 * wq) << 16);
        bool ok = true;
        int tile = blockIdx.x, j = 0, t = 0;
        const uint32_t ys = sb + uint32_t(C::OFF_Y + 2048 * (warp - 4));
        // 32 channels at a time of this warp's rows of Y; the tile of the call before has left `ys`
        auto drain = [&](int of_tile) -> bool {
            if (!wait_warp(bar(C::OF), uint32_t(t) & 1u, abort_flag)) return false;
            ptx::tc_fence_after();
            const int m0 = 128 * of_tile + 32 * wq;
#pragma unroll 1
            for (int c = 0; c < CN / 128; ++c) {
                float v[32];
                const int c0 = CN / 4 * quarter + 32 * c;
                ptx::tmem_ld_x32(tl + uint32_t(256 + c0), reinterpret_cast<uint32_t*>(v));
                ptx::tmem_ld_wait_x32(reinterpret_cast<uint32_t*>(v));
                if (c == CN / 128 - 1) {
                    ptx::tc_fence_before();
                    ptx::mbar_arrive_elect(bar(C::OE));
                }
                if (p.wide_store) {
                    ptx::bulk_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ptx::st_shared_v4(ys + swz_chunk<64>(lane, e),
                                          make_uint4(tr_pack<F16>(v[8 * e], v[8 * e + 1]), tr_pack<F16>(v[8 * e + 2], v[8 * e + 3]),
                                                     tr_pack<F16>(v[8 * e + 4], v[8 * e + 5]),
                                                     tr_pack<F16>(v[8 * e + 6], v[8 * e + 7])));
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && m0 < p.M && c0 < p.C) ptx::tma_store_2d(&maps.m[4], ys, c0, m0);
                    __syncwarp();
                } else {
                    if (m0 < p.M && c0 < p.C) tr_store_rows<F16>(ys, lane, v, p.out, p.C, c0, m0, p.M);
                }
            }
            ++t;
            return true;
        };
        for (int q = 0; q < total && ok; ++q) {
            ok = wait_warp(bar(C::GF), uint32_t(q) & 1u, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            float g[32], u[32];
            ptx::tmem_ld_x32(tl + uint32_t(32 * quarter), reinterpret_cast<uint32_t*>(g));
            ptx::tmem_ld_x32(tl + uint32_t(128 + 32 * quarter), reinterpret_cast<uint32_t*>(u));
            ptx::tmem_ld_wait_x32(reinterpret_cast<uint32_t*>(g));
            ptx::reg_fence_x32(reinterpret_cast<uint32_t*>(u));
            ptx::tc_fence_before();
            ptx::mbar_arrive_elect(bar(C::GE));
            uint32_t w[16];
            tr_gate_all<ACT>(g, u);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = tr_pack<F16>(g[2 * e], g[2 * e + 1]);
            // the product of the chunk before has read the H tile
            ok = wait_warp(bar(C::HE), uint32_t(q & 1) ^ 1u, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            if constexpr (C::H_TMEM) {
                ptx::tmem_st_x16(tl + uint32_t(384 + 16 * quarter), w);
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
            } else {
                const uint32_t h = sb + uint32_t(C::OFF_H + 16384 * (quarter >> 1));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    ptx::st_shared_v4(h + swz_chunk<128>(r, 4 * (quarter & 1) + e),
                                      make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]));
                ptx::fence_proxy_async_smem();  // H is read by the tensor cores
                __syncwarp();
            }
            ptx::mbar_arrive_elect(bar(C::HF));
            if (j == 0 && q > 0) ok = drain(tile - G);
            if (++j == p.chunks) {
                j = 0;
                tile += G;
            }
        }
        if (ok && total > 0) drain(tile - G);
        ptx::bulk_wait_all();  // the stores have left shared memory and are done
        __syncwarp();
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
}

// -------------------------------- dG, dU and the weight gradients in one kernel

// For C <= 128 the three arrays [M, F] that GRAD writes and DW reads outweigh
// everything else (147456 rows x 512 features: 0.9 GB, 138 us at the copy rate).
// Here a CTA owns 64 features and a share of the row tiles: the features' weights
// stay in shared memory, and the gradients of these weights stay in tensor memory
// over all its tiles, 192 columns ([X^T dG | X^T dU] and dY^T H, channels in the
// lanes).  H is never written, dG and dU only for dX's product.
//
// Per row tile: X and dY arrive once (two buffers of 64 KB) and serve G, U and dH
// K-major and the weight gradients MN-major; eight warps turn G, U, dH (192
// columns, G and U twice) into tiles of dG, dU and H in shared memory.  Warp 1
// issues G, U and dH, warp 2 the weight gradients.  147456 rows x 512 features, C = 128:
// 159 us, beside dX's 56 and the slots' sum 7; dG and dU leave at 1.9 TB/s, and X
// and dY come once for every 64 features, from L2.
struct TrGradwParams {
    uint16_t* d[2];  // dG, dU [M, ldf], or null where dX is not asked for
    float* part;     // [3][splits][C][ldp]: dWg^T, dWu^T, dWd of each share of the rows
    int ldf, ldp;
    int M, C, F;
    int num_tiles;   // ceil(M / 128)
    int kc;          // 64-deep blocks of C: 1 or 2
    int slices;      // ceil(F / 64)
    int splits;
    int first;       // the slots start here
};

template <bool F16>
struct TrGradwCfg {
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int FC = 64;
    static constexpr int XBUF = 65536;             // X's blocks (128 rows x 64 k, 16 KB each), dY's from 32768
    static constexpr int OFF_W = 2 * XBUF;         // Wg, Wu of each block (8 KB each), Wd's blocks from 32768
    static constexpr int OFF_D = OFF_W + 49152;    // dG, dU, H: 128 rows x 64 features each
    static constexpr int OFF_BAR = OFF_D + 49152;
    static constexpr int WF = 0, XF = 1, XE = XF + 2, GF = XE + 2, GE = GF + 2, DF = GE + 2, DE = DF + 1, OF = DE + 1,
                         DRAIN = OF + 1, NUM_BARS = DRAIN + 2;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    // G, U: 128 columns from 0 and from 128; dH: 256; X^T dG, X^T dU: 320; dY^T H: 448
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t AB = F16 ? 0u : ((1u << 7) | (1u << 10));
    __host__ __device__ static constexpr uint32_t idesc(bool a_mn, bool b_mn, int n) {
        return (1u << 4) | AB | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t(n) >> 3) << 17) |
               ((128u >> 4) << 24);
    }
};

// maps: X, dY (boxes of 128 rows), Wg, Wu, Wd (64 rows)
template <int ACT, bool F16>
__global__ void __launch_bounds__(384, 1)
evo_tr_gradw_kernel(const __grid_constant__ TrMaps maps, const TrGradwParams p) {
    using C = TrGradwCfg<F16>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = ptx::smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8u * uint32_t(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    const int slice = int(blockIdx.x) % p.slices, split = int(blockIdx.x) / p.slices;
    const int total = (p.num_tiles - split + p.splits - 1) / p.splits;  // row tiles split, split + splits, ...

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NUM_BARS; ++i)
            ptx::mbar_init(bar(i), i == C::GE || i == C::GE + 1 || i == C::DF ? C::EPI_WARPS : 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::pdl_launch();
    ptx::pdl_wait();

    if (warp == 0) {
        // -------------------------------------------------------------- loads
        if (lane == 0 && total > 0) {
            const uint32_t d = sb + uint32_t(C::OFF_W), f = bar(C::WF);
            ptx::mbar_arrive_expect_tx(f, uint32_t(p.kc) * 24576u);
            for (int k = 0; k < p.kc; ++k) {
                ptx::tma_load_2d(d + 16384 * k, &maps.m[2], f, 64 * k, C::FC * slice);
                ptx::tma_load_2d(d + 16384 * k + 8192, &maps.m[3], f, 64 * k, C::FC * slice);
                ptx::tma_load_2d(d + 32768 + 8192 * k, &maps.m[4], f, C::FC * slice, 64 * k);
            }
        }
        __syncwarp();
        bool ok = true;
        int q = 0;
        for (; q < total; ++q) {
            const int b = q & 1;
            ok = wait_warp(bar(C::XE + b), uint32_t((q >> 1) & 1) ^ 1u, abort_flag);
            if (!ok) break;
            if (lane == 0) {
                const uint32_t d = sb + uint32_t(C::XBUF * b), f = bar(C::XF + b);
                const int m = 128 * (split + q * p.splits);
                ptx::mbar_arrive_expect_tx(f, uint32_t(p.kc) * 32768u);
                for (int k = 0; k < p.kc; ++k) {
                    ptx::tma_load_2d(d + 16384 * k, &maps.m[0], f, 64 * k, m);
                    ptx::tma_load_2d(d + 32768 + 16384 * k, &maps.m[1], f, 64 * k, m);
                }
            }
            __syncwarp();
        }
        if (!ok && lane == 0) {
            // the last load of each buffer lands before the CTA exits
            wait_bounded(bar(C::WF), 0u, nullptr);
            for (int b = 0; b < 2; ++b)
                if (q - 1 >= b) wait_bounded(bar(C::XF + b), uint32_t((q - 1 - b) / 2) & 1u, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------- G, U, dH products
        bool ok = total == 0 || wait_warp(bar(C::WF), 0u, abort_flag), issued = false;
        const uint32_t w = sb + uint32_t(C::OFF_W);
        for (int q = 0; q < total && ok; ++q) {
            const int b = q & 1;
            const uint32_t ph = uint32_t(q >> 1) & 1u, x = sb + uint32_t(C::XBUF * b);
            ok = wait_warp(bar(C::GE + b), ph ^ 1u, abort_flag);  // G and U of tile q - 2 have been read
            if (!ok) break;
            ok = wait_warp(bar(C::XF + b), ph, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            for (int k = 0; k < p.kc; ++k)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_ss_elect(tmem + 128u * uint32_t(b), desc_k_major<128>(x + 16384 * k + 32 * kk),
                                      desc_k_major<128>(w + 16384 * k + 32 * kk), C::idesc(false, false, 128),
                                      (k > 0 || kk > 0) ? 1u : 0u);
            issued = true;
            if (q > 0) {  // and dH of tile q - 1
                ok = wait_warp(bar(C::GE + (b ^ 1)), uint32_t((q - 1) >> 1) & 1u, abort_flag);
                if (!ok) break;
                ptx::tc_fence_after();
            }
            for (int k = 0; k < p.kc; ++k)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_ss_elect(tmem + 256u, desc_k_major<128>(x + 32768 + 16384 * k + 32 * kk),
                                      desc_mn_major<128>(w + 32768 + 8192 * k + 2048 * kk, 8192), C::idesc(false, true, 64),
                                      (k > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit_elect(bar(C::GF + b));
        }
        if (!ok && issued) {
            ptx::mma_commit_elect(bar(C::DRAIN));
            wait_bounded(bar(C::DRAIN), 0, nullptr);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------ weight gradients
        bool ok = true, issued = false;
        const uint32_t d = sb + uint32_t(C::OFF_D);
        for (int q = 0; q < total && ok; ++q) {
            const int b = q & 1;
            // the tiles are in place, so X and dY landed long ago
            ok = wait_warp(bar(C::DF), uint32_t(q) & 1u, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t x = sb + uint32_t(C::XBUF * b), add = q > 0 ? 1u : 0u;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 rows
                ptx::mma_ss_elect(tmem + 320u, desc_mn_major<128>(x + 2048 * kk, 16384), desc_mn_major<128>(d + 2048 * kk, 16384),
                                  C::idesc(true, true, 128), kk > 0 ? 1u : add);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                ptx::mma_ss_elect(tmem + 448u, desc_mn_major<128>(x + 32768 + 2048 * kk, 16384),
                                  desc_mn_major<128>(d + 32768 + 2048 * kk, 16384), C::idesc(true, true, 64), kk > 0 ? 1u : add);
            issued = true;
            ptx::mma_commit_elect(bar(C::XE + b));
            ptx::mma_commit_elect(bar(C::DE));
        }
        if (ok) ptx::mma_commit_elect(bar(C::OF));
        if (!ok && issued) {
            ptx::mma_commit_elect(bar(C::DRAIN + 1));
            wait_bounded(bar(C::DRAIN + 1), 0, nullptr);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------- activations
        const int wq = warp & 3, half = (warp - 4) >> 2;
        const int r = 32 * wq + lane;
        const uint32_t tl = tmem + (uint32_t(32 * wq) << 16), dt = sb + uint32_t(C::OFF_D);
        bool ok = true;
        for (int q = 0; q < total && ok; ++q) {
            const int b = q & 1;
            ok = wait_warp(bar(C::GF + b), uint32_t(q >> 1) & 1u, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            float g[32], u[32], d[32];
            ptx::tmem_ld_x32(tl + uint32_t(128 * b + 32 * half), reinterpret_cast<uint32_t*>(g));
            ptx::tmem_ld_x32(tl + uint32_t(128 * b + 64 + 32 * half), reinterpret_cast<uint32_t*>(u));
            ptx::tmem_ld_x32(tl + uint32_t(256 + 32 * half), reinterpret_cast<uint32_t*>(d));
            ptx::tmem_ld_wait_x32(reinterpret_cast<uint32_t*>(g));
            ptx::reg_fence_x32(reinterpret_cast<uint32_t*>(u));
            ptx::reg_fence_x32(reinterpret_cast<uint32_t*>(d));
            ptx::tc_fence_before();
            ptx::mbar_arrive_elect(bar(C::GE + b));
            tr_grad_all<ACT>(g, u, d);
            __syncwarp();
            // the products of the tile before have read its dG, dU and H
            ok = wait_warp(bar(C::DE), uint32_t(q & 1) ^ 1u, abort_flag);
            if (!ok) break;
#pragma unroll
            for (int o = 0; o < 3; ++o) {
                const float* v = o == 0 ? g : o == 1 ? u : d;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    ptx::st_shared_v4(dt + uint32_t(16384 * o) + swz_chunk<128>(r, 4 * half + e),
                                      make_uint4(tr_pack<F16>(v[8 * e], v[8 * e + 1]), tr_pack<F16>(v[8 * e + 2], v[8 * e + 3]),
                                                 tr_pack<F16>(v[8 * e + 4], v[8 * e + 5]),
                                                 tr_pack<F16>(v[8 * e + 6], v[8 * e + 7])));
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            ptx::mbar_arrive_elect(bar(C::DF));
            if (p.d[0] != nullptr) {
                // this warp's 32 rows x 64 bytes of dG and dU, 8 rows at a time
                const int m0 = 128 * (split + q * p.splits) + 32 * wq;
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    uint16_t* out = p.d[o] + size_t(m0 + (lane >> 2)) * p.ldf + C::FC * slice + 32 * half + 8 * (lane & 3);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 8 * e + (lane >> 2);
                        const uint4 v = ptx::ld_shared_v4(dt + uint32_t(16384 * o) + swz_chunk<128>(32 * wq + row, 4 * half + (lane & 3)));
                        if (m0 + row < p.M) *reinterpret_cast<uint4*>(out + size_t(8 * e) * p.ldf) = v;
                    }
                }
                __syncwarp();
            }
        }
        // the sums: this lane's channel, 32 features at a time
        if (ok && wait_warp(bar(C::OF), 0u, abort_flag)) {
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 3; ++c) {  // half 0: dWg, half 1: dWu, each in two parts; then half of dWd
                float v[32];
                const int which = c == 2 ? 2 : half, f = c == 2 ? 32 * half : 32 * c;
                ptx::tmem_ld_x32(tl + uint32_t(c == 2 ? 448 + 32 * half : 320 + 64 * half + 32 * c), reinterpret_cast<uint32_t*>(v));
                ptx::tmem_ld_wait_x32(reinterpret_cast<uint32_t*>(v));
                if (r < p.C) {
                    float4* o = reinterpret_cast<float4*>(p.part + ((size_t(which) * p.splits + split) * p.C + r) * p.ldp +
                                                          C::FC * slice + f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float4 s = total > 0 ? make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3])
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
                        if (!p.first) {
                            const float4 y = o[e];
                            s = make_float4(s.x + y.x, s.y + y.y, s.z + y.z, s.w + y.w);
                        }
                        o[e] = s;
                    }
                }
                __syncwarp();
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
}

// The weight gradients from the shares' sums, added in order and rounded to the
// type, a thread an element: [3][splits][C][ldp], the first two turned into [F, C].
template <typename T>
__global__ void __launch_bounds__(256) evo_tr_gradw_reduce_kernel(const float* part, int splits, int C, int F, int ldp,
                                                                  T* dwg, T* dwu, T* dwd) {
    ptx::pdl_launch();
    ptx::pdl_wait();
    const int which = blockIdx.z, f = blockIdx.x * 32 + (threadIdx.x & 31), c = blockIdx.y * 8 + (threadIdx.x >> 5);
    T* out = which == 0 ? dwg : which == 1 ? dwu : dwd;
    if (out == nullptr || c >= C || f >= F) return;
    const size_t slot = size_t(C) * ldp;
    const float* x = part + size_t(which) * splits * slot + size_t(c) * ldp + f;
    float s = 0.0f;
    int k = 0;
    for (; k + 8 <= splits; k += 8) {  // eight loads on their way at a time
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x[(k + e) * slot];
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
    }
    for (; k < splits; ++k) s += x[k * slot];
    tr_store(out + (which == 2 ? size_t(c) * F + f : size_t(f) * C + c), s);
}

// Rows of `w` elements copied to rows of `wp` (w rounded up to 8; zeros behind
// column w), for up to five matrices at once: TMA reads rows of whole 16-byte
// units only.  A lane forms one 16-byte unit, from 4-byte loads where the source
// has them on such boundaries, all in flight at once (a warp a row, an element a
// lane at a time, waited for memory 13 times a row: 22.8 us for the copies of 1733 x
// 388 with 1555 features, 5.5 so).
struct TrPads {
    const uint16_t* src[5];
    uint16_t* dst[5];
    int rows[5], w[5], wp[5];
    int n;
};

static __global__ void __launch_bounds__(256) evo_tr_pad_kernel(const TrPads p) {
    ptx::pdl_launch();
    ptx::pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long step = ((long long)gridDim.x * blockDim.x) >> 5;
    long long t = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;  // a warp's run of 32 units
    for (int k = 0; k < p.n; ++k) {
        const int w = p.w[k], runs = (p.wp[k] + 255) / 256;
        const long long all = (long long)p.rows[k] * runs;
        const bool words = w % 2 == 0 && (reinterpret_cast<uintptr_t>(p.src[k]) & 3) == 0;
        for (; t < all; t += step) {
            const long long r = all <= 0x7fffffff ? int(t) / runs : t / runs;
            const int c = (int(t - r * runs) * 32 + lane) * 8, n = w - c;
            if (n <= 0) continue;
            const uint16_t* x = p.src[k] + r * w + c;
            uint32_t v[4];
            if (words) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = 2 * e < n ? *reinterpret_cast<const uint32_t*>(x + 2 * e) : 0u;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = (2 * e < n ? uint32_t(x[2 * e]) : 0u) | (2 * e + 1 < n ? uint32_t(x[2 * e + 1]) << 16 : 0u);
            }
            *reinterpret_cast<uint4*>(p.dst[k] + r * p.wp[k] + c) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        t -= all;
    }
}

// The weight gradients from their slots, added in order and rounded to the type:
// slots [splits][R][ld] of each gradient [R, N].
template <typename T>
struct TrReduceParams {
    const float* part[3];
    T* out[3];
    int R[3], N[3], ld[3];
    int splits;
};

template <typename T>
__global__ void __launch_bounds__(256) evo_tr_mma_reduce_kernel(const TrReduceParams<T> p) {
    ptx::pdl_launch();
    ptx::pdl_wait();
    const int w = blockIdx.z, n = (blockIdx.y * 64 + (threadIdx.x & 63)) * 4, r = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (p.out[w] == nullptr || r >= p.R[w] || n >= p.N[w]) return;
    const size_t slot = size_t(p.R[w]) * p.ld[w];
    const float* x = p.part[w] + size_t(r) * p.ld[w] + n;
    float4 s = *reinterpret_cast<const float4*>(x);
#pragma unroll 4
    for (int k = 1; k < p.splits; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(x + k * slot);
        s.x += y.x, s.y += y.y, s.z += y.z, s.w += y.w;
    }
    T* o = p.out[w] + size_t(r) * p.N[w] + n;
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < p.N[w]) tr_store(o + e, v[e]);
}

}  // namespace evo
