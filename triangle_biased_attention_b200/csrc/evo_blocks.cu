// Host side of the operators around the attention: the gated transition and the
// learned relative-position bias (argument checks, workspace layouts and
// launches of the C entry points declared in include/evo_attn.h).
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <type_traits>

#include "evo_attn.h"
#include "common.cuh"
#include "host_util.cuh"
#include "relpos.cuh"
#include "transition_few.cuh"
#include "transition_simt.cuh"
#include "transition_sm100.cuh"

namespace evo {

int take_blocks_status(cudaStream_t stream, int* status) {
    return take_status_word(g_status, stream, status) ? EVO_OK : EVO_ERR_CUDA;
}

}  // namespace evo

namespace {

constexpr int64_t kIntMax = 2147483647;

int64_t elem_bytes(int dtype) { return dtype == EVO_DTYPE_FP32 ? 4 : 2; }

bool dtype_ok(int dtype) { return dtype == EVO_DTYPE_BF16 || dtype == EVO_DTYPE_FP32 || dtype == EVO_DTYPE_FP16; }

int sm_count(int dev) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

struct Buf {
    const void* p;
    int64_t bytes;
    bool written;
};

// Written buffers must not overlap any other buffer of the call.
bool any_overlap(std::initializer_list<Buf> bufs) {
    for (const Buf* a = bufs.begin(); a != bufs.end(); ++a)
        for (const Buf* b = a + 1; b != bufs.end(); ++b)
            if ((a->written || b->written) && overlap(a->p, a->bytes, b->p, b->bytes)) return true;
    return false;
}

// Every buffer must live on the first one's device; makes it current.
int select_device(std::initializer_list<const void*> ptrs, DeviceScope& scope) {
    int dev = -1;
    for (const void* p : ptrs) {
        if (p == nullptr) continue;
        if (dev < 0) {
            dev = select_device_of(p, scope);
            if (dev < 0) return dev;
            if (dev >= kMaxDevices) return EVO_ERR_UNSUPPORTED_SHAPE;
        } else if (device_of(p) != dev) {
            return EVO_ERR_INVALID_ARG;
        }
    }
    return dev;
}

// ------------------------------------------------------------------ transition

// Rows are taken in chunks, which bound the workspace: forward ones so that the
// [rows, F] intermediate stays in the 126 MB L2 between the kernel that writes it
// and the one that reads it, backward ones of 512 MB, because every chunk adds to
// the partial weight gradients once.  A chunk is a whole number of 128-row tiles
// for each of 148 SMs.
constexpr int64_t kTrWave = 148 * 128;

int64_t tr_chunk_rows(int64_t M, int64_t row_bytes, bool backward) {
    const int64_t target = int64_t(backward ? 512 : 64) << 20;
    // (and no more row tiles than a grid's y dimension, 65535, takes)
    const int64_t waves = std::min<int64_t>(440, std::max<int64_t>(1, target / (kTrWave * std::max<int64_t>(row_bytes, 1))));
    return std::min(M, waves * kTrWave);
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// fp32 products in parts: tiles of `rows` x `cols`, `splits` ranges of K with slots of
// their own (0: the kernel without parts).
struct TrPart {
    int rows = 128, cols = 128, splits = 0;
};

// Estimated microseconds of one 16-deep slab of a block's walk over K: with one block on an SM,
// for each of several, and how much longer where the rows are no whole 16-byte units.
// Measured at 1184 to 16384 rows, 512 x 1024 and 509 x 1021; blocks of one SM take turns on its
// shared memory and FMA units, so two take about twice as long as one.
struct TrTile {
    int rows, cols;
    double lone, shared, odd;
};
constexpr TrTile kTrTiles[] = {{128, 128, 1.95, 1.72, 1.07}, {128, 64, 1.08, 1.0, 1.17}, {32, 128, 0.95, 0.74, 1.15}};
constexpr TrTile kTrGate = {128, 64, 2.35, 1.84, 1.2}, kTrGrad = {128, 64, 2.85, 2.77, 1.15}, kTrDw = {128, 128, 3.1, 1.65, 1.13};

double tr_walk(const TrTile& t, int64_t blocks, int64_t K, bool odd) {
    const int64_t per = (blocks + 147) / 148;
    return double((K + evo::kTrK - 1) / evo::kTrK) * (per == 1 ? t.lone : double(per) * t.shared) * (odd ? t.odd : 1.0);
}

int64_t tr_tiles(const TrTile& t, int64_t rows, int64_t cols) { return (rows + t.rows - 1) / t.rows * ((cols + t.cols - 1) / t.cols); }

// Time of the kernels without parts.
double tr_gate_time(int64_t rows, int64_t C, int64_t F, bool backward) {
    const TrTile& t = backward ? kTrGrad : kTrGate;
    return tr_walk(t, tr_tiles(t, rows, F), C, C % 4 != 0);
}
double tr_out_time(int64_t rows, int64_t C, int64_t F, bool backward) {
    const TrTile& t = kTrTiles[tr_tiles(kTrTiles[0], rows, C) < 2 * 148 ? 1 : 0];
    return tr_walk(t, tr_tiles(t, rows, C), backward ? 2 * F : F, (backward ? C : F) % 4 != 0);
}

// The tile and ranges of `jobs` products [rows, K] x [K, N] in parts, or none where the
// kernel without parts (`whole`) is estimated faster.
TrPart tr_parts(int64_t rows, int64_t N, int64_t K, int64_t jobs, bool odd, double whole) {
    TrPart best;
    double least = 0.95 * whole;  // (what an estimate may be off by is not worth two launches)
    for (const TrTile& t : kTrTiles)
        for (int splits = 1; splits <= 64; splits += std::max(1, splits / 4)) {
            const int64_t slabs = (K + splits * evo::kTrK - 1) / (splits * evo::kTrK);
            const double bytes = 4.0 * double(rows) * double(N) * double(jobs) * splits;  // of the slots
            if ((splits > 1 && slabs < 2) || bytes > 128e6 || (rows + t.rows - 1) / t.rows > 65535) break;
            // another launch, the host's side of it included, and the slots read at 4 TB/s
            const double time = tr_walk(t, tr_tiles(t, rows, N) * jobs * splits, slabs * evo::kTrK, odd) + 7.0 + bytes / 4e6;
            if (time < least) {
                least = time;
                best.rows = t.rows, best.cols = t.cols, best.splits = splits;
            }
        }
    return best;
}

// Ranges of rows of the weight gradients, each with slots of its own: as estimated
// fastest, with the slots written and read at 4 TB/s.
int64_t tr_dw_splits(int64_t rows, int64_t C, int64_t F) {
    int64_t best = 1;
    double least = 0;
    for (int64_t splits = 1; splits <= 148; splits += std::max<int64_t>(1, splits / 8)) {
        const int64_t per = (rows + splits - 1) / splits;
        if (splits > 1 && per < 4 * evo::kTrK) break;
        const double time = tr_walk(kTrDw, 3 * tr_tiles(kTrDw, F, C) * splits, per, C % 4 != 0) + double(splits) * 24.0 * double(C) * double(F) / 4e6;
        if (splits == 1 || time < least) least = time, best = splits;
    }
    return best;
}

struct TrLayout {
    int64_t chunk = 0;                            // rows of a chunk
    int64_t h = 0, dg = 0, du = 0;                // [chunk, F] (16-bit: rows up to 128, F up to 128; fp32: F up to 4)
    int64_t part = 0, part2 = 0, part3 = 0;       // partial weight gradients, fp32: [splits][R][N up to 4] (fp32 call: one)
    bool direct = false;                          // 16-bit: the last products are the weight gradients
    int64_t splits = 0, split_rows = 0;           // ranges of rows with a slot of their own
    bool gradw = false;                           // the backward that keeps weight gradients on chip: no H, [C, F up to 64] slots
    TrPart grad, out;                             // fp32: G, U (and dH); Y or dX
    int64_t slots = 0;                            // their slots, one after the other
    bool few = false;                             // the forward's form for a few rows: H [M, F] in fp32
    bool fused = false;                           // the forward's one-kernel form: no [M, F] array at all
    int64_t x = 0, dy = 0, wg = 0, wu = 0, wd = 0;  // 16-bit, odd C or F: copies with rows of whole 16-byte units
    bool pad = false;
    int64_t total = 0;
};

// The form for a few rows reads X and H from shared memory, in groups of 8 rows.
// 16-bit, us, against the tensor cores: one row 2.9 / 5.3 (C = 64, F = 256) to 11.3 / 20.5
// (1024, 4096); 4 rows 5.1 / 7.1 (128, 512), 11.1 / 9.2 (256, 1024); 8 rows 7.5 / 7.1 (128, 512);
// where rows would have to be copied for TMA first, 8 rows 8.3 / 9.5 (100, 397), 14.9 / 16.7
// (388, 1555). With fp32 its time grows with M C F, and with the features of each group where
// rows of weights are short. Measured, us of the kernels, groups (two launches) against tiles in
// parts (four, so that a call not in a graph takes 26 at least): C = 64, F = 256: 128 rows 13.4 / 15.3,
// 256 18.0 / 15.4; C = 128, F = 512: 64 rows 15.8 / 16.7, 128 21.6 / 16.8; C = 256, F = 1024: 16 rows 17.5 /
// 18.4, 32 24.5 / 18.7; C = 384, F = 1536: 4 rows 15.0 / 20.6, 16 24.8 / 21.0, 32 44.7 / 21.2; C = 752, F = 3008:
// one row 14.2 / 32.9, 4 38.0 / 32.9 (odd rows read 4 bytes at a time, without bank
// conflicts: 896 x 3494, 5 rows 30 / 51; 987 x 564, 20 rows 22 / 30); C = 16, F = 2775: 16 rows 21.9 / 17.5, 64
// 38.6 / 18.6.
bool tr_few(int64_t M, int64_t C, int64_t F, int dtype) {
    if (8 * C * 4 > evo::kTrFewBytes || 8 * F * 4 > evo::kTrFewBytes) return false;
    if (dtype == EVO_DTYPE_FP32) {
        const int64_t most = C % 4 == 0 && F % 4 == 0 ? 10000000 : 26000000;
        return M <= 4 || (M * C * F <= most && (M + evo::kTrFewRows - 1) / evo::kTrFewRows * F <= 15000);
    }
    if (C % 8 == 0 && F % 8 == 0) return M == 1 || (M <= 4 && C * F <= 100000);
    return M == 1 || (M <= evo::kTrFewRows && C * F <= 700000);
}

// The one-kernel forward holds Y of 128 rows in tensor memory (C <= 256) and
// gives a tile of rows to one SM, which walks all features; the two-kernel form
// spreads the features of few rows over the SMs. Measured in turn, us, one kernel
// against two: C = 128, F = 512: 2048 rows 8.9 / 8.4, 4096 9.1 / 8.6, 6000 9.1 / 10.0,
// 147456 50 / 85; F = 1024: 6000 rows 14.2 / 13.5, 8192 14.5 / 15.0; C = 64, F = 256: 64 rows
// 5.4 / 6.6, 12000 6.2 / 9.3; C = 256, F = 512: 8192 rows 13.4 / 11.5, 12000 14.1 / 14.7,
// 131072 x 1024 144 / 194.
bool tr_fused(int64_t M, int64_t C, int64_t F, int dtype) {
    if (dtype == EVO_DTYPE_FP32 || C > 256) return false;
    const int64_t tiles = (M + 127) / 128, chunks = (F + 127) / 128;
    return C <= 128 ? chunks <= 2 || tiles >= 4 * (chunks + 6) : tiles > 90;
}

// The backward that holds 64 features' weight gradients in tensor memory, with up
// to 128 channels in its lanes. Against GRAD and DW apart, us: C = 128, F = 512: 64
// rows 16.3 / 14.9, 1024 18.3 / 22.3, 19000 42 / 51, 147456 215 / 271; C = 64, F = 256: 64 rows
// 11.1 / 12.4, 8192 17.0 / 21.7.
bool tr_gradw(int64_t C, int dtype) { return dtype != EVO_DTYPE_FP32 && C <= 128; }

// Sections on 256-byte boundaries.  False when a byte count passes int64.
bool tr_layout(int64_t M, int64_t C, int64_t F, int dtype, bool backward, TrLayout* L) {
    const int64_t es = elem_bytes(dtype);
    // C, F <= 2^20 and M < 2^31 (check_transition): the products below fit
    const int64_t fc = F * C;
    if (!backward && tr_few(M, C, F, dtype)) {
        L->few = true;
        L->chunk = M;
        L->total = round_up(M * F * 4, 256);
        return true;
    }
    const int64_t ldf = round_up(F, dtype == EVO_DTYPE_FP32 ? 4 : 128);
    L->pad = dtype != EVO_DTYPE_FP32 && (C % 8 != 0 || F % 8 != 0);
    L->fused = !backward && tr_fused(M, C, F, dtype);
    L->gradw = backward && tr_gradw(C, dtype);
    // (the one-kernel forward needs chunks only for the copy of X)
    L->chunk = L->fused ? (L->pad ? tr_chunk_rows(M, round_up(C, 8) * 2, false) : M)
                        : tr_chunk_rows(M, ldf * es * (backward ? (L->gradw ? 2 : 3) : 1), backward);
    const int64_t hbytes = (dtype == EVO_DTYPE_FP32 ? L->chunk : round_up(L->chunk, 128)) * ldf * es;
    int64_t off = 0;
    auto take = [&off](int64_t bytes) {
        const int64_t at = off;
        off += round_up(bytes, 256);
        return at;
    };
    if (!L->fused && !L->gradw) L->h = take(hbytes);
    if (dtype == EVO_DTYPE_FP32) {
        const int64_t jobs = backward ? 3 : 2, sums = backward ? 2 : 1;
        L->grad = tr_parts(L->chunk, F, C, jobs, C % 4 != 0, tr_gate_time(L->chunk, C, F, backward));
        L->out = tr_parts(L->chunk, C, F, sums, (backward ? C : F) % 4 != 0, tr_out_time(L->chunk, C, F, backward));
        const int64_t most = std::max(L->grad.splits * jobs * round_up(F, 4), L->out.splits * sums * round_up(C, 4));
        L->slots = take(L->chunk * most * 4);
    }
    if (backward) {
        L->dg = take(hbytes);
        L->du = take(hbytes);
        if (dtype == EVO_DTYPE_FP32) {
            L->splits = tr_dw_splits(L->chunk, C, F);
            L->split_rows = (L->chunk + L->splits - 1) / L->splits;
            L->part = take(L->splits * 3 * fc * 4);
        } else if (L->gradw) {
            // a share of the row tiles for each SM left by the feature slices
            L->splits = std::max<int64_t>(1, std::min(148 / ((F + 63) / 64), (L->chunk + 127) / 128));
            L->part = take(3 * L->splits * C * round_up(F, 64) * 4);
        } else {
            // as many ranges as keep the tiles within one wave of 148 SMs, none under 512
            // rows; one range, without slots, where the rows are few beside the weights,
            // so that the slots cost more than the shorter sums save. Whole backward with
            // one range against 512-row ones, us: C = 256, F = 512: 1024 rows 22.4 / 24.3,
            // 2048 28.8 / 25.6; C = 256, F = 1024: 2048 rows 32.7 / 39.3, 4096 48.9 / 44.4;
            // C = 384, F = 1536: 1024 rows 30.3 / 50.8, 4096 76.1 / 76.0
            const int64_t bn = C > 128 ? 256 : 128;
            const int64_t tiles = 2 * ((F + 127) / 128) * ((C + bn - 1) / bn) + ((C + 127) / 128) * ((F + 255) / 256);
            L->splits = !L->pad && L->chunk * 128 <= fc ? 1 : std::max<int64_t>(1, std::min(148 / tiles, (L->chunk + 511) / 512));
            L->split_rows = round_up((L->chunk + L->splits - 1) / L->splits, 64);
            L->direct = L->splits == 1 && L->chunk == M && !L->pad;
            if (!L->direct) {
                const int64_t fc4 = F * round_up(C, 4) * 4;
                L->part = take(L->splits * fc4);
                L->part2 = take(L->splits * fc4);
                L->part3 = take(L->splits * C * round_up(F, 4) * 4);
            }
        }
    }
    if (L->pad) {
        const int64_t cp = round_up(C, 8), fp = round_up(F, 8);
        L->x = take(L->chunk * cp * 2);
        if (backward) L->dy = take(L->chunk * cp * 2);
        L->wg = take(F * cp * 2);
        L->wu = take(F * cp * 2);
        L->wd = take(C * fp * 2);
    }
    L->total = off;
    return true;
}

int check_transition(int64_t M, int64_t C, int64_t F, int act, int dtype) {
    if (M < 0 || C < 0 || F < 0 || (act != EVO_ACT_SILU && act != EVO_ACT_GELU)) return EVO_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return EVO_ERR_UNSUPPORTED_DTYPE;
    // tile counts and row offsets inside a chunk are 32-bit
    if (M > kIntMax || C > (1 << 20) || F > (1 << 20)) return EVO_ERR_UNSUPPORTED_SHAPE;
    return EVO_OK;
}

constexpr int kTrSmem = 4 * evo::kTrK * evo::kTrLd * int(sizeof(float));

// Launches a kernel; `dependent`: it may start while the kernel before it in the
// stream still runs (it waits for that one's end itself).
template <typename K, typename... P>
bool launch_any(bool dependent, K kernel, dim3 grid, int threads, int smem, cudaStream_t st, const P&... p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    if (dependent) {
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, p...) == cudaSuccess;
}

template <typename K, typename P>
bool launch(K kernel, dim3 grid, int threads, int smem, cudaStream_t st, const P& p) {
    return launch_any(false, kernel, grid, threads, smem, st, p);
}

template <typename K, typename... P>
bool launch_dependent(K kernel, dim3 grid, int threads, int smem, cudaStream_t st, const P&... p) {
    return launch_any(true, kernel, grid, threads, smem, st, p...);
}

unsigned blocks_of(int64_t n, int64_t tile) { return unsigned((n + tile - 1) / tile); }

// Y or dX of one chunk.
template <bool BWD>
bool launch_simt_out(const evo::TrSimtParams& p, cudaStream_t st) {
    const unsigned mt = blocks_of(p.rows, 128);
    if (int64_t(blocks_of(p.C, 128)) * mt < 2 * 148)
        return launch(evo::evo_tr_simt_out_kernel<BWD, 1>, dim3(blocks_of(p.C, 64), mt), evo::kTrThreads, kTrSmem, st, p);
    return launch(evo::evo_tr_simt_out_kernel<BWD, 2>, dim3(blocks_of(p.C, 128), mt), evo::kTrThreads, kTrSmem, st, p);
}

// One stage of products in parts; the slots' sums are the caller's.
template <int B_LAYOUT>
bool launch_parts(const TrPart& t, evo::TrPartParams& p, cudaStream_t st) {
    p.splits = t.splits;
    p.ld = int(round_up(p.N, 4));
    const dim3 grid(blocks_of(p.N, t.cols), blocks_of(p.rows, t.rows), unsigned(p.jobs * t.splits));
    if (t.rows == 32) return launch(evo::evo_tr_simt_part_kernel<32, 2, B_LAYOUT>, grid, evo::kTrThreads, kTrSmem, st, p);
    return t.cols == 128 ? launch(evo::evo_tr_simt_part_kernel<128, 2, B_LAYOUT>, grid, evo::kTrThreads, kTrSmem, st, p)
                         : launch(evo::evo_tr_simt_part_kernel<128, 1, B_LAYOUT>, grid, evo::kTrThreads, kTrSmem, st, p);
}

// G and U (and dH with `backward`) in parts, then H (dG, dU).
template <int ACT, bool BWD>
bool run_gate_parts(const TrPart& t, const evo::TrSimtParams& p, float* slots, cudaStream_t st) {
    evo::TrPartParams q = {};
    q.jobs = BWD ? 3 : 2;
    q.job[0] = {p.x, p.wg, p.C, true, p.vc, p.vc};
    q.job[1] = {p.x, p.wu, p.C, true, p.vc, p.vc};
    q.job[2] = {p.dy, p.wd, p.C, false, p.vc, p.vd};
    q.rows = p.rows;
    q.N = p.F;
    q.K = p.C;
    q.slots = slots;
    return launch_parts<BWD ? evo::TR_B_MIXED : evo::TR_B_K>(t, q, st) &&
           launch_any(false, evo::evo_tr_join_act_kernel<ACT, BWD>, dim3(blocks_of(int64_t(q.rows) * q.ld / 4, 256)), 256, 0, st,
                      (const float*)slots, q.splits, q.rows, q.ld, p.h, p.dg, p.du);
}

// Y or dX in parts.
template <bool BWD>
bool run_out_parts(const TrPart& t, const evo::TrSimtParams& p, float* slots, cudaStream_t st) {
    evo::TrPartParams q = {};
    q.jobs = BWD ? 2 : 1;
    q.job[0] = {BWD ? p.dg : p.h, BWD ? p.wg : p.wd, p.ldf, !BWD, true, BWD ? p.vc : p.vd};
    q.job[1] = {p.du, p.wu, p.ldf, false, true, p.vc};
    q.rows = p.rows;
    q.N = p.C;
    q.K = p.F;
    q.slots = slots;
    return launch_parts<BWD ? evo::TR_B_N : evo::TR_B_K>(t, q, st) &&
           launch_any(false, evo::evo_tr_join_out_kernel, dim3(blocks_of(int64_t(q.rows) * q.ld / 4, 256)), 256, 0, st,
                      (const float*)slots, q.jobs * q.splits, q.rows, q.N, q.ld, p.out, int(p.vo));
}

template <int ACT>
int run_fwd_simt(const TrLayout& L, const float* X, const float* Wg, const float* Wu, const float* Wd, float* Y, char* ws, int64_t M,
                 int64_t C, int64_t F, cudaStream_t st) {
    evo::TrSimtParams p = {};
    p.wg = Wg;
    p.wu = Wu;
    p.wd = Wd;
    p.h = reinterpret_cast<float*>(ws + L.h);
    float* const slots = reinterpret_cast<float*>(ws + L.slots);
    p.C = int(C);
    p.F = int(F);
    p.ldf = int(round_up(F, 4));
    p.vc = C % 4 == 0 && aligned(X, 16) && aligned(Wg, 16) && aligned(Wu, 16);
    p.vd = F % 4 == 0 && aligned(Wd, 16);
    p.vo = C % 4 == 0 && aligned(Y, 16);
    for (int64_t m = 0; m < M; m += L.chunk) {
        p.rows = int(std::min(L.chunk, M - m));
        p.x = X + m * C;
        p.out = Y + m * C;
        const unsigned mt = blocks_of(p.rows, 128);
        if (!(L.grad.splits ? run_gate_parts<ACT, false>(L.grad, p, slots, st)
                            : launch(evo::evo_tr_simt_gate_kernel<ACT>, dim3(blocks_of(F, 64), mt), evo::kTrThreads, kTrSmem, st, p)) ||
            !(L.out.splits ? run_out_parts<false>(L.out, p, slots, st) : launch_simt_out<false>(p, st)))
            return EVO_ERR_CUDA;
    }
    return EVO_OK;
}

template <int ACT>
int run_bwd_simt(const TrLayout& L, const float* X, const float* Wg, const float* Wu, const float* Wd, const float* dY, float* dX,
                 float* dWg, float* dWu, float* dWd, char* ws, int64_t M, int64_t C, int64_t F, cudaStream_t st) {
    evo::TrSimtParams p = {};
    p.wg = Wg;
    p.wu = Wu;
    p.wd = Wd;
    p.h = reinterpret_cast<float*>(ws + L.h);
    p.dg = reinterpret_cast<float*>(ws + L.dg);
    p.du = reinterpret_cast<float*>(ws + L.du);
    p.part = reinterpret_cast<float*>(ws + L.part);
    float* const slots = reinterpret_cast<float*>(ws + L.slots);
    p.C = int(C);
    p.F = int(F);
    p.splits = int(L.splits);
    p.split_rows = int(L.split_rows);
    p.dw_mask = (dWg ? 1 : 0) | (dWu ? 2 : 0) | (dWd ? 4 : 0);
    p.ldf = int(round_up(F, 4));
    p.vc = C % 4 == 0 && aligned(X, 16) && aligned(dY, 16) && aligned(Wg, 16) && aligned(Wu, 16);
    p.vd = F % 4 == 0 && aligned(Wd, 16);
    p.vo = C % 4 == 0 && aligned(dX, 16);
    for (int64_t m = 0; m < M; m += L.chunk) {
        p.rows = int(std::min(L.chunk, M - m));
        p.x = X + m * C;
        p.dy = dY + m * C;
        p.out = dX ? dX + m * C : nullptr;
        p.first = m == 0;
        const unsigned mt = blocks_of(p.rows, 128), big = blocks_of(std::max(C, F), 128);
        if (!(L.grad.splits ? run_gate_parts<ACT, true>(L.grad, p, slots, st)
                            : launch(evo::evo_tr_simt_grad_kernel<ACT>, dim3(blocks_of(F, 64), mt), evo::kTrThreads, kTrSmem, st, p)) ||
            (dX && !(L.out.splits ? run_out_parts<true>(L.out, p, slots, st) : launch_simt_out<true>(p, st))) ||
            (p.dw_mask && !launch(evo::evo_tr_simt_dw_kernel, dim3(big, big, unsigned(3 * L.splits)),
                                  evo::kTrThreads, kTrSmem, st, p)))
            return EVO_ERR_CUDA;
    }
    if (p.dw_mask) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(blocks_of(F * C, 256), 1, 1);
        cfg.blockDim = dim3(256, 1, 1);
        cfg.stream = st;
        if (cudaLaunchKernelEx(&cfg, evo::evo_tr_dw_reduce_kernel, (const float*)p.part, p.splits, (long long)(F * C),
                               dWg, dWu, dWd) != cudaSuccess)
            return EVO_ERR_CUDA;
    }
    return EVO_OK;
}

// A 16-bit matrix of `rows` rows of `cols` elements, `ld` apart; a box is 64 (or
// 32) columns of `box_rows` rows, swizzled over its 128 B (64 B) rows.
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool f16,
                 int box_cols = 64) {
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld * 2)};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return encode_fn()(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                       const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One product over one chunk of rows, a CTA per SM.
template <int KIND, int ACT, bool F16, int BN>
int launch_mma(int dev, int sms, const evo::TrMaps& maps, const evo::TrMmaParams& p, cudaStream_t st) {
    using Cfg = evo::TrCfg<KIND, BN, F16>;
    auto kernel = evo::evo_tr_mma_kernel<KIND, ACT, F16, BN>;
    static AttrOnce attr;
    if (!attr.ensure(dev, kernel, Cfg::SMEM_BYTES)) return EVO_ERR_CUDA;
    const int tiles = KIND == evo::TR_DW ? p.num_tiles * p.tiles_n : p.num_tiles;
    return launch_dependent(kernel, dim3(unsigned(std::min(tiles, sms))), Cfg::THREADS, Cfg::SMEM_BYTES, st, maps, p)
               ? EVO_OK
               : EVO_ERR_CUDA;
}

// What a 16-bit call reads through TMA: the tensors themselves, or copies with
// rows of whole 16-byte units.
struct TrSource {
    const void *x, *dy, *wg, *wu, *wd;
    int64_t ldc, ldf;  // row strides of x, dy, wg, wu and of wd
};

struct PadList {
    evo::TrPads p = {};
    void add(const void* src, void* dst, int64_t rows, int64_t w) {
        p.src[p.n] = static_cast<const uint16_t*>(src);
        p.dst[p.n] = static_cast<uint16_t*>(dst);
        p.rows[p.n] = int(rows);
        p.w[p.n] = int(w);
        p.wp[p.n++] = int(round_up(w, 8));
    }
    bool run(int sms, cudaStream_t st) {
        int64_t runs = 0;  // of 32 16-byte units, a warp's work
        for (int k = 0; k < p.n; ++k) runs += int64_t(p.rows[k]) * ((p.wp[k] + 255) / 256);
        return launch_dependent(evo::evo_tr_pad_kernel, dim3(unsigned(std::min<int64_t>((runs + 7) / 8, int64_t(sms) * 8))), 256, 0, st, p);
    }
};

// Copies of the chunk's rows of x and dy and, with the first chunk, of the weights.
bool pad_chunk(const TrLayout& L, char* ws, TrSource* s, const void** x, const void** dy, int64_t rows, bool weights,
               int64_t C, int64_t F, int sms, cudaStream_t st) {
    PadList list;
    list.add(*x, ws + L.x, rows, C);
    *x = ws + L.x;
    if (dy) {
        list.add(*dy, ws + L.dy, rows, C);
        *dy = ws + L.dy;
    }
    if (weights) {
        list.add(s->wg, ws + L.wg, F, C);
        list.add(s->wu, ws + L.wu, F, C);
        list.add(s->wd, ws + L.wd, C, F);
        s->wg = ws + L.wg;
        s->wu = ws + L.wu;
        s->wd = ws + L.wd;
        s->ldc = round_up(C, 8);
        s->ldf = round_up(F, 8);
    }
    return list.run(sms, st);
}

// Whether TMA can store rows of C 16-bit elements at p.
bool tma_rows(const void* p, int64_t C) { return C % 8 == 0 && aligned(p, 16); }

int tiles_of(int64_t n, int64_t tile) { return int((n + tile - 1) / tile); }

// Channels of a tile of Y or dX: 256 where there are more than 128 and tiles
// enough for the SMs, 64 where tiles of 128 would leave half of the SMs idle.
int out_width(int rows, int64_t C, int sms) {
    const int tiles = tiles_of(rows, 128) * tiles_of(C, 128);
    return C > 128 && tiles > sms ? 256 : 2 * tiles <= sms ? 64 : 128;
}

// Y or dX of one chunk.
template <int KIND, bool F16>
int launch_out(int dev, int sms, evo::TrMaps& maps, evo::TrMmaParams p, void* out, cudaStream_t st) {
    p.out = static_cast<uint16_t*>(out);
    p.tma_out = tma_rows(out, p.C);
    if (p.tma_out && !encode_rows(&maps.m[KIND == evo::TR_OUT ? 2 : 4], out, p.rows, p.C, p.C, 32, F16, 32)) return EVO_ERR_CUDA;
    const int width = out_width(p.rows, p.C, sms);
    p.tiles_m = tiles_of(p.rows, 128);
    p.tiles_n = tiles_of(p.C, width);
    p.num_tiles = p.tiles_m * p.tiles_n;
    p.kb = tiles_of(p.F, 64);
    return width == 256   ? launch_mma<KIND, 0, F16, 256>(dev, sms, maps, p, st)
           : width == 128 ? launch_mma<KIND, 0, F16, 128>(dev, sms, maps, p, st)
                          : launch_mma<KIND, 0, F16, 64>(dev, sms, maps, p, st);
}

template <int ACT, bool F16, int CN>
int launch_fused(int dev, int sms, const void* x, const TrSource& s, uint16_t* y, int rows, int64_t C, int64_t F, int wide,
                 cudaStream_t st) {
    using Cfg = evo::TrFusedCfg<F16, CN>;
    auto kernel = evo::evo_tr_fused_kernel<ACT, F16, CN>;
    static AttrOnce attr;
    if (!attr.ensure(dev, kernel, Cfg::SMEM_BYTES)) return EVO_ERR_CUDA;
    evo::TrMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    if (!encode_rows(&maps.m[0], x, rows, C, s.ldc, 128, F16) || !encode_rows(&maps.m[1], s.wg, F, C, s.ldc, 128, F16) ||
        !encode_rows(&maps.m[2], s.wu, F, C, s.ldc, 128, F16) || !encode_rows(&maps.m[3], s.wd, C, F, s.ldf, 128, F16) ||
        (wide && !encode_rows(&maps.m[4], y, rows, C, C, 32, F16, 32)))
        return EVO_ERR_CUDA;
    evo::TrFusedParams p = {};
    p.out = y;
    p.M = rows;
    p.C = int(C);
    p.F = int(F);
    p.num_tiles = tiles_of(rows, 128);
    p.kc = tiles_of(C, 64);
    p.chunks = tiles_of(F, 128);
    p.wide_store = wide;
    return launch_dependent(kernel, dim3(unsigned(std::min(p.num_tiles, sms))), Cfg::THREADS, Cfg::SMEM_BYTES, st, maps, p)
               ? EVO_OK
               : EVO_ERR_CUDA;
}

template <bool F16, int ACT>
int run_fwd_mma(int dev, const void* X, const void* Wg, const void* Wu, const void* Wd, void* Y, char* ws, int64_t M,
                int64_t C, int64_t F, int dtype, cudaStream_t st) {
    const int sms = sm_count(dev);
    if (sms <= 0 || encode_fn() == nullptr) return EVO_ERR_CUDA;
    TrLayout L;
    tr_layout(M, C, F, dtype, false, &L);
    TrSource s = {X, nullptr, Wg, Wu, Wd, C, F};
    evo::TrMmaParams p = {};
    p.C = int(C);
    p.F = int(F);
    const int64_t ldf = round_up(F, 128);
    for (int64_t m = 0; m < M; m += L.chunk) {
        p.rows = int(std::min(L.chunk, M - m));
        const void* x = static_cast<const char*>(X) + m * C * 2;
        uint16_t* y = static_cast<uint16_t*>(Y) + m * C;
        if (L.pad && !pad_chunk(L, ws, &s, &x, nullptr, p.rows, m == 0, C, F, sms, st)) return EVO_ERR_CUDA;
        if (L.fused) {
            const int fst = C > 128 ? launch_fused<ACT, F16, 256>(dev, sms, x, s, y, p.rows, C, F, tma_rows(y, C), st)
                                    : launch_fused<ACT, F16, 128>(dev, sms, x, s, y, p.rows, C, F, tma_rows(y, C), st);
            if (fst != EVO_OK) return fst;
            continue;
        }
        evo::TrMaps gate, out;
        std::memset(&gate, 0, sizeof(gate));
        std::memset(&out, 0, sizeof(out));
        if (!encode_rows(&gate.m[0], x, p.rows, C, s.ldc, 128, F16) || !encode_rows(&gate.m[1], s.wg, F, C, s.ldc, 128, F16) ||
            !encode_rows(&gate.m[2], s.wu, F, C, s.ldc, 128, F16) ||
            !encode_rows(&gate.m[3], ws + L.h, p.rows, ldf, ldf, 32, F16, 32) ||
            !encode_rows(&out.m[0], ws + L.h, p.rows, ldf, ldf, 128, F16) || !encode_rows(&out.m[1], s.wd, C, F, s.ldf, out_width(p.rows, C, sms) == 64 ? 64 : 128, F16))
            return EVO_ERR_CUDA;
        p.tiles_m = tiles_of(p.rows, 128);
        p.tiles_n = tiles_of(F, 128);
        p.num_tiles = p.tiles_m * p.tiles_n;
        p.kb = tiles_of(C, 64);
        if (launch_mma<evo::TR_GATE, ACT, F16, 256>(dev, sms, gate, p, st) != EVO_OK ||
            launch_out<evo::TR_OUT, F16>(dev, sms, out, p, y, st) != EVO_OK)
            return EVO_ERR_CUDA;
    }
    return EVO_OK;
}

// The slots of one weight gradient as a 3-D tensor {N, R, splits} of fp32; a box
// is 32 columns (128 B rows, 128 B swizzle) of 32 rows.
bool encode_slots(CUtensorMap* m, void* base, int64_t splits, int64_t R, int64_t N) {
    const int64_t ld = round_up(N, 4);
    const cuuint64_t dims[3] = {cuuint64_t(N), cuuint64_t(R), cuuint64_t(splits)};
    const cuuint64_t strides[2] = {cuuint64_t(ld * 4), cuuint64_t(R * ld * 4)};
    const cuuint32_t box[3] = {32, 32, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// dG, dU and the weight gradients' sums of one chunk (C <= 128), with the maps of GRAD and DX.
template <int ACT, bool F16>
int launch_gradw(int dev, const evo::TrMaps& grad, const evo::TrMaps& dx, const TrLayout& L, char* ws, bool need_dx, int rows,
                 bool first, int64_t C, int64_t F, cudaStream_t st) {
    using Cfg = evo::TrGradwCfg<F16>;
    auto kernel = evo::evo_tr_gradw_kernel<ACT, F16>;
    static AttrOnce attr;
    if (!attr.ensure(dev, kernel, Cfg::SMEM_BYTES)) return EVO_ERR_CUDA;
    evo::TrGradwParams p = {};
    p.d[0] = need_dx ? reinterpret_cast<uint16_t*>(ws + L.dg) : nullptr;
    p.d[1] = need_dx ? reinterpret_cast<uint16_t*>(ws + L.du) : nullptr;
    p.part = reinterpret_cast<float*>(ws + L.part);
    p.ldf = int(round_up(F, 128));
    p.ldp = int(round_up(F, 64));
    p.M = rows;
    p.C = int(C);
    p.F = int(F);
    p.num_tiles = tiles_of(rows, 128);
    p.kc = tiles_of(C, 64);
    p.slices = tiles_of(F, Cfg::FC);
    p.splits = int(L.splits);
    p.first = first;
    evo::TrMaps a;  // X, dY, Wg, Wu (boxes of 64 rows), Wd
    std::memset(&a, 0, sizeof(a));
    a.m[0] = grad.m[0];
    a.m[1] = grad.m[3];
    a.m[2] = dx.m[1];
    a.m[3] = dx.m[3];
    a.m[4] = grad.m[4];
    return launch_dependent(kernel, dim3(unsigned(p.slices * p.splits)), Cfg::THREADS, Cfg::SMEM_BYTES, st, a, p) ? EVO_OK
                                                                                                                : EVO_ERR_CUDA;
}

template <bool F16, int ACT>
int run_bwd_mma(int dev, const void* X, const void* Wg, const void* Wu, const void* Wd, const void* dY, void* dX,
                void* dWg, void* dWu, void* dWd, char* ws, int64_t M, int64_t C, int64_t F, int dtype, cudaStream_t st) {
    using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
    const int sms = sm_count(dev);
    if (sms <= 0 || encode_fn() == nullptr) return EVO_ERR_CUDA;
    TrLayout L;
    tr_layout(M, C, F, dtype, true, &L);
    TrSource s = {X, dY, Wg, Wu, Wd, C, F};
    evo::TrMmaParams p = {};
    p.C = int(C);
    p.F = int(F);
    const int64_t ldf = round_up(F, 128);
    p.split_rows = int(L.split_rows);
    p.direct = L.direct;
    p.bn01 = C > 128 ? 256 : 128;
    p.tn01 = tiles_of(C, p.bn01);
    p.tn2 = tiles_of(F, 256);
    p.tiles01 = p.tn01 * tiles_of(F, 128);
    p.tiles2 = p.tn2 * tiles_of(C, 128);
    void* const dw[3] = {dWg, dWu, dWd};
    char* const part[3] = {ws + L.part, ws + L.part2, ws + L.part3};
    int dw_tiles = 0;
    for (int w = 0; w < 3; ++w)
        if (dw[w]) {
            p.which[p.num_which++] = w;
            dw_tiles += w == 2 ? p.tiles2 : p.tiles01;
        }
    for (int64_t m = 0; m < M; m += L.chunk) {
        p.rows = int(std::min(L.chunk, M - m));
        p.first = m == 0;
        const void* x = static_cast<const char*>(X) + m * C * 2;
        const void* dy = static_cast<const char*>(dY) + m * C * 2;
        if (L.pad && !pad_chunk(L, ws, &s, &x, &dy, p.rows, m == 0, C, F, sms, st)) return EVO_ERR_CUDA;
        char *h = ws + L.h, *dg = ws + L.dg, *du = ws + L.du;
        evo::TrMaps grad, out, wgt;
        std::memset(&grad, 0, sizeof(grad));
        std::memset(&out, 0, sizeof(out));
        std::memset(&wgt, 0, sizeof(wgt));
        if (!encode_rows(&grad.m[0], x, p.rows, C, s.ldc, 128, F16) || !encode_rows(&grad.m[3], dy, p.rows, C, s.ldc, 128, F16) ||
            !encode_rows(&grad.m[4], s.wd, C, F, s.ldf, 64, F16))
            return EVO_ERR_CUDA;
        if (!L.gradw &&
            (!encode_rows(&grad.m[1], s.wg, F, C, s.ldc, 128, F16) || !encode_rows(&grad.m[2], s.wu, F, C, s.ldc, 128, F16) ||
             !encode_rows(&grad.m[5], h, p.rows, ldf, ldf, 32, F16, 32) || !encode_rows(&grad.m[6], dg, p.rows, ldf, ldf, 32, F16, 32) ||
             !encode_rows(&grad.m[7], du, p.rows, ldf, ldf, 32, F16, 32)))
            return EVO_ERR_CUDA;
        if ((L.gradw || dX) &&
            (!encode_rows(&out.m[1], s.wg, F, C, s.ldc, 64, F16) || !encode_rows(&out.m[3], s.wu, F, C, s.ldc, 64, F16)))
            return EVO_ERR_CUDA;
        if (dX && (!encode_rows(&out.m[0], dg, p.rows, ldf, ldf, 128, F16) || !encode_rows(&out.m[2], du, p.rows, ldf, ldf, 128, F16)))
            return EVO_ERR_CUDA;
        if (!L.gradw && p.num_which > 0 &&
            (!encode_rows(&wgt.m[0], x, p.rows, C, s.ldc, 64, F16) || !encode_rows(&wgt.m[1], dy, p.rows, C, s.ldc, 64, F16) ||
             !encode_rows(&wgt.m[2], dg, p.rows, ldf, ldf, 64, F16) || !encode_rows(&wgt.m[3], du, p.rows, ldf, ldf, 64, F16) ||
             !encode_rows(&wgt.m[4], h, p.rows, ldf, ldf, 64, F16)))
            return EVO_ERR_CUDA;
        for (int w = 0; w < 3; ++w) {
            const int64_t R = w == 2 ? C : F, N = w == 2 ? F : C;
            if (dw[w] && !L.gradw && !(L.direct ? encode_rows(&wgt.m[5 + w], dw[w], R, N, N, 32, F16, 32)
                                    : encode_slots(&wgt.m[5 + w], part[w], L.splits, R, N)))
                return EVO_ERR_CUDA;
        }
        p.tiles_m = tiles_of(p.rows, 128);
        p.tiles_n = tiles_of(F, 128);
        p.num_tiles = p.tiles_m * p.tiles_n;
        p.kb = tiles_of(C, 64);
        if (L.gradw) {
            if (launch_gradw<ACT, F16>(dev, grad, out, L, ws, dX != nullptr, p.rows, m == 0, C, F, st) != EVO_OK)
                return EVO_ERR_CUDA;
        } else if (launch_mma<evo::TR_GRAD, ACT, F16, 256>(dev, sms, grad, p, st) != EVO_OK) {
            return EVO_ERR_CUDA;
        }
        if (dX && launch_out<evo::TR_DX, F16>(dev, sms, out, p, static_cast<uint16_t*>(dX) + m * C, st) != EVO_OK)
            return EVO_ERR_CUDA;
        if (p.num_which > 0 && !L.gradw) {
            p.num_tiles = dw_tiles;
            p.tiles_n = int(L.splits);
            if (launch_mma<evo::TR_DW, 0, F16, 256>(dev, sms, wgt, p, st) != EVO_OK) return EVO_ERR_CUDA;
        }
    }
    if (L.gradw) {
        if (p.num_which > 0 &&
            !launch_dependent(evo::evo_tr_gradw_reduce_kernel<T>, dim3(blocks_of(F, 32), blocks_of(C, 8), 3), 256, 0, st,
                              reinterpret_cast<const float*>(ws + L.part), int(L.splits), p.C, p.F, int(round_up(F, 64)),
                              static_cast<T*>(dWg), static_cast<T*>(dWu), static_cast<T*>(dWd)))
            return EVO_ERR_CUDA;
        return EVO_OK;
    }
    if (p.num_which > 0 && !L.direct) {
        evo::TrReduceParams<T> r = {};
        r.splits = int(L.splits);
        for (int w = 0; w < 3; ++w) {
            r.part[w] = reinterpret_cast<const float*>(part[w]);
            r.out[w] = static_cast<T*>(dw[w]);
            r.R[w] = int(w == 2 ? C : F);
            r.N[w] = int(w == 2 ? F : C);
            r.ld[w] = int(round_up(r.N[w], 4));
        }
        const int64_t big = std::max(C, F);
        if (!launch_dependent(evo::evo_tr_mma_reduce_kernel<T>, dim3(blocks_of(big, 4), blocks_of(big, 256), 3), 256, 0, st, r))
            return EVO_ERR_CUDA;
    }
    return EVO_OK;
}

template <typename T, int ACT, int MB>
int run_few(int dev, const evo::TrFewParams<T>& p, bool vec, cudaStream_t st) {
    constexpr int VE = 16 / int(sizeof(T));
    constexpr int WIDE = MB == 8 && sizeof(T) == 2 ? 1 : VE;  // (tr_few: no whole 16-byte units there)
    auto gate = vec ? evo::evo_tr_few_gate_kernel<T, ACT, MB, WIDE> : evo::evo_tr_few_gate_kernel<T, ACT, MB, 1>;
    auto out = vec ? evo::evo_tr_few_out_kernel<T, MB, WIDE> : evo::evo_tr_few_out_kernel<T, MB, 1>;
    static AttrOnce attr[2][2];
    if (!attr[0][vec].ensure(dev, gate, evo::kTrFewBytes) || !attr[1][vec].ensure(dev, out, evo::kTrFewBytes))
        return EVO_ERR_CUDA;
    const unsigned blocks = std::min(blocks_of(p.F, 8), 148u * 8);
    const unsigned channels = blocks_of(p.C, 8 / p.split), groups = blocks_of(p.M, MB);
    return launch_dependent(gate, dim3(blocks, groups), evo::kTrFewThreads, MB * p.C * 4, st, p) &&
                   launch_dependent(out, dim3(channels, groups), evo::kTrFewThreads, MB * p.F * 4, st, p)
               ? EVO_OK
               : EVO_ERR_CUDA;
}

template <typename T>
int run_fwd_few(int dev, const void* X, const void* Wg, const void* Wu, const void* Wd, void* Y, char* ws, int64_t M, int64_t C,
                int64_t F, int act, cudaStream_t st) {
    constexpr int VE = 16 / int(sizeof(T));
    evo::TrFewParams<T> p = {};
    p.x = static_cast<const T*>(X);
    p.wg = static_cast<const T*>(Wg);
    p.wu = static_cast<const T*>(Wu);
    p.wd = static_cast<const T*>(Wd);
    p.y = static_cast<T*>(Y);
    p.h = reinterpret_cast<float*>(ws);
    p.M = int(M);
    p.C = int(C);
    p.F = int(F);
    // warps enough for every SM, while each still reads whole rounds of its row
    p.split = 1;
    while (p.split < 8 && C * p.split < 148 * 8 && F >= int64_t(2) * p.split * 32 * VE) p.split *= 2;
    const bool vec = C % VE == 0 && F % VE == 0 && aligned(Wg, 16) && aligned(Wu, 16) && aligned(Wd, 16);
    const bool silu = act == EVO_ACT_SILU;
    if (M == 1) return silu ? run_few<T, EVO_ACT_SILU, 1>(dev, p, vec, st) : run_few<T, EVO_ACT_GELU, 1>(dev, p, vec, st);
    if (M <= 4) return silu ? run_few<T, EVO_ACT_SILU, 4>(dev, p, vec, st) : run_few<T, EVO_ACT_GELU, 4>(dev, p, vec, st);
    return silu ? run_few<T, EVO_ACT_SILU, 8>(dev, p, vec, st) : run_few<T, EVO_ACT_GELU, 8>(dev, p, vec, st);
}

int64_t tr_workspace(int64_t M, int64_t C, int64_t F, int dtype, bool backward) {
    const int st = check_transition(M, C, F, EVO_ACT_SILU, dtype);
    if (st != EVO_OK) return st;
    if (M == 0 || C == 0 || F == 0) return 0;
    TrLayout L;
    if (!tr_layout(M, C, F, dtype, backward, &L)) return EVO_ERR_UNSUPPORTED_SHAPE;
    return L.total;
}

// the alignment every tensor of a transition call needs
uintptr_t tr_alignment(int64_t C, int64_t F, int dtype) {
    if (dtype == EVO_DTYPE_FP32) return 4;
    return C % 8 == 0 && F % 8 == 0 ? 16 : 2;
}

bool zero(void* p, int64_t bytes, cudaStream_t st) {
    return p == nullptr || bytes == 0 || cudaMemsetAsync(p, 0, size_t(bytes), st) == cudaSuccess;
}

}  // namespace

extern "C" EVO_API int64_t evo_transition_fwd_workspace_size(int64_t M, int64_t C, int64_t F, int dtype) {
    return tr_workspace(M, C, F, dtype, false);
}

extern "C" EVO_API int64_t evo_transition_bwd_workspace_size(int64_t M, int64_t C, int64_t F, int dtype) {
    return tr_workspace(M, C, F, dtype, true);
}

extern "C" EVO_API int evo_transition_fwd(const void* X, const void* Wg, const void* Wu, const void* Wd, void* Y,
                                          void* workspace, int64_t workspace_bytes, int64_t M, int64_t C, int64_t F,
                                          int act, int dtype, evo_stream_t stream) {
    const int chk = check_transition(M, C, F, act, dtype);
    if (chk != EVO_OK) return chk;
    if (workspace_bytes < 0) return EVO_ERR_INVALID_ARG;
    if (M == 0 || C == 0) return EVO_OK;  // Y is empty
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t es = elem_bytes(dtype);
    if (!Y || (F > 0 && (!X || !Wg || !Wu || !Wd))) return EVO_ERR_INVALID_ARG;
    TrLayout L;
    if (F > 0 && !tr_layout(M, C, F, dtype, false, &L)) return EVO_ERR_UNSUPPORTED_SHAPE;
    const int64_t xb = M * C * es, wb = F * C * es;
    if (F > 0) {
        if (workspace_bytes < L.total || (!workspace && L.total > 0)) return EVO_ERR_INVALID_ARG;
        if (L.total == 0) workspace = nullptr;  // not used
        for (const void* p : {X, Wg, Wu, Wd, static_cast<const void*>(Y)})
            if (!aligned(p, tr_alignment(C, F, dtype))) return EVO_ERR_MISALIGNED;
        if (!aligned(workspace, 256)) return EVO_ERR_MISALIGNED;
        if (any_overlap({{Y, xb, true}, {workspace, L.total, true}, {X, xb, false}, {Wg, wb, false}, {Wu, wb, false},
                         {Wd, wb, false}}))
            return EVO_ERR_INVALID_ARG;
    }
    RelaxedCapture relaxed;
    DeviceScope scope;
    if (F == 0) {  // an empty sum
        const int dev = select_device({Y}, scope);
        return dev < 0 ? dev : zero(Y, xb, st) ? EVO_OK : EVO_ERR_CUDA;
    }
    const int dev = select_device({X, Wg, Wu, Wd, Y, workspace}, scope);
    if (dev < 0) return dev;
    char* ws = static_cast<char*>(workspace);
    if (L.few) {
        auto run = dtype == EVO_DTYPE_FP32 ? run_fwd_few<float> : dtype == EVO_DTYPE_FP16 ? run_fwd_few<__half> : run_fwd_few<__nv_bfloat16>;
        return run(dev, X, Wg, Wu, Wd, Y, ws, M, C, F, act, st);
    }
    if (dtype == EVO_DTYPE_FP32) {
        auto f = [](const void* p) { return static_cast<const float*>(p); };
        auto run = act == EVO_ACT_SILU ? run_fwd_simt<EVO_ACT_SILU> : run_fwd_simt<EVO_ACT_GELU>;
        return run(L, f(X), f(Wg), f(Wu), f(Wd), static_cast<float*>(Y), ws, M, C, F, st);
    }
    auto run = dtype == EVO_DTYPE_FP16
                   ? (act == EVO_ACT_SILU ? run_fwd_mma<true, EVO_ACT_SILU> : run_fwd_mma<true, EVO_ACT_GELU>)
                   : (act == EVO_ACT_SILU ? run_fwd_mma<false, EVO_ACT_SILU> : run_fwd_mma<false, EVO_ACT_GELU>);
    return run(dev, X, Wg, Wu, Wd, Y, ws, M, C, F, dtype, st);
}

extern "C" EVO_API int evo_transition_bwd(const void* X, const void* Wg, const void* Wu, const void* Wd,
                                          const void* dY, void* dX, void* dWg, void* dWu, void* dWd, void* workspace,
                                          int64_t workspace_bytes, int64_t M, int64_t C, int64_t F, int act, int dtype,
                                          evo_stream_t stream) {
    const int chk = check_transition(M, C, F, act, dtype);
    if (chk != EVO_OK) return chk;
    if (workspace_bytes < 0) return EVO_ERR_INVALID_ARG;
    if (C == 0 || (!dX && !dWg && !dWu && !dWd)) return EVO_OK;  // nothing to write
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t es = elem_bytes(dtype);
    const bool empty = M == 0 || F == 0;
    if (!empty && (!X || !Wg || !Wu || !Wd || !dY || !workspace)) return EVO_ERR_INVALID_ARG;
    TrLayout L;
    if (!empty && !tr_layout(M, C, F, dtype, true, &L)) return EVO_ERR_UNSUPPORTED_SHAPE;
    const int64_t xb = M * C * es, wb = F * C * es;
    for (const void* p : {X, Wg, Wu, Wd, dY, static_cast<const void*>(dX), static_cast<const void*>(dWg),
                          static_cast<const void*>(dWu), static_cast<const void*>(dWd)})
        if (p && !aligned(p, tr_alignment(C, F, dtype))) return EVO_ERR_MISALIGNED;
    if (!empty) {
        if (workspace_bytes < L.total) return EVO_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return EVO_ERR_MISALIGNED;
    }
    if (any_overlap({{dX, xb, true}, {dWg, wb, true}, {dWu, wb, true}, {dWd, wb, true},
                     {workspace, empty ? 0 : L.total, true}, {X, xb, false}, {dY, xb, false}, {Wg, wb, false},
                     {Wu, wb, false}, {Wd, wb, false}}))
        return EVO_ERR_INVALID_ARG;
    RelaxedCapture relaxed;
    DeviceScope scope;
    if (empty) {  // empty sums
        if (xb == 0) dX = nullptr;
        if (wb == 0) dWg = dWu = dWd = nullptr;
        if (!dX && !dWg && !dWu && !dWd) return EVO_OK;
        const int dev = select_device({dX, dWg, dWu, dWd}, scope);
        if (dev < 0) return dev;
        return zero(dX, xb, st) && zero(dWg, wb, st) && zero(dWu, wb, st) && zero(dWd, wb, st) ? EVO_OK : EVO_ERR_CUDA;
    }
    const int dev = select_device({X, Wg, Wu, Wd, dY, dX, dWg, dWu, dWd, workspace}, scope);
    if (dev < 0) return dev;
    char* ws = static_cast<char*>(workspace);
    if (dtype == EVO_DTYPE_FP32) {
        auto f = [](const void* p) { return static_cast<const float*>(p); };
        auto o = [](void* p) { return static_cast<float*>(p); };
        auto run = act == EVO_ACT_SILU ? run_bwd_simt<EVO_ACT_SILU> : run_bwd_simt<EVO_ACT_GELU>;
        return run(L, f(X), f(Wg), f(Wu), f(Wd), f(dY), o(dX), o(dWg), o(dWu), o(dWd), ws, M, C, F, st);
    }
    auto run = dtype == EVO_DTYPE_FP16
                   ? (act == EVO_ACT_SILU ? run_bwd_mma<true, EVO_ACT_SILU> : run_bwd_mma<true, EVO_ACT_GELU>)
                   : (act == EVO_ACT_SILU ? run_bwd_mma<false, EVO_ACT_SILU> : run_bwd_mma<false, EVO_ACT_GELU>);
    return run(dev, X, Wg, Wu, Wd, dY, dX, dWg, dWu, dWd, ws, M, C, F, dtype, st);
}

// ------------------------------------------------- relative-position bias

namespace {

int check_relpos(int64_t B, int64_t Sq, int64_t Sk, int64_t H, int64_t nb, int dtype) {
    if (B < 0 || Sq < 0 || Sk < 0 || H < 0 || nb < 0) return EVO_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return EVO_ERR_UNSUPPORTED_DTYPE;
    if (nb > evo::kRelMaxBorders || B > 65535 || Sq > kIntMax / 4 || Sk > kIntMax / 4 || H > 65535)
        return EVO_ERR_UNSUPPORTED_SHAPE;
    int64_t n;
    if (!mul_ok(B * H, Sq, &n) || !mul_ok(n, Sk, &n) || n > INT64_MAX / 16) return EVO_ERR_UNSUPPORTED_SHAPE;
    return EVO_OK;
}

// Threads of a block along j, as a power of two: no more than the key columns need.
int rel_lane_cols(int64_t Sk, int cols, int most) {
    int l = 0;
    while (l < most && (int64_t(cols) << l) < Sk) ++l;
    return l;
}

struct RelTiles {
    int lane_cols, ti;
    int64_t jt, it, chunks;
    int64_t part_bytes;
};

// Backward blocks: a tile of query rows high enough that its rows outweigh
// clearing and adding up the block's bins, low enough that the blocks fill the SMs.
RelTiles rel_bwd_tiles(int64_t B, int64_t Sq, int64_t Sk, int64_t H, int64_t rows) {
    RelTiles t;
    t.lane_cols = rel_lane_cols(Sk, evo::kRelBwdCols, 7);
    const int64_t width = int64_t(evo::kRelBwdCols) << t.lane_cols;
    t.jt = (Sk + width - 1) / width;
    t.chunks = (rows + evo::kRelBins - 1) / evo::kRelBins;
    const int64_t per = evo::kRelBwdThreads >> t.lane_cols;  // query rows at once
    const int64_t others = std::max<int64_t>(1, B * H * t.jt * t.chunks);
    // one wave: a block's shared memory sets how many an SM holds (five by their registers)
    const int64_t held = std::min<int64_t>(5, (226 << 10) / (1024 + evo::rel_bwd_smem(int(std::min<int64_t>(rows, evo::kRelBins)), int(rows))));
    // at most kRelBwdRows rows a thread, which bounds the depth of its fp32 sums; where one
    // wave of blocks would have more, as few whole waves as keep to it (8192 x 8192 x 8
    // heads, us: 2 waves of 357 rows 386, 1.6 waves of 480 rows 502, one wave of 745 393)
    const int64_t most = evo::kRelBwdRows * per, wave = 148 * std::max<int64_t>(1, held);
    const int64_t waves = std::max<int64_t>(1, ((Sq + most - 1) / most * others + wave - 1) / wave);
    const int64_t want = std::max<int64_t>(1, wave * waves / others);
    int64_t ti = std::max<int64_t>((Sq + want - 1) / want, 8 * per);
    ti = std::min<int64_t>((ti + per - 1) / per * per, most);
    // element offsets inside a tile are 32-bit (Sk < 2^29, and below 1024 unless `per` is 1)
    t.ti = int(std::min<int64_t>(ti, kIntMax / Sk / per * per));
    t.it = (Sq + t.ti - 1) / t.ti;
    t.part_bytes = B * t.it * t.jt * H * rows * 4;
    return t;
}

template <typename T, int NW, bool VEC>
int launch_relpos_fwd(int dev, evo::RelParams<T> p, cudaStream_t st) {
    constexpr int heads = NW * 4 / int(sizeof(T)), cols = VEC ? 16 / int(sizeof(T)) : evo::kRelCols;
    p.groups = (p.H + heads - 1) / heads;
    p.lane_cols = rel_lane_cols(p.Sk, cols, 8);
    const int64_t width = int64_t(cols) << p.lane_cols, jt = (p.Sk + width - 1) / width;
    const int64_t per = evo::kRelThreads >> p.lane_cols;
    // about six blocks a SM: each fills its tables once for all its rows
    const int64_t others = jt * p.B * p.groups;
    int64_t ti = (p.Sq * others + 148 * 6 - 1) / (148 * 6);
    ti = std::max<int64_t>(ti, (int64_t(p.Sq) + 65534) / 65535);
    p.ti = int((ti + per - 1) / per * per);
    const int smem = evo::rel_smem((p.rows * NW * 4 + 15) / 16 * 16, p.nb);
    auto kernel = evo::evo_relpos_fwd_kernel<T, NW, VEC>;
    static AttrOnce attr;
    if (!attr.ensure(dev, kernel, evo::rel_smem((evo::kRelMaxBorders + 4) * NW * 4, evo::kRelMaxBorders))) return EVO_ERR_CUDA;
    // as many batches at once as the grid's z dimension takes with their groups of heads
    const int step = std::max(1, 65535 / p.groups), all = p.B;
    for (int b = 0; b < all; b += step) {
        p.B = std::min(step, all - b);
        if (!launch_dependent(kernel, dim3(unsigned(jt), blocks_of(p.Sq, p.ti), unsigned(p.B * p.groups)), evo::kRelThreads, smem, st, p))
            return EVO_ERR_CUDA;
        const int64_t pairs = int64_t(p.B) * p.H * p.Sq * p.Sk;
        p.pos_q += int64_t(p.B) * p.Sq;
        p.pos_k += int64_t(p.B) * p.Sk;
        if (p.chain_q) p.chain_q += int64_t(p.B) * p.Sq;
        if (p.chain_k) p.chain_k += int64_t(p.B) * p.Sk;
        if (p.base) p.base += pairs;
        p.pair += pairs;
    }
    return EVO_OK;
}

template <typename T>
int run_relpos_fwd(int dev, evo::RelParams<T> p, const void* table, const void* base, void* pair, cudaStream_t st) {
    p.table = static_cast<const T*>(table);
    p.base = static_cast<const T*>(base);
    p.pair = static_cast<T*>(pair);
    const bool vec = p.Sk % (16 / int(sizeof(T))) == 0 && aligned(pair, 16) && (!base || aligned(base, 16));
    // as many heads in a 16-, 8- or 4-byte table row as there are
    const int words = int((p.H * int64_t(sizeof(T)) + 3) / 4);
    if (words > 2) return vec ? launch_relpos_fwd<T, 4, true>(dev, p, st) : launch_relpos_fwd<T, 4, false>(dev, p, st);
    if (words > 1) return vec ? launch_relpos_fwd<T, 2, true>(dev, p, st) : launch_relpos_fwd<T, 2, false>(dev, p, st);
    return vec ? launch_relpos_fwd<T, 1, true>(dev, p, st) : launch_relpos_fwd<T, 1, false>(dev, p, st);
}

template <typename T>
int run_relpos_bwd(int dev, evo::RelParams<T> p, const void* dpair, void* dtable, void* ws, cudaStream_t st) {
    const RelTiles t = rel_bwd_tiles(p.B, p.Sq, p.Sk, p.H, p.rows);
    p.dpair = static_cast<const T*>(dpair);
    p.part = static_cast<float*>(ws);
    p.lane_cols = t.lane_cols;
    p.ti = t.ti;
    const bool vec = p.Sk % (16 / int(sizeof(T))) == 0 && aligned(dpair, 16);
    const bool chains = p.chain_q != nullptr;
    auto kernel = vec ? (chains ? evo::evo_relpos_bwd_kernel<T, true, true> : evo::evo_relpos_bwd_kernel<T, true, false>)
                      : (chains ? evo::evo_relpos_bwd_kernel<T, false, true> : evo::evo_relpos_bwd_kernel<T, false, false>);
    static AttrOnce attrs[4];
    if (!attrs[2 * vec + chains].ensure(dev, kernel, evo::rel_bwd_smem(evo::kRelBins, evo::kRelMaxBorders)))
        return EVO_ERR_CUDA;
    const int smem = evo::rel_bwd_smem(std::min(p.rows, evo::kRelBins), p.nb);
    p.jt = int(t.jt);
    p.it = int(t.it);
    const dim3 grid{unsigned(t.jt * t.it), unsigned(p.B * p.H * t.chunks)};
    // (not dependent itself: its one wave of blocks would be laid out around the
    // blocks of the kernel before; 1733 x 1733 x 16 heads: 101 instead of 69 us)
    return launch(kernel, grid, evo::kRelBwdThreads, smem, st, p) &&
                   launch_dependent(evo::evo_relpos_bwd_sum_kernel<T>, dim3(blocks_of(int64_t(p.H) * p.rows, 8)), 256, 0, st,
                                    (const float*)p.part, (long long)(p.B * t.it * t.jt), p.H, p.rows, static_cast<T*>(dtable))
               ? EVO_OK
               : EVO_ERR_CUDA;
}

template <typename T>
evo::RelParams<T> rel_params(const int32_t* borders, const int32_t* pos_q, const int32_t* pos_k, const int32_t* chain_q,
                             const int32_t* chain_k, int64_t B, int64_t Sq, int64_t Sk, int64_t H, int64_t nb) {
    evo::RelParams<T> p = {};
    p.borders = borders;
    p.pos_q = pos_q;
    p.pos_k = pos_k;
    p.chain_q = chain_q;
    p.chain_k = chain_k;
    p.B = int(B);
    p.Sq = int(Sq);
    p.Sk = int(Sk);
    p.H = int(H);
    p.nb = int(nb);
    p.rows = int(nb) + 1 + (chain_q != nullptr);
    return p;
}

}  // namespace

extern "C" EVO_API int evo_relpos_fwd(const void* table, const int32_t* borders, const int32_t* pos_q,
                                      const int32_t* pos_k, const int32_t* chain_q, const int32_t* chain_k,
                                      const void* base, void* pair, int64_t B, int64_t Sq, int64_t Sk, int64_t H,
                                      int64_t num_borders, int dtype, evo_stream_t stream) {
    const int chk = check_relpos(B, Sq, Sk, H, num_borders, dtype);
    if (chk != EVO_OK) return chk;
    if ((chain_q == nullptr) != (chain_k == nullptr)) return EVO_ERR_INVALID_ARG;
    if (B == 0 || Sq == 0 || Sk == 0 || H == 0) return EVO_OK;
    if (!table || (!borders && num_borders > 0) || !pos_q || !pos_k || !pair) return EVO_ERR_INVALID_ARG;
    const int64_t es = elem_bytes(dtype), pb = B * H * Sq * Sk * es;
    for (const void* p : {table, base, static_cast<const void*>(pair)})
        if (p && !aligned(p, uintptr_t(es))) return EVO_ERR_MISALIGNED;
    for (const int32_t* p : {borders, pos_q, pos_k, chain_q, chain_k})
        if (p && !aligned(p, 4)) return EVO_ERR_MISALIGNED;
    const int64_t rows = num_borders + 1 + (chain_q != nullptr);
    if (any_overlap({{pair, pb, true}, {table, rows * H * es, false}, {borders, num_borders * 4, false},
                     {pos_q, B * Sq * 4, false}, {pos_k, B * Sk * 4, false}, {chain_q, B * Sq * 4, false},
                     {chain_k, B * Sk * 4, false}, {base, pb, false}}))
        return EVO_ERR_INVALID_ARG;
    RelaxedCapture relaxed;
    DeviceScope scope;
    const int dev = select_device({pair, table, num_borders ? borders : nullptr, pos_q, pos_k, chain_q, chain_k, base}, scope);
    if (dev < 0) return dev;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
#define EVO_REL_FWD(T) \
    return run_relpos_fwd<T>(dev, rel_params<T>(borders, pos_q, pos_k, chain_q, chain_k, B, Sq, Sk, H, num_borders), table, base, pair, st)
    if (dtype == EVO_DTYPE_FP32) EVO_REL_FWD(float);
    if (dtype == EVO_DTYPE_FP16) EVO_REL_FWD(__half);
    EVO_REL_FWD(__nv_bfloat16);
#undef EVO_REL_FWD
}

extern "C" EVO_API int64_t evo_relpos_bwd_workspace_size(int64_t B, int64_t Sq, int64_t Sk, int64_t H, int64_t num_borders,
                                                         int has_chain) {
    const int chk = check_relpos(B, Sq, Sk, H, num_borders, EVO_DTYPE_BF16);
    if (chk != EVO_OK) return chk;
    if (B == 0 || Sq == 0 || Sk == 0 || H == 0) return 0;
    return rel_bwd_tiles(B, Sq, Sk, H, num_borders + 1 + (has_chain != 0)).part_bytes;
}

extern "C" EVO_API int evo_relpos_bwd(const void* dpair, const int32_t* borders, const int32_t* pos_q,
                                      const int32_t* pos_k, const int32_t* chain_q, const int32_t* chain_k, void* dtable,
                                      void* workspace, int64_t workspace_bytes, int64_t B, int64_t Sq, int64_t Sk,
                                      int64_t H, int64_t num_borders, int dtype, evo_stream_t stream) {
    const int chk = check_relpos(B, Sq, Sk, H, num_borders, dtype);
    if (chk != EVO_OK) return chk;
    if (workspace_bytes < 0 || (chain_q == nullptr) != (chain_k == nullptr)) return EVO_ERR_INVALID_ARG;
    if (H == 0) return EVO_OK;
    if (!dtable) return EVO_ERR_INVALID_ARG;
    const int64_t es = elem_bytes(dtype), pb = B * H * Sq * Sk * es;
    const int64_t rows = num_borders + 1 + (chain_q != nullptr), tb = rows * H * es;
    if (!aligned(dtable, uintptr_t(es))) return EVO_ERR_MISALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    RelaxedCapture relaxed;
    DeviceScope scope;
    if (pb == 0) {  // no pair: an empty sum
        const int dev = select_device({dtable}, scope);
        return dev < 0 ? dev : zero(dtable, tb, st) ? EVO_OK : EVO_ERR_CUDA;
    }
    if (!dpair || (!borders && num_borders > 0) || !pos_q || !pos_k || !workspace) return EVO_ERR_INVALID_ARG;
    const RelTiles t = rel_bwd_tiles(B, Sq, Sk, H, rows);
    // the grid's y and x dimensions
    if (B * H * t.chunks > 65535 || t.it * t.jt > kIntMax) return EVO_ERR_UNSUPPORTED_SHAPE;
    if (workspace_bytes < t.part_bytes) return EVO_ERR_INVALID_ARG;
    if (!aligned(dpair, uintptr_t(es)) || !aligned(workspace, 256)) return EVO_ERR_MISALIGNED;
    for (const int32_t* p : {borders, pos_q, pos_k, chain_q, chain_k})
        if (p && !aligned(p, 4)) return EVO_ERR_MISALIGNED;
    if (any_overlap({{dtable, tb, true}, {workspace, t.part_bytes, true}, {borders, num_borders * 4, false},
                     {pos_q, B * Sq * 4, false}, {pos_k, B * Sk * 4, false}, {chain_q, B * Sq * 4, false},
                     {chain_k, B * Sk * 4, false}, {dpair, pb, false}}))
        return EVO_ERR_INVALID_ARG;
    const int dev = select_device({dpair, dtable, workspace, num_borders ? borders : nullptr, pos_q, pos_k, chain_q, chain_k}, scope);
    if (dev < 0) return dev;
#define EVO_REL_BWD(T)                                                                                             \
    return run_relpos_bwd<T>(dev, rel_params<T>(borders, pos_q, pos_k, chain_q, chain_k, B, Sq, Sk, H, num_borders), \
                             dpair, dtable, workspace, st)
    if (dtype == EVO_DTYPE_FP32) EVO_REL_BWD(float);
    if (dtype == EVO_DTYPE_FP16) EVO_REL_BWD(__half);
    EVO_REL_BWD(__nv_bfloat16);
#undef EVO_REL_BWD
}
