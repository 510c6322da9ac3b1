// Host entry points of the operators around the product (include/tgemm_ops.h):
// argument checks, the choice of kernel and split, workspace layout, launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm_ops.h"
#include "tgemm_ops_kernels.h"
#include "tgemm_ops_small.h"
#include "tgemm_plan.h"

namespace tg {

int hip_failed(hipError_t e);               // tgemm.hip
int device_compute_units(int* ncu);

namespace {

constexpr int64_t kMaxDim = 2147483647;
constexpr int kFewRows = 32;                // rows of X that a workgroup of the few-rows kernels takes
constexpr int kFewMost = 1024;              // the most rows, in such blocks
constexpr int kMaxSplits = 64;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;   // of one launch along a grid's axis
constexpr int64_t kFewCols = int64_t(1) << 26;            // columns of one launch of the few-rows kernel
enum : int { kPathNone = 0, kPathFew, kPathTile, kPathGeneral, kPathEmpty };

int esize(int t) { return t == TGEMM_F32 ? 4 : 2; }
bool is16(int t) { return t == TGEMM_F16 || t == TGEMM_BF16; }
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Workgroups of the row and column joins, which take the rest in turn.
int64_t join_grid(int64_t n) { return n < (1 << 20) ? n : 1 << 20; }

// Row stride of the cross entropy's coefficients: whole 128-byte lines, an odd
// number of them, so that the rows a K step reads of one column range spread
// over the memory channels (weight gradient 128000 x 4096 x 8192: 6975 us with
// rows of 2000 lines, 6617 with 2003).
int64_t coef_stride(int64_t columns) { return (ceil_div(columns, 64) | 1) * 64; }

// A wave's offsets into an array of stride ld and n columns stay below 2^31
// (128 rows from its first).
bool fits31(int64_t ld, int64_t n, int es) { return (127 * ld + n) * es + 16 < (int64_t(1) << 31); }

// ---------------------------------------------------------------- arrays --
struct Mem {
    const void* p;
    uint64_t bytes;
};

// Checks one rows x cols array: stride, NULL, alignment, span.
bool array_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int es, Mem* m) {
    if (ld < (cols > 1 ? cols : 1)) return false;
    uint64_t n;
    if (!span_bytes(rows, cols, ld, &n, es)) return false;
    if (n && !p) return false;
    if ((uintptr_t)p % es) return false;
    *m = Mem{p, n};
    return true;
}

bool meet(const Mem& a, const Mem& b) { return overlaps(a.p, a.bytes, b.p, b.bytes); }

// Whether an output meets an input or another output.
bool outputs_meet(const Mem* in, int nin, const Mem* out, int nout) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (meet(out[i], in[j])) return true;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return true;
    }
    return false;
}

// ------------------------------------------------------------------ plan --
struct OpPlan {
    int path;
    int tile_m, k_step;
    int splits, kper;       // parts of the K axis, k of each
    int grid_m, grid_n, W;
    bool join;              // sums go to the workspace and the join kernel ends the product
    int64_t ws;             // workspace bytes
};

// K parts of kper (a multiple of 64), the last one not empty and, for kernels
// with 64-deep steps, holding more than 64 (they run at least two steps).
void fit_splits(int64_t K, int want, int k_step, int* splits, int* kper) {
    for (int s = want; s > 1; --s) {
        const int64_t per = up(ceil_div(K, s), 64);
        const int64_t n = ceil_div(K, per);
        if (per <= 64 || n < 2) continue;
        if (k_step == 64 && K - (n - 1) * per <= 64) continue;
        *splits = (int)n;
        *kper = (int)per;
        return;
    }
    *splits = 1;
    *kper = (int)K;
}

// Estimated time (us) of a tile choice: workgroups per compute unit in turn, or
// two at a time (32-deep steps of 128 and 64 rows), each its steps and a fixed
// part (first loads, end of tile), no faster than the operands' traffic, and the
// join's launch and traffic where the K axis is split. Per 32 k of a tile:
//   rows, K step      256, 64   128, 64   64, 64   128, 32   64, 32
//   B stored N x K     0.572     0.364    0.277     0.474     0.345
//   B stored K x N     0.675     0.431    0.274     0.441     0.298
//   A^T B              0.645     0.416    0.244     0.428     0.272
// The vector L1 serves a 128-byte line at a time whatever part of it is asked
// for: 64-deep steps of a K-contiguous operand take whole lines, 32-deep ones
// half (1024 x 4096 x 4096: 53.8 us with 32-deep steps, 39.7 with 64-deep);
// operands stored along the rows or columns take 512 bytes either way, and
// there two workgroups of 32-deep steps, which cover each other's fixed parts,
// stay ahead. Rows that start between 16-byte boundaries touch one line more
// (`late`). Fitted to 3300 timings of 124 random products and weight gradients
// (33 <= M <= 8192, N to 110000, K to 60000, 15 splits, graph launches): over
// that same set the choice takes 1.0% longer than the fastest on average, 32% at
// worst.
double tile_time(int64_t M, int64_t N, int64_t kper, int tile_m, int k_step, int layout, int splits, int ncu, bool join,
                 bool odd) {
    static const double cost[5][3] = {{0.572, 0.675, 0.645}, {0.364, 0.431, 0.416}, {0.277, 0.274, 0.244},
                                      {0.474, 0.441, 0.428}, {0.345, 0.298, 0.272}};
    static const double fixed[5] = {10.5, 8.75, 6.5, 8.1, 5.7}, late[5] = {1.23, 1.20, 1.36, 1.19, 1.27};
    const int v = tile_m == 256 ? 0 : (tile_m == 128 ? 1 : 2) + (k_step == 64 ? 0 : 2);
    const int64_t wgs = ceil_div(M, tile_m) * ceil_div(N, 256) * splits;
    const double steps = (double)ceil_div(kper, 32);
    const double walk = steps * cost[v][layout] * (odd ? late[v] : 1.0);
    double t;
    if (v < 3) {
        t = (double)ceil_div(wgs, ncu) * (walk + fixed[v]);
    } else {
        const double both = walk * (v == 3 ? 2.02 : 2.32);
        const int64_t full = wgs / (2 * ncu), left = wgs - full * 2 * ncu;
        t = (double)full * (both + 0.52 * fixed[v]);
        if (left > ncu)
            t += both + fixed[v];
        else if (left > 0)
            t += walk + fixed[v];
    }
    const double traffic = (double)wgs * steps * (tile_m + 256) * 64.0 / 13.0e6;
    t = t > traffic ? t : traffic;
    if (join) t += 6.7 + (double)splits * (double)M * (double)N * 8.0 / 6.0e6;
    return t;
}

// The same for the few-rows kernel over blocks of 32 rows of X: rounds of 512
// resident workgroups, each its pieces of 128 k (eight waves side by side), or
// what the vector L1s let through (40 bytes a nanosecond and compute unit: a block
// reads 32 rows of X for every 16 of the weight). Ahead where a product is small:
// 46 x 1984 x 968 6.5 us against 13.3 for tiles, 107 x 950 x 4296 13.0 against
// 23.0; behind from some 600 KB a compute unit on (74 x 5345 x 5996: 49.0
// against 27.8).
double few_time(int64_t M, int64_t N, int64_t K, int ncu, bool odd) {
    const int64_t wgs = ceil_div(M, kFewRows) * ceil_div(N, 16);
    const double own = (double)ceil_div(wgs, 2 * ncu) * (2.5 + 1.5 * (double)ceil_div(ceil_div(K, kFewK), 8));
    const double traffic = (double)wgs * 96.0 * (double)K / (double)ncu / 40.0e3;
    return 2.0 + (odd ? 1.35 : 1.0) * (own > traffic ? own : traffic);
}

// nxk / akm: layouts; direct: the tile kernel may end the product itself;
// one_part: no split; tile_m, k_step, splits: 0 or the caller's choice.
int plan_product(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int nxk, int akm, bool direct,
                 bool one_part, bool few_ok, int tile_m, int k_step, int splits, int ncu, OpPlan* pl) {
    *pl = OpPlan{};
    pl->splits = 1;
    pl->kper = (int)K;
    if (M == 0 || N == 0) {
        pl->path = kPathNone;
        return TGEMM_OK;
    }
    if (K == 0) {
        pl->path = kPathEmpty;
        pl->splits = 0;
        pl->join = true;
        return TGEMM_OK;
    }
    const bool few = few_ok && nxk && !akm && M <= kFewMost && lda <= kMaxDmaLd && ldb <= kMaxDmaLd;
    // (N bounds the row stride of the fp32 sums, which a product in one part that
    // its own end of tile finishes does not have)
    const bool tile = lda >= 8 && ldb >= 8 && lda <= kMaxDmaLd && ldb <= kMaxDmaLd &&
                      (N <= kMaxDmaLd || (direct && one_part));
    if ((tile_m == 16 && !few) || (tile_m > 16 && !tile)) return TGEMM_ERR_UNSUPPORTED;
    if (few && (tile_m == 16 || (tile_m == 0 && k_step == 0 && splits <= 1 && M <= kFewRows))) {
        if (splits > 1) return TGEMM_ERR_UNSUPPORTED;
        pl->path = kPathFew;
        return TGEMM_OK;
    }
    if (!tile || tile_m == 1) {
        if (splits > 1 || one_part) return TGEMM_ERR_UNSUPPORTED;
        pl->path = kPathGeneral;
        pl->join = true;
        pl->ws = M * N * 4;
        return TGEMM_OK;
    }
    pl->path = kPathTile;
    double best = 0;
    static const int choices[5][2] = {{256, 64}, {128, 64}, {64, 64}, {128, 32}, {64, 32}};
    for (const auto& ch : choices) {
        const int tm = ch[0], ks = ch[1];
        if ((tile_m && tm != tile_m) || (k_step && ks != k_step)) continue;
        if (ks == 64 && K <= 64) continue;                    // 64-deep steps come in twos at least
        for (int s = 1; s <= kMaxSplits; ++s) {
            if (splits && s != splits) continue;
            if (one_part && s > 1) break;
            if (!splits && s > 1 && K / s < 256) break;
            int sp, per;
            fit_splits(K, s, ks, &sp, &per);
            if (!splits && sp != s && s > 1) continue;
            const bool join = sp > 1 || !direct;
            if (ceil_div(M, tm) * ceil_div(N, 256) * sp * NTHREADS > kMaxThreads) continue;
            const double t = tile_time(M, N, per, tm, ks, akm ? 2 : (nxk ? 0 : 1), sp, ncu, join,
                                       lda % 8 != 0 || ldb % 8 != 0);
            if (best == 0 || t < best) {
                best = t;
                pl->tile_m = tm;
                pl->k_step = ks;
                pl->splits = sp;
                pl->kper = per;
                pl->join = join;
            }
        }
    }
    if (best == 0) {
        // (no choice, or, past a billion rows, no grid that one launch takes)
        if (tile_m || k_step || splits > 1 || one_part) return TGEMM_ERR_UNSUPPORTED;
        return plan_product(M, N, K, lda, ldb, nxk, akm, direct, one_part, few_ok, 1, 0, 0, ncu, pl);
    }
    if (few && !tile_m && !k_step && splits <= 1 && few_time(M, N, K, ncu, lda % 8 != 0 || ldb % 8 != 0) < best) {
        *pl = OpPlan{};
        pl->splits = 1;
        pl->kper = (int)K;
        pl->path = kPathFew;
        return TGEMM_OK;
    }
    const int64_t gm = ceil_div(M, pl->tile_m), gn = ceil_div(N, 256);
    if (gm * gn * pl->splits > kMaxDim) return TGEMM_ERR_UNSUPPORTED;
    pl->grid_m = (int)gm;
    pl->grid_n = (int)gn;
    pl->W = (int)(gm * gn);
    pl->ws = pl->join ? (int64_t)pl->splits * M * N * 4 : 0;
    return TGEMM_OK;
}

// ---------------------------------------------------------------- launch --
int launch_k(const void* fn, int64_t gx, int64_t gy, int threads, void** args, void* stream) {
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)gx, (unsigned)gy), dim3((unsigned)threads), args, 0,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? TGEMM_OK : hip_failed(e);
}

const void* tile_kernel(int ab, int end, int act, int nxk, int akm, const OpPlan& pl) {
#define TG_OP(e, ac) \
    if (end == e && act == ac) return ab ? op_kernel<1, e, ac>(nxk, akm, pl.tile_m, pl.k_step) \
                                         : op_kernel<0, e, ac>(nxk, akm, pl.tile_m, pl.k_step);
    TG_OP(kEndLin16, kActNone)
    TG_OP(kEndLin16, kActRelu)
    TG_OP(kEndLin16, kActSilu)
    TG_OP(kEndLin16, kActGelu)
    TG_OP(kEndLin16, kActGeluTanh)
    TG_OP(kEndLin32, kActNone)
    TG_OP(kEndLin32, kActRelu)
    TG_OP(kEndLin32, kActSilu)
    TG_OP(kEndLin32, kActGelu)
    TG_OP(kEndLin32, kActGeluTanh)
    TG_OP(kEndAcc32, kActNone)
    TG_OP(kEndXentFwd, kActNone)
    TG_OP(kEndXentBwd, kActNone)
    if (end == kEndXentExp && ab) return op_kernel<1, kEndXentExp, kActNone>(nxk, akm, pl.tile_m, pl.k_step);
#undef TG_OP
    return nullptr;
}

// The tile kernel of a plan (a.A .. a.C, sizes and strides set by the caller).
int launch_tile(OpArgs& a, int ab, int end, int act, int nxk, int akm, const OpPlan& pl, int ncu, void* stream) {
    const void* fn = tile_kernel(ab, end, act, nxk, akm, pl);
    if (!fn) return TGEMM_ERR_UNSUPPORTED;
    a.grid_m = pl.grid_m;
    a.grid_n = pl.grid_n;
    a.W = pl.W;
    // tile rows of a raster group: a die's 32 tiles side by side then read 4 x 8
    // panels of 256 rows and columns, or 8 x 4 of 128 (64) rows and 256 columns
    // (700 x 9000 x 5000, 128-row tiles: 75.8 us with four, 69.7 with eight)
    const int group = pl.tile_m == 256 ? kDefaultGroupM : 2 * kDefaultGroupM;
    a.group_m = group < pl.grid_m ? group : pl.grid_m;
    a.num_xcd = num_xcd_for(ncu);
    a.splits = pl.splits;
    a.kper = pl.kper;
    // 64-deep steps: one workgroup per compute unit walks several tiles (a
    // workgroup needs two steps per tile for its load stream)
    const bool walk = pl.splits == 1 && pl.tile_m == 256 && pl.k_step == 64 && a.K >= 128 && pl.W > ncu;
    a.grid = walk ? ncu : pl.W;
    const int es = end == kEndAcc32 || end == kEndLin32 ? 4 : 2;
    a.c16 = 1;
    a.c8 = 0;
    a.c_stream = end != kEndAcc32 && (uintptr_t)a.C % 128 == 0 && (a.ldc * es) % 128 == 0;
    // exponentials are read again at once: streamed only past twice the Infinity
    // Cache (8192 x 128000 x 4096: 19310 -> 19075 us; 4096 x 32768 x 2048: 1373 -> 1392)
    if (end == kEndXentExp) a.c_stream = a.c_stream && (int64_t)a.M * a.ldc * es > (int64_t(512) << 20);
    void* kargs[] = {&a};
    return launch_k(fn, (int64_t)a.grid * pl.splits, 1, NTHREADS, kargs, stream);
}

int launch_join(OpArgs& a, int ab, const float* sums, int splits, bool c32, bool rf32, void* stream) {
    a.splits = splits;
    int c = c32, rf = rf32;
    void* kargs[] = {&a, &sums, &c, &rf};
    const int64_t quads = ceil_div(a.N, 4) * a.M;
    const int64_t blocks = ceil_div(quads, 256);
    return launch_k(ab ? (const void*)&tgemm_join_kernel<1> : (const void*)&tgemm_join_kernel<0>,
                    blocks < 16384 ? blocks : 16384, 1, 256, kargs, stream);
}

// Rows of A up to which the few-rows kernels load it in the operand's layout.
constexpr int kFewPlain = 4;

template <int AB, int KW>
const void* few_kernel(int64_t M) {
    return M <= kFewPlain ? (const void*)&tgemm_few_kernel<AB, 1, 0, KW>
           : M <= 16      ? (const void*)&tgemm_few_kernel<AB, 1, 1, KW>
                          : (const void*)&tgemm_few_kernel<AB, 2, 1, KW>;
}

template <int AB>
const void* xent_few_kernel(int64_t R) {
    return R <= kFewPlain ? (const void*)&tgemm_xent_few_kernel<AB, 1, 0>
           : R <= 16      ? (const void*)&tgemm_xent_few_kernel<AB, 1, 1>
                          : (const void*)&tgemm_xent_few_kernel<AB, 2, 1>;
}

OpArgs op_args() {
    OpArgs a{};
    a.alpha = 1.0f;
    a.splits = 1;
    return a;
}

// ---------------------------------------------------------------- linear --
// The product of a plan with the linear epilogue. `a` holds operands, C,
// epilogue and strides; ws the plan's workspace.
int run_linear(OpArgs& a, int ab, int nxk, bool c32, int type, const OpPlan& pl, int ncu, void* ws, void* stream) {
    if (pl.path == kPathNone) return TGEMM_OK;
    if (pl.path == kPathFew) {
        // waves along K: eight, or four where there are few pieces of 128 (1 x
        // 12288 x 512: 5.4 us with four, 6.4 with eight; 1 x 8192 x 4096: 16.6
        // and 14.6)
        const bool four = a.K <= 4 * kFewK;
        int c = c32;
        const void* fn = four ? (ab ? few_kernel<1, 4>(a.M) : few_kernel<0, 4>(a.M))
                              : (ab ? few_kernel<1, 8>(a.M) : few_kernel<0, 8>(a.M));
        const int64_t N = a.N;
        const OpArgs all = a;
        for (int64_t n0 = 0; n0 < N; n0 += kFewCols) {
            auto at = [n0](const void* p, int es) { return p ? static_cast<const char*>(p) + n0 * es : nullptr; };
            OpArgs q = all;
            q.N = (int)(N - n0 < kFewCols ? N - n0 : kFewCols);
            q.B = all.B + n0 * all.ldb;
            q.C = const_cast<char*>(at(all.C, c32 ? 4 : 2));
            q.biasv = at(all.biasv, all.bias_f32 ? 4 : 2);
            q.res = at(all.res, 2);
            q.pre = const_cast<char*>(at(all.pre, 2));
            void* kargs[] = {&q, &c};
            const int rc = launch_k(fn, ceil_div(q.N, 16), a.M <= 16 ? 1 : ceil_div(a.M, kFewRows), four ? 256 : 512, kargs,
                                    stream);
            if (rc != TGEMM_OK) return rc;
        }
        return TGEMM_OK;
    }
    float* sums = static_cast<float*>(ws);
    if (pl.path == kPathTile && !pl.join) return launch_tile(a, ab, c32 ? kEndLin32 : kEndLin16, a.act, nxk, 0, pl, ncu, stream);
    if (pl.path == kPathTile) {
        OpArgs p = op_args();
        p.A = a.A;
        p.B = a.B;
        p.lda = a.lda;
        p.ldb = a.ldb;
        p.M = a.M;
        p.N = a.N;
        p.K = a.K;
        p.C = sums;
        p.ldc = a.N;
        const int rc = launch_tile(p, ab, kEndAcc32, kActNone, nxk, 0, pl, ncu, stream);
        if (rc != TGEMM_OK) return rc;
    } else if (pl.path == kPathGeneral) {
        const int rc = tgemm_gemm(a.M, a.N, a.K, type, a.A, a.lda, a.B, a.ldb, nxk ? TGEMM_B_NxK : TGEMM_B_KxN, TGEMM_F32,
                                  sums, a.N, 1.0f, nullptr, TGEMM_ACT_NONE, stream);
        if (rc != TGEMM_OK) return rc;
    }
    return launch_join(a, ab, sums, pl.path == kPathEmpty ? 0 : pl.splits, c32, false, stream);
}

int check_dims(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim ? TGEMM_ERR_INVALID : TGEMM_OK;
}

// Whether an output of M x N has a workspace that 63 bits count (64 parts of fp32
// sums; no memory holds an output anywhere near the bound).
bool countable(int64_t M, int64_t N) { return N == 0 || M <= (int64_t(1) << 54) / N; }

// The plan of a linear layer. What the tile kernel cannot end itself (offsets
// past 31 bits, fewer than 8 columns) goes through the join.
int plan_linear(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw, int w_layout, int y_type,
                int64_t ldy, int tile_m, int k_step, int splits, int* ncu, OpPlan* pl) {
    if (check_dims(M, N, K) != TGEMM_OK || !is16(type) || (y_type != type && y_type != TGEMM_F32)) return TGEMM_ERR_INVALID;
    if (w_layout != TGEMM_B_KxN && w_layout != TGEMM_B_NxK) return TGEMM_ERR_INVALID;
    if (tile_m != 0 && tile_m != 1 && tile_m != 16 && tile_m != 64 && tile_m != 128 && tile_m != 256) return TGEMM_ERR_INVALID;
    if ((k_step != 0 && k_step != 32 && k_step != 64) || splits < 0 || splits > kMaxSplits) return TGEMM_ERR_INVALID;
    const int64_t wmin = w_layout == TGEMM_B_NxK ? K : N;
    if (ldx < (K > 1 ? K : 1) || ldw < (wmin > 1 ? wmin : 1) || ldy < (N > 1 ? N : 1)) return TGEMM_ERR_INVALID;
    if (!countable(M, N)) return TGEMM_ERR_UNSUPPORTED;
    const bool direct = N >= 8 && fits31(ldy, N, esize(y_type));
    *ncu = 256;
    if (M > 0 && N > 0 && K > 0) {
        const int rc = device_compute_units(ncu);
        if (rc != TGEMM_OK) return rc;
    }
    return plan_product(M, N, K, ldx, ldw, w_layout == TGEMM_B_NxK, 0, direct, false, true, tile_m, k_step, splits, *ncu, pl);
}

// ------------------------------------------------------------ transposed --
int plan_tn(int64_t M, int64_t N, int64_t K, int type, int64_t lda, int64_t ldb, int c_type, int64_t ldc, int tile_m,
            int k_step, int splits, int* ncu, OpPlan* pl) {
    if (tile_m != 0 && tile_m != 64 && tile_m != 128 && tile_m != 256) return TGEMM_ERR_INVALID;
    if (check_dims(M, N, K) != TGEMM_OK || !is16(type) || (c_type != type && c_type != TGEMM_F32)) return TGEMM_ERR_INVALID;
    if ((k_step != 0 && k_step != 32 && k_step != 64) || splits < 0 || splits > kMaxSplits) return TGEMM_ERR_INVALID;
    if (lda < (M > 1 ? M : 1) || ldb < (N > 1 ? N : 1) || ldc < (N > 1 ? N : 1)) return TGEMM_ERR_INVALID;
    if (!countable(M, N)) return TGEMM_ERR_UNSUPPORTED;
    const bool direct = N >= 8 && fits31(ldc, N, esize(c_type));
    *ncu = 256;
    if (M > 0 && N > 0 && K > 0) {
        const int rc = device_compute_units(ncu);
        if (rc != TGEMM_OK) return rc;
    }
    return plan_product(M, N, K, lda, ldb, 0, 1, direct, false, false, tile_m, k_step, splits, *ncu, pl);
}

// C = alpha A^T B + residual (a.res: C itself, or null).
int run_tn(OpArgs& a, int ab, bool c32, const OpPlan& pl, int ncu, void* ws, void* stream) {
    if (pl.path == kPathNone) return TGEMM_OK;
    float* sums = static_cast<float*>(ws);
    if (pl.path == kPathTile && !pl.join)
        return launch_tile(a, ab, c32 ? kEndAcc32 : kEndLin16, kActNone, 0, 1, pl, ncu, stream);
    if (pl.path == kPathTile) {
        OpArgs p = op_args();
        p.A = a.A;
        p.B = a.B;
        p.lda = a.lda;
        p.ldb = a.ldb;
        p.M = a.M;
        p.N = a.N;
        p.K = a.K;
        p.C = sums;
        p.ldc = a.N;
        const int rc = launch_tile(p, ab, kEndAcc32, kActNone, 0, 1, pl, ncu, stream);
        if (rc != TGEMM_OK) return rc;
    } else if (pl.path == kPathGeneral) {
        void* kargs[] = {&a, &sums};
        const int64_t blocks = ceil_div(a.N, 32) * a.M;
        const int rc = launch_k(ab ? (const void*)&tgemm_tn_narrow_kernel<1> : (const void*)&tgemm_tn_narrow_kernel<0>,
                                blocks < 65536 ? blocks : 65536, 1, 256, kargs, stream);
        if (rc != TGEMM_OK) return rc;
    }
    return launch_join(a, ab, sums, pl.path == kPathEmpty ? 0 : pl.splits, c32, c32, stream);
}

// --------------------------------------------------------- cross entropy --
struct XentPlan {
    bool few;
    OpPlan tile;
    int waves;              // parts of the few-rows kernel
    int64_t parts, ws;
};

int plan_xent(int64_t R, int64_t V, int64_t D, int type, int64_t ldh, int64_t ldw, int* ncu, XentPlan* x) {
    if (check_dims(R, V, D) != TGEMM_OK || !is16(type) || D < 8 || V < 1 || V > kMaxDim / 4) return TGEMM_ERR_INVALID;
    if (ldh < D || ldw < D) return TGEMM_ERR_INVALID;
    if (ldh > kMaxDmaLd || ldw > kMaxDmaLd) return TGEMM_ERR_UNSUPPORTED;
    int rc = device_compute_units(ncu);
    if (rc != TGEMM_OK) return rc;
    *x = XentPlan{};
    x->few = R <= kFewRows;
    if (x->few) {
        // eight waves per compute unit, each an equal number of 16-column groups
        const int64_t groups = ceil_div(V, 16);
        x->waves = (int)ceil_div(groups, ceil_div(groups, (int64_t)*ncu * 8));
        x->parts = x->waves;
    } else {
        rc = plan_product(R, V, D, ldh, ldw, 1, 0, true, true, false, 0, 0, 0, *ncu, &x->tile);
        if (rc != TGEMM_OK) return rc;
        x->parts = ceil_div(V, 128);
    }
    x->ws = up(x->parts * R * 8, 16) + up(R * 4, 16);
    return TGEMM_OK;
}

// lse and losses from the parts (a.part, a.zt), then their sum or mean; recs and
// scale: null, or the row records and the scale of the total's gradient.
int xent_finish(const OpArgs& a, int64_t nparts, int64_t vocab, int64_t ignore, int reduction, float* lse, float* loss,
                float* total, float* count, XentRow* recs, float* scale, void* stream) {
    const float2* part = a.part;
    const float* zt = a.zt;
    const int64_t* target = a.target;
    int parts = (int)nparts, r = a.M;
    {
        void* kargs[] = {&part, &parts, &r, &zt, &target, &vocab, &ignore, &lse, &loss, &recs};
        const bool wide = r >= 512;
        const int rc = launch_k(wide ? (const void*)&tgemm_xent_join_kernel<16> : (const void*)&tgemm_xent_join_kernel<2>,
                                join_grid(ceil_div(r, wide ? 16 : 2)), 1, 256, kargs, stream);
        if (rc != TGEMM_OK || reduction == TGEMM_REDUCE_NONE) return rc;
    }
    int mean = reduction == TGEMM_REDUCE_MEAN;
    const float* closs = loss;
    void* kargs[] = {&closs, &target, &ignore, &r, &mean, &total, &count, &scale};
    return launch_k((const void*)&tgemm_xent_reduce_kernel, 1, 1, 1024, kargs, stream);
}

// Loss and gradients in one call: the exponentials of all rows and columns stay
// in the workspace, at most kExpElems of them (2 GiB).
constexpr int64_t kExpElems = int64_t(1) << 30;

struct XentBothPlan {
    OpPlan fwd, dh, dw;
    int64_t parts, ldg;
    int64_t off_zt, off_recs, off_scale, off_g, off_area, ws;
};

int plan_xent_both(int64_t R, int64_t V, int64_t D, int type, int64_t ldh, int64_t ldw, int64_t lddh, int64_t lddw,
                   int* ncu, XentBothPlan* x) {
    if (check_dims(R, V, D) != TGEMM_OK || !is16(type) || D < 8 || V < 1 || V > kMaxDim / 4 || R < 1) return TGEMM_ERR_INVALID;
    if (ldh < D || ldw < D || lddh < D || lddw < D) return TGEMM_ERR_INVALID;
    if (ldh > kMaxDmaLd || ldw > kMaxDmaLd || lddh > kMaxDmaLd || lddw > kMaxDmaLd) return TGEMM_ERR_UNSUPPORTED;
    *x = XentBothPlan{};
    x->ldg = coef_stride(V);
    if (type != TGEMM_BF16 || x->ldg > kMaxDmaLd || R * x->ldg > kExpElems) return TGEMM_ERR_UNSUPPORTED;
    int rc = device_compute_units(ncu);
    if (rc == TGEMM_OK) rc = plan_product(R, V, D, ldh, ldw, 1, 0, true, true, false, 0, 0, 0, *ncu, &x->fwd);
    if (rc == TGEMM_OK) rc = plan_product(R, D, V, x->ldg, ldw, 0, 0, true, false, false, 0, 0, 0, *ncu, &x->dh);
    if (rc == TGEMM_OK) rc = plan_product(V, D, R, x->ldg, ldh, 0, 1, true, false, false, 0, 0, 0, *ncu, &x->dw);
    if (rc != TGEMM_OK) return rc;
    x->parts = ceil_div(V, 128);
    x->off_zt = up(x->parts * R * 8, 256);
    x->off_recs = x->off_zt + up(R * 4, 256);
    x->off_scale = x->off_recs + up(R * (int64_t)sizeof(XentRow), 256);
    x->off_g = x->off_scale + 256;
    x->off_area = x->off_g + up(R * x->ldg * 2, 256);
    x->ws = x->off_area + (x->dh.ws > x->dw.ws ? x->dh.ws : x->dw.ws);
    return TGEMM_OK;
}

// The gradient walks the vocabulary in pieces whose coefficients (R x piece, 16
// bits) stay at or below kPieceElems.
constexpr int64_t kPieceElems = int64_t(1) << 28;

struct XentGradPlan {
    int64_t piece, pieces, ldg;
    OpPlan dh;              // full piece
    bool dh_sums;           // dH through fp32 sums and a join
    int64_t dw_ws;
    int64_t off_scale, off_g, off_sums, off_dw, ws;
};

int plan_xent_grad(int64_t R, int64_t V, int64_t D, int type, int64_t ldh, int64_t ldw, int64_t lddh, int64_t lddw,
                   int* ncu, XentGradPlan* x) {
    if (check_dims(R, V, D) != TGEMM_OK || !is16(type) || D < 8 || V < 1 || V > kMaxDim / 4) return TGEMM_ERR_INVALID;
    if (ldh < D || ldw < D || lddh < D || lddw < D) return TGEMM_ERR_INVALID;
    if (ldh > kMaxDmaLd || ldw > kMaxDmaLd || lddh > kMaxDmaLd || lddw > kMaxDmaLd) return TGEMM_ERR_UNSUPPORTED;
    int rc = device_compute_units(ncu);
    if (rc != TGEMM_OK) return rc;
    *x = XentGradPlan{};
    const int64_t rows = R > 0 ? R : 1;
    int64_t most = kPieceElems / rows / 256 * 256;
    // the coefficients' row stride is bounded like any operand's
    most = most < 256 ? 256 : (most > 2 * 1000 * 1000 ? 2 * 1000 * 1000 : most);
    x->pieces = ceil_div(V, most);
    x->piece = up(ceil_div(V, x->pieces), 256);
    x->pieces = ceil_div(V, x->piece);
    if (x->piece > V) x->piece = V;
    x->ldg = coef_stride(x->piece);
    rc = plan_product(rows, D, x->piece, x->ldg, ldw, 0, 0, x->pieces == 1, false, false, 0, 0, 0, *ncu, &x->dh);
    if (rc != TGEMM_OK) return rc;
    x->dh_sums = x->dh.join;
    OpPlan dw;
    for (int last = 0; last < 2; ++last) {
        const int64_t n = last ? V - (x->pieces - 1) * x->piece : x->piece;
        rc = plan_product(n, D, rows, x->ldg, ldh, 0, 1, true, false, false, 0, 0, 0, *ncu, &dw);
        if (rc != TGEMM_OK) return rc;
        if (dw.ws > x->dw_ws) x->dw_ws = dw.ws;
    }
    x->off_scale = up(rows * (int64_t)sizeof(XentRow), 256);
    x->off_g = x->off_scale + 256;
    x->off_sums = x->off_g + up(rows * x->ldg * 2, 256);
    x->off_dw = x->off_sums + (x->dh_sums ? up((int64_t)x->dh.splits * rows * D * 4, 256) : 0);
    x->ws = x->off_dw + x->dw_ws;
    return TGEMM_OK;
}

// Rows of a column-sum block: 128, halved (to 16 at least) while there are fewer
// than 512 workgroups of 256 columns, doubled while the blocks exceed a grid's
// 65535 in y.
int col_rows(int64_t M, int64_t N) {
    int r = 128;
    while (r > 16 && ceil_div(M, r) * ceil_div(N, 256) < 512) r /= 2;
    while (ceil_div(M, r) > 65535) r *= 2;
    return r;
}

bool ws_ok(const void* ws, int64_t have, int64_t need) {
    return need == 0 || (ws && have >= need && (uintptr_t)ws % 16 == 0);
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int64_t tgemm_linear_config_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw,
                                                 int w_layout, int y_type, int64_t ldy, int tile_m, int k_step,
                                                 int splits) {
    OpPlan pl;
    int ncu;
    const int rc = plan_linear(M, N, K, type, ldx, ldw, w_layout, y_type, ldy, tile_m, k_step, splits, &ncu, &pl);
    return rc != TGEMM_OK ? rc : pl.ws;
}

extern "C" int64_t tgemm_linear_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw,
                                          int w_layout, int y_type, int64_t ldy) {
    return tgemm_linear_config_workspace(M, N, K, type, ldx, ldw, w_layout, y_type, ldy, 0, 0, 0);
}

namespace tg {
namespace {

// tgemm_linear_config; alpha_dev: null, or one device value alpha is multiplied by.
int linear_call(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W, int64_t ldw,
                int w_layout, const void* bias, int bias_type, int act, const void* residual, int64_t ldr, int y_type,
                void* Y, int64_t ldy, void* pre, int64_t ldpre, float alpha, const float* alpha_dev, void* workspace,
                int64_t workspace_bytes, void* stream, int tile_m, int k_step, int splits) {
    if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_INVALID;
    if (check_dims(M, N, K) != TGEMM_OK || !is16(type) || (y_type != type && y_type != TGEMM_F32)) return TGEMM_ERR_INVALID;
    if (w_layout != TGEMM_B_KxN && w_layout != TGEMM_B_NxK) return TGEMM_ERR_INVALID;
    if (bias && bias_type != type && bias_type != TGEMM_F32) return TGEMM_ERR_INVALID;
    Mem mx, mw, my, mr{}, mp{}, mb{};
    const bool nxk = w_layout == TGEMM_B_NxK;
    if (!array_ok(X, M, K, ldx, 2, &mx) || !array_ok(W, nxk ? N : K, nxk ? K : N, ldw, 2, &mw) ||
        !array_ok(Y, M, N, ldy, esize(y_type), &my))
        return TGEMM_ERR_INVALID;
    if (residual && !array_ok(residual, M, N, ldr, 2, &mr)) return TGEMM_ERR_INVALID;
    if (pre && !array_ok(pre, M, N, ldpre, 2, &mp)) return TGEMM_ERR_INVALID;
    if (bias && !array_ok(bias, 1, N, N > 1 ? N : 1, esize(bias_type), &mb)) return TGEMM_ERR_INVALID;
    const bool in_place = residual == Y && ldr == ldy && y_type == type;
    if (meet(my, mx) || meet(my, mw) || meet(my, mb) || meet(my, mp) || (!in_place && meet(my, mr))) return TGEMM_ERR_INVALID;
    if (meet(mp, mx) || meet(mp, mw) || meet(mp, mb) || meet(mp, mr)) return TGEMM_ERR_INVALID;
    OpPlan pl;
    int ncu;
    // (longer rows than that never run on tiles, whose offsets the limit is for)
    if (N <= kMaxDmaLd && ((residual && ldr > kMaxDmaLd) || (pre && ldpre > kMaxDmaLd))) return TGEMM_ERR_UNSUPPORTED;
    int rc = plan_linear(M, N, K, type, ldx, ldw, w_layout, y_type, ldy, tile_m, k_step, splits, &ncu, &pl);
    if (rc != TGEMM_OK) return rc;
    if (!ws_ok(workspace, workspace_bytes, pl.ws)) return TGEMM_ERR_INVALID;
    const Mem mws{workspace, (uint64_t)pl.ws};
    if (meet(mws, mx) || meet(mws, mw) || meet(mws, mb) || meet(mws, mp) || meet(mws, mr) || meet(mws, my))
        return TGEMM_ERR_INVALID;
    OpArgs a = op_args();
    a.A = static_cast<const uint16_t*>(X);
    a.B = static_cast<const uint16_t*>(W);
    a.C = Y;
    a.lda = ldx;
    a.ldb = ldw;
    a.ldc = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.alpha = alpha;
    a.alpha_dev = alpha_dev;
    a.biasv = bias;
    a.bias_f32 = bias_type == TGEMM_F32;
    a.act = act;
    a.pre = pre;
    a.ldpre = pre ? ldpre : 0;
    a.res = residual;
    a.ldres = residual ? ldr : 0;
    return run_linear(a, type == TGEMM_BF16, nxk, y_type == TGEMM_F32, type, pl, ncu, workspace, stream);
}

}  // namespace
}  // namespace tg

extern "C" int tgemm_linear_config(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W,
                                   int64_t ldw, int w_layout, const void* bias, int bias_type, int act,
                                   const void* residual, int64_t ldr, int y_type, void* Y, int64_t ldy, void* pre,
                                   int64_t ldpre, float alpha, void* workspace, int64_t workspace_bytes, void* stream,
                                   int tile_m, int k_step, int splits) {
    return linear_call(M, N, K, type, X, ldx, W, ldw, w_layout, bias, bias_type, act, residual, ldr, y_type, Y, ldy, pre,
                       ldpre, alpha, nullptr, workspace, workspace_bytes, stream, tile_m, k_step, splits);
}

extern "C" int tgemm_linear(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W,
                            int64_t ldw, int w_layout, const void* bias, int bias_type, int act, const void* residual,
                            int64_t ldr, int y_type, void* Y, int64_t ldy, void* pre, int64_t ldpre, float alpha,
                            void* workspace, int64_t workspace_bytes, void* stream) {
    return tgemm_linear_config(M, N, K, type, X, ldx, W, ldw, w_layout, bias, bias_type, act, residual, ldr, y_type, Y,
                               ldy, pre, ldpre, alpha, workspace, workspace_bytes, stream, 0, 0, 0);
}

extern "C" int64_t tgemm_tn_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t lda, int64_t ldb, int c_type,
                                      int64_t ldc, int tile_m, int k_step, int splits) {
    OpPlan pl;
    int ncu;
    const int rc = plan_tn(M, N, K, type, lda, ldb, c_type, ldc, tile_m, k_step, splits, &ncu, &pl);
    return rc != TGEMM_OK ? rc : pl.ws;
}

namespace tg {
namespace {

// tgemm_tn; alpha_dev as in linear_call.
int tn_call(int64_t M, int64_t N, int64_t K, int type, const void* A, int64_t lda, const void* B, int64_t ldb, int c_type,
            void* C, int64_t ldc, float alpha, const float* alpha_dev, int accumulate, void* workspace,
            int64_t workspace_bytes, void* stream, int tile_m, int k_step, int splits) {
    if (accumulate != 0 && accumulate != 1) return TGEMM_ERR_INVALID;
    if (check_dims(M, N, K) != TGEMM_OK || !is16(type) || (c_type != type && c_type != TGEMM_F32)) return TGEMM_ERR_INVALID;
    Mem ma, mb, mc;
    if (!array_ok(A, K, M, lda, 2, &ma) || !array_ok(B, K, N, ldb, 2, &mb) || !array_ok(C, M, N, ldc, esize(c_type), &mc))
        return TGEMM_ERR_INVALID;
    if (meet(mc, ma) || meet(mc, mb)) return TGEMM_ERR_INVALID;
    OpPlan pl;
    int ncu;
    const int rc = plan_tn(M, N, K, type, lda, ldb, c_type, ldc, tile_m, k_step, splits, &ncu, &pl);
    if (rc != TGEMM_OK) return rc;
    if (!ws_ok(workspace, workspace_bytes, pl.ws)) return TGEMM_ERR_INVALID;
    const Mem mws{workspace, (uint64_t)pl.ws};
    if (meet(mws, ma) || meet(mws, mb) || meet(mws, mc)) return TGEMM_ERR_INVALID;
    OpArgs a = op_args();
    a.A = static_cast<const uint16_t*>(A);
    a.B = static_cast<const uint16_t*>(B);
    a.C = C;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.alpha = alpha;
    a.alpha_dev = alpha_dev;
    a.res = accumulate ? C : nullptr;
    a.ldres = accumulate ? ldc : 0;
    return run_tn(a, type == TGEMM_BF16, c_type == TGEMM_F32, pl, ncu, workspace, stream);
}

}  // namespace
}  // namespace tg

extern "C" int tgemm_tn(int64_t M, int64_t N, int64_t K, int type, const void* A, int64_t lda, const void* B, int64_t ldb,
                        int c_type, void* C, int64_t ldc, float alpha, int accumulate, void* workspace,
                        int64_t workspace_bytes, void* stream, int tile_m, int k_step, int splits) {
    return tn_call(M, N, K, type, A, lda, B, ldb, c_type, C, ldc, alpha, nullptr, accumulate, workspace, workspace_bytes,
                   stream, tile_m, k_step, splits);
}

extern "C" int64_t tgemm_act_grad_workspace(int64_t M, int64_t N) {
    if (check_dims(M, N, 0) != TGEMM_OK) return TGEMM_ERR_INVALID;
    return ceil_div(M, col_rows(M, N)) * N * 4;
}

namespace tg {
namespace {

// Workgroups of tgemm_largest_kernel: 256 columns and 64 rows each at least, 1024
// at most (every workgroup of the kernel after it reads all their maxima).
void largest_grid(int64_t M, int64_t N, int64_t* gx, int64_t* gy) {
    *gx = ceil_div(N, 256) < 256 ? ceil_div(N, 256) : 256;
    const int64_t most = 1024 / *gx;
    *gy = ceil_div(M, 64) < most ? ceil_div(M, 64) : most;
}

template <int AB, bool G32>
const void* act_grad_kernel(int act) {
    static const void* const fns[5] = {
        (const void*)&tgemm_act_grad_kernel<AB, kActNone, G32>, (const void*)&tgemm_act_grad_kernel<AB, kActRelu, G32>,
        (const void*)&tgemm_act_grad_kernel<AB, kActSilu, G32>, (const void*)&tgemm_act_grad_kernel<AB, kActGelu, G32>,
        (const void*)&tgemm_act_grad_kernel<AB, kActGeluTanh, G32>};
    return fns[act];
}

// Workspace: the column blocks' sums, behind them (fp32 dY) the parts' maxima.
int64_t act_grad_parts(int64_t M, int64_t N) { return ceil_div(M, col_rows(M, N)) * N * 4; }
constexpr int64_t kTopsBytes = 1024 * 4;

// tgemm_act_grad, tgemm_act_grad_f32 (f32).
int act_grad_call(int64_t M, int64_t N, int type, bool f32, const void* dY, int64_t lddy, int act, const void* pre,
                  int64_t ldpre, void* dP, int64_t lddp, float* scale, int dbias_type, void* dbias, void* workspace,
                  int64_t workspace_bytes, void* stream) {
    if (check_dims(M, N, 0) != TGEMM_OK || !is16(type)) return TGEMM_ERR_INVALID;
    if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_INVALID;
    if (dbias && dbias_type != type && dbias_type != TGEMM_F32) return TGEMM_ERR_INVALID;
    Mem in[2] = {}, out[3] = {};
    if (!array_ok(dY, M, N, lddy, f32 ? 4 : 2, &in[0])) return TGEMM_ERR_INVALID;
    if (act == TGEMM_ACT_NONE ? pre != nullptr : !array_ok(pre, M, N, ldpre, 2, &in[1])) return TGEMM_ERR_INVALID;
    const bool may = f32 ? !dP : act == TGEMM_ACT_NONE;       // calls without dP
    if (may ? dP != nullptr : !array_ok(dP, M, N, lddp, 2, &out[0])) return TGEMM_ERR_INVALID;
    if (dbias && !array_ok(dbias, 1, N, N > 1 ? N : 1, esize(dbias_type), &out[1])) return TGEMM_ERR_INVALID;
    if (f32 && ((scale != nullptr) != (dP != nullptr) || (scale && !array_ok(scale, 1, 1, 1, 4, &out[2])))) return TGEMM_ERR_INVALID;
    if (outputs_meet(in, 2, out, 3)) return TGEMM_ERR_INVALID;
    int per = col_rows(M, N);
    const int64_t blocks = ceil_div(M, per);
    const int64_t parts = dbias ? blocks * N * 4 : 0;
    const bool largest = f32 && dP && type == TGEMM_F16 && M > 0 && N > 0;
    const int64_t need = parts + (largest ? kTopsBytes : 0);
    if (!ws_ok(workspace, workspace_bytes, need)) return TGEMM_ERR_INVALID;
    const Mem mws{workspace, (uint64_t)need};
    if (outputs_meet(in, 2, &mws, 1) || outputs_meet(out, 3, &mws, 1)) return TGEMM_ERR_INVALID;
    if (N == 0 || (!dP && !dbias)) return TGEMM_OK;
    const int ab = type == TGEMM_BF16;
    float* part = dbias ? static_cast<float*>(workspace) : nullptr;
    int m = (int)M, n = (int)N;
    if (M > 0) {
        const float* tops = nullptr;
        int ntops = 0;
        if (largest) {
            int64_t gx, gy;
            largest_grid(M, N, &gx, &gy);
            ntops = (int)(gx * gy);
            float* t = reinterpret_cast<float*>(static_cast<char*>(workspace) + parts);
            tops = t;
            void* kargs[] = {&dY, &lddy, &m, &n, &t};
            const int rc = launch_k((const void*)&tgemm_largest_kernel, gx, gy, 256, kargs, stream);
            if (rc != TGEMM_OK) return rc;
        }
        void* kargs[] = {&dY, &lddy, &pre, &ldpre, &dP, &lddp, &part, &m, &n, &per, &tops, &ntops, &scale};
        const void* fn = f32 ? (ab ? act_grad_kernel<1, true>(act) : act_grad_kernel<0, true>(act))
                             : (ab ? act_grad_kernel<1, false>(act) : act_grad_kernel<0, false>(act));
        const int rc = launch_k(fn, ceil_div(N, 256), blocks, 256, kargs, stream);
        if (rc != TGEMM_OK) return rc;
    }
    if (!dbias) return TGEMM_OK;
    int nb = (int)blocks, out32 = dbias_type == TGEMM_F32;
    const float* cpart = part;
    void* kargs[] = {&cpart, &nb, &n, &dbias, &out32};
    return launch_k(ab ? (const void*)&tgemm_colsum_join_kernel<1> : (const void*)&tgemm_colsum_join_kernel<0>,
                    join_grid(ceil_div(N, 64)), 1, 256, kargs, stream);
}

}  // namespace
}  // namespace tg

extern "C" int tgemm_act_grad(int64_t M, int64_t N, int type, const void* dY, int64_t lddy, int act, const void* pre,
                              int64_t ldpre, void* dP, int64_t lddp, int dbias_type, void* dbias, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    return act_grad_call(M, N, type, false, dY, lddy, act, pre, ldpre, dP, lddp, nullptr, dbias_type, dbias, workspace,
                         workspace_bytes, stream);
}

extern "C" int64_t tgemm_act_grad_f32_workspace(int64_t M, int64_t N) {
    if (check_dims(M, N, 0) != TGEMM_OK) return TGEMM_ERR_INVALID;
    return act_grad_parts(M, N) + kTopsBytes;
}

extern "C" int tgemm_act_grad_f32(int64_t M, int64_t N, int type, const float* dY, int64_t lddy, int act, const void* pre,
                                  int64_t ldpre, void* dP, int64_t lddp, float* scale, int dbias_type, void* dbias,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    return act_grad_call(M, N, type, true, dY, lddy, act, pre, ldpre, dP, lddp, scale, dbias_type, dbias, workspace,
                         workspace_bytes, stream);
}

namespace tg {
namespace {

// Gradients of a linear layer: dP (with an activation, or from an fp32 dY, whose
// factor lies behind it) in rows of a multiple of 64 elements, then one area that
// the three steps use in turn.
struct LinGradPlan {
    int64_t ldp, off_scale, off, ws;
};

int plan_linear_grad(int64_t M, int64_t N, int64_t K, int type, bool f32, int64_t ldx, int64_t ldw, int w_layout, int act,
                     int64_t lddy, int64_t lddx, int64_t lddw, LinGradPlan* x) {
    if (check_dims(M, N, K) != TGEMM_OK || !is16(type)) return TGEMM_ERR_INVALID;
    if (w_layout != TGEMM_B_KxN && w_layout != TGEMM_B_NxK) return TGEMM_ERR_INVALID;
    if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_INVALID;
    if (lddy < (N > 1 ? N : 1)) return TGEMM_ERR_INVALID;
    if (!countable(M, N) || !countable(M, K) || !countable(N, K)) return TGEMM_ERR_UNSUPPORTED;
    const bool nxk = w_layout == TGEMM_B_NxK, own = f32 || act != TGEMM_ACT_NONE;
    x->ldp = own ? up(N > 0 ? N : 1, 64) : lddy;
    x->off_scale = own ? up(M * x->ldp * 2, 256) : 0;
    x->off = x->off_scale + (f32 ? 256 : 0);
    OpPlan dx, dw;
    int ncu;
    int rc = plan_linear(M, K, N, type, x->ldp, ldw, nxk ? TGEMM_B_KxN : TGEMM_B_NxK, type, lddx, 0, 0, 0, &ncu, &dx);
    if (rc != TGEMM_OK) return rc;
    rc = nxk ? plan_tn(N, K, M, type, x->ldp, ldx, type, lddw, 0, 0, 0, &ncu, &dw)
             : plan_tn(K, N, M, type, ldx, x->ldp, type, lddw, 0, 0, 0, &ncu, &dw);
    if (rc != TGEMM_OK) return rc;
    int64_t most = act_grad_parts(M, N) + (f32 ? kTopsBytes : 0);
    most = most > dx.ws ? most : dx.ws;
    most = most > dw.ws ? most : dw.ws;
    x->ws = x->off + most;
    return TGEMM_OK;
}

// tgemm_linear_grad, tgemm_linear_grad_f32 (f32).
int linear_grad_call(int64_t M, int64_t N, int64_t K, int type, bool f32, const void* X, int64_t ldx, const void* W,
                     int64_t ldw, int w_layout, int act, const void* pre, int64_t ldpre, const void* dY, int64_t lddy,
                     void* dX, int64_t lddx, void* dW, int64_t lddw, int dbias_type, void* dbias, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    if (check_dims(M, N, K) != TGEMM_OK || !is16(type)) return TGEMM_ERR_INVALID;
    if (w_layout != TGEMM_B_KxN && w_layout != TGEMM_B_NxK) return TGEMM_ERR_INVALID;
    if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GELU_TANH) return TGEMM_ERR_INVALID;
    if (dbias && dbias_type != type && dbias_type != TGEMM_F32) return TGEMM_ERR_INVALID;
    const bool nxk = w_layout == TGEMM_B_NxK;
    const int64_t wr = nxk ? N : K, wc = nxk ? K : N;
    Mem in[4] = {}, out[3] = {};
    if (!array_ok(X, M, K, ldx, 2, &in[0]) || !array_ok(W, wr, wc, ldw, 2, &in[1]) ||
        !array_ok(dY, M, N, lddy, f32 ? 4 : 2, &in[2]))
        return TGEMM_ERR_INVALID;
    if (act == TGEMM_ACT_NONE ? pre != nullptr : !array_ok(pre, M, N, ldpre, 2, &in[3])) return TGEMM_ERR_INVALID;
    if (dX && !array_ok(dX, M, K, lddx, 2, &out[0])) return TGEMM_ERR_INVALID;
    if (dW && !array_ok(dW, wr, wc, lddw, 2, &out[1])) return TGEMM_ERR_INVALID;
    if (dbias && !array_ok(dbias, 1, N, N > 1 ? N : 1, esize(dbias_type), &out[2])) return TGEMM_ERR_INVALID;
    if (outputs_meet(in, 4, out, 3)) return TGEMM_ERR_INVALID;
    LinGradPlan x;
    int rc = plan_linear_grad(M, N, K, type, f32, ldx, ldw, w_layout, act, lddy, dX ? lddx : (K > 1 ? K : 1),
                              dW ? lddw : (wc > 1 ? wc : 1), &x);
    if (rc != TGEMM_OK) return rc;
    if (!ws_ok(workspace, workspace_bytes, x.ws)) return TGEMM_ERR_INVALID;
    const Mem mws{workspace, (uint64_t)x.ws};
    if (outputs_meet(in, 4, &mws, 1) || outputs_meet(out, 3, &mws, 1)) return TGEMM_ERR_INVALID;
    const bool products = (dX && M > 0 && K > 0) || (dW && N > 0 && K > 0);
    const void* dP = dY;
    int64_t ldp = lddy;
    float* scale = f32 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + x.off_scale) : nullptr;
    char* area = static_cast<char*>(workspace) + x.off;
    const int64_t left = x.ws - x.off;
    if ((f32 || act != TGEMM_ACT_NONE) && (products || (dbias && !f32))) {
        rc = act_grad_call(M, N, type, f32, dY, lddy, act, pre, ldpre, workspace, x.ldp, scale, dbias_type, dbias, area, left,
                           stream);
        dP = workspace;
        ldp = x.ldp;
    } else if (dbias) {
        rc = act_grad_call(M, N, type, f32, dY, lddy, act, f32 ? pre : nullptr, ldpre, nullptr, 0, nullptr, dbias_type, dbias,
                           area, left, stream);
    }
    if (rc != TGEMM_OK) return rc;
    // (the factor of binary16's dP; of an empty dP none has been written)
    const float* undo = f32 && type == TGEMM_F16 && M > 0 && N > 0 ? scale : nullptr;
    if (dX) {
        rc = linear_call(M, K, N, type, dP, ldp, W, ldw, nxk ? TGEMM_B_KxN : TGEMM_B_NxK, nullptr, TGEMM_F32, TGEMM_ACT_NONE,
                         nullptr, 0, type, dX, lddx, nullptr, 0, 1.0f, undo, area, left, stream, 0, 0, 0);
        if (rc != TGEMM_OK) return rc;
    }
    if (dW)
        rc = nxk ? tn_call(N, K, M, type, dP, ldp, X, ldx, type, dW, lddw, 1.0f, undo, 0, area, left, stream, 0, 0, 0)
                 : tn_call(K, N, M, type, X, ldx, dP, ldp, type, dW, lddw, 1.0f, undo, 0, area, left, stream, 0, 0, 0);
    return rc;
}

}  // namespace
}  // namespace tg

extern "C" int64_t tgemm_linear_grad_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw,
                                               int w_layout, int act, int64_t lddy, int64_t lddx, int64_t lddw) {
    LinGradPlan x;
    const int rc = plan_linear_grad(M, N, K, type, false, ldx, ldw, w_layout, act, lddy, lddx, lddw, &x);
    return rc != TGEMM_OK ? rc : x.ws;
}

extern "C" int tgemm_linear_grad(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W,
                                 int64_t ldw, int w_layout, int act, const void* pre, int64_t ldpre, const void* dY,
                                 int64_t lddy, void* dX, int64_t lddx, void* dW, int64_t lddw, int dbias_type, void* dbias,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
    return linear_grad_call(M, N, K, type, false, X, ldx, W, ldw, w_layout, act, pre, ldpre, dY, lddy, dX, lddx, dW, lddw,
                            dbias_type, dbias, workspace, workspace_bytes, stream);
}

extern "C" int64_t tgemm_linear_grad_f32_workspace(int64_t M, int64_t N, int64_t K, int type, int64_t ldx, int64_t ldw,
                                                   int w_layout, int act, int64_t lddy, int64_t lddx, int64_t lddw) {
    LinGradPlan x;
    const int rc = plan_linear_grad(M, N, K, type, true, ldx, ldw, w_layout, act, lddy, lddx, lddw, &x);
    return rc != TGEMM_OK ? rc : x.ws;
}

extern "C" int tgemm_linear_grad_f32(int64_t M, int64_t N, int64_t K, int type, const void* X, int64_t ldx, const void* W,
                                     int64_t ldw, int w_layout, int act, const void* pre, int64_t ldpre, const float* dY,
                                     int64_t lddy, void* dX, int64_t lddx, void* dW, int64_t lddw, int dbias_type,
                                     void* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
    return linear_grad_call(M, N, K, type, true, X, ldx, W, ldw, w_layout, act, pre, ldpre, dY, lddy, dX, lddx, dW, lddw,
                            dbias_type, dbias, workspace, workspace_bytes, stream);
}

extern "C" int64_t tgemm_xent_workspace(int64_t rows, int64_t vocab, int64_t dim, int type, int64_t ldh, int64_t ldw) {
    XentPlan x;
    int ncu;
    const int rc = plan_xent(rows, vocab, dim, type, ldh, ldw, &ncu, &x);
    return rc != TGEMM_OK ? rc : x.ws;
}

extern "C" int tgemm_xent(int64_t rows, int64_t vocab, int64_t dim, int type, const void* H, int64_t ldh, const void* W,
                          int64_t ldw, const int64_t* target, int64_t ignore, int reduction, float* lse, float* loss,
                          float* total, float* count, void* workspace, int64_t workspace_bytes, void* stream) {
    if (check_dims(rows, vocab, dim) != TGEMM_OK || !is16(type) || dim < 8 || vocab < 1 || vocab > kMaxDim / 4)
        return TGEMM_ERR_INVALID;
    if (reduction < TGEMM_REDUCE_NONE || reduction > TGEMM_REDUCE_MEAN) return TGEMM_ERR_INVALID;
    const bool reduced = reduction != TGEMM_REDUCE_NONE;
    if (reduced != (total != nullptr) || reduced != (count != nullptr) || (reduced && rows == 0)) return TGEMM_ERR_INVALID;
    Mem in[3], out[4] = {};
    if (!array_ok(H, rows, dim, ldh, 2, &in[0]) || !array_ok(W, vocab, dim, ldw, 2, &in[1]) ||
        !array_ok(target, 1, rows, rows > 1 ? rows : 1, 8, &in[2]) ||
        !array_ok(lse, 1, rows, rows > 1 ? rows : 1, 4, &out[0]) ||
        !array_ok(loss, 1, rows, rows > 1 ? rows : 1, 4, &out[1]))
        return TGEMM_ERR_INVALID;
    if (reduced && (!array_ok(total, 1, 1, 1, 4, &out[2]) || !array_ok(count, 1, 1, 1, 4, &out[3]))) return TGEMM_ERR_INVALID;
    if (outputs_meet(in, 3, out, 4)) return TGEMM_ERR_INVALID;
    XentPlan x;
    int ncu;
    int rc = plan_xent(rows, vocab, dim, type, ldh, ldw, &ncu, &x);
    if (rc != TGEMM_OK) return rc;
    if (!ws_ok(workspace, workspace_bytes, x.ws)) return TGEMM_ERR_INVALID;
    const Mem mws{workspace, (uint64_t)x.ws};
    if (outputs_meet(in, 3, &mws, 1) || outputs_meet(out, 4, &mws, 1)) return TGEMM_ERR_INVALID;
    if (rows == 0) return TGEMM_OK;
    OpArgs a = op_args();
    a.A = static_cast<const uint16_t*>(H);
    a.B = static_cast<const uint16_t*>(W);
    a.lda = ldh;
    a.ldb = ldw;
    a.M = (int)rows;
    a.N = (int)vocab;
    a.K = (int)dim;
    a.target = target;
    a.part = static_cast<float2*>(workspace);
    a.zt = reinterpret_cast<float*>(static_cast<char*>(workspace) + up(x.parts * rows * 8, 16));
    const int ab = type == TGEMM_BF16;
    if (x.few) {
        void* kargs[] = {&a};
        const void* fn = ab ? xent_few_kernel<1>(rows) : xent_few_kernel<0>(rows);
        rc = launch_k(fn, x.waves, 1, 64, kargs, stream);
    } else {
        rc = launch_tile(a, ab, kEndXentFwd, kActNone, 1, 0, x.tile, ncu, stream);
    }
    if (rc != TGEMM_OK) return rc;
    return xent_finish(a, x.parts, vocab, ignore, reduction, lse, loss, total, count, nullptr, nullptr, stream);
}

extern "C" int64_t tgemm_xent_grad_workspace(int64_t rows, int64_t vocab, int64_t dim, int type, int64_t ldh, int64_t ldw,
                                             int64_t lddh, int64_t lddw) {
    XentGradPlan x;
    int ncu;
    const int rc = plan_xent_grad(rows, vocab, dim, type, ldh, ldw, lddh, lddw, &ncu, &x);
    return rc != TGEMM_OK ? rc : x.ws;
}

extern "C" int tgemm_xent_grad(int64_t rows, int64_t vocab, int64_t dim, int type, const void* H, int64_t ldh,
                               const void* W, int64_t ldw, const int64_t* target, int64_t ignore, const float* lse,
                               const float* dloss, int dloss_stride, const float* count, const float* dlse, void* dH,
                               int64_t lddh, void* dW, int64_t lddw, void* workspace, int64_t workspace_bytes,
                               void* stream) {
    if (check_dims(rows, vocab, dim) != TGEMM_OK || !is16(type) || dim < 8 || vocab < 1 || vocab > kMaxDim / 4)
        return TGEMM_ERR_INVALID;
    if (dloss_stride != 0 && dloss_stride != 1) return TGEMM_ERR_INVALID;
    const int64_t rl = rows > 1 ? rows : 1;
    Mem in[7] = {}, out[2] = {};
    if (!array_ok(H, rows, dim, ldh, 2, &in[0]) || !array_ok(W, vocab, dim, ldw, 2, &in[1]) ||
        !array_ok(target, 1, rows, rl, 8, &in[2]) || !array_ok(lse, 1, rows, rl, 4, &in[3]))
        return TGEMM_ERR_INVALID;
    if (dloss && !array_ok(dloss, 1, dloss_stride ? rows : 1, dloss_stride ? rl : 1, 4, &in[4])) return TGEMM_ERR_INVALID;
    if (count && !array_ok(count, 1, 1, 1, 4, &in[5])) return TGEMM_ERR_INVALID;
    if (dlse && !array_ok(dlse, 1, rows, rl, 4, &in[6])) return TGEMM_ERR_INVALID;
    if (dH && !array_ok(dH, rows, dim, lddh, 2, &out[0])) return TGEMM_ERR_INVALID;
    if (dW && !array_ok(dW, vocab, dim, lddw, 2, &out[1])) return TGEMM_ERR_INVALID;
    if (outputs_meet(in, 7, out, 2)) return TGEMM_ERR_INVALID;
    XentGradPlan x;
    int ncu;
    int rc = plan_xent_grad(rows, vocab, dim, type, ldh, ldw, dH ? lddh : dim, dW ? lddw : dim, &ncu, &x);
    if (rc != TGEMM_OK) return rc;
    if (!ws_ok(workspace, workspace_bytes, x.ws)) return TGEMM_ERR_INVALID;
    const Mem mws{workspace, (uint64_t)x.ws};
    if (outputs_meet(in, 7, &mws, 1) || outputs_meet(out, 2, &mws, 1)) return TGEMM_ERR_INVALID;
    if (!dH && !dW) return TGEMM_OK;
    const int ab = type == TGEMM_BF16;
    if (rows == 0) {
        // no rows: dW is zero
        if (!dW) return TGEMM_OK;
        OpArgs z = op_args();
        z.C = dW;
        z.ldc = lddw;
        z.M = (int)vocab;
        z.N = (int)dim;
        return launch_join(z, ab, nullptr, 0, false, false, stream);
    }
    char* ws = static_cast<char*>(workspace);
    XentRow* recs = reinterpret_cast<XentRow*>(ws);
    float* scale = reinterpret_cast<float*>(ws + x.off_scale);
    uint16_t* G = reinterpret_cast<uint16_t*>(ws + x.off_g);
    float* sums = reinterpret_cast<float*>(ws + x.off_sums);
    {
        int r = (int)rows, shift = type == TGEMM_F16 ? 15 : 0, st = dloss_stride;
        void* kargs[] = {&lse, &target, &vocab, &ignore, &dloss, &st, &count, &dlse, &r, &shift, &recs, &scale};
        rc = launch_k((const void*)&tgemm_xent_rows_kernel, 1, 1, 1024, kargs, stream);
        if (rc != TGEMM_OK) return rc;
    }
    const uint16_t* Wp = static_cast<const uint16_t*>(W);
    for (int64_t q = 0; q < x.pieces; ++q) {
        const int64_t v0 = q * x.piece;
        const int64_t n = vocab - v0 < x.piece ? vocab - v0 : x.piece;
        OpPlan pl;
        {
            // G = the coefficients of the piece
            rc = plan_product(rows, n, dim, ldh, ldw, 1, 0, true, true, false, 0, 0, 0, ncu, &pl);
            if (rc != TGEMM_OK) return rc;
            OpArgs a = op_args();
            a.A = static_cast<const uint16_t*>(H);
            a.B = Wp + v0 * ldw;
            a.C = G;
            a.lda = ldh;
            a.ldb = ldw;
            a.ldc = x.ldg;
            a.M = (int)rows;
            a.N = (int)n;
            a.K = (int)dim;
            a.rows = recs;
            a.v0 = (int)v0;
            rc = launch_tile(a, ab, kEndXentBwd, kActNone, 1, 0, pl, ncu, stream);
            if (rc != TGEMM_OK) return rc;
        }
        if (dH) {
            OpArgs a = op_args();
            a.A = G;
            a.B = Wp + v0 * ldw;
            a.lda = x.ldg;
            a.ldb = ldw;
            a.M = (int)rows;
            a.N = (int)dim;
            a.K = (int)n;
            if (!x.dh_sums) {
                a.C = dH;
                a.ldc = lddh;
                a.alpha_dev = scale;
                rc = launch_tile(a, ab, kEndLin16, kActNone, 0, 0, x.dh, ncu, stream);
            } else {
                // running sums over the pieces: every part of the first piece
                // writes its array, later pieces add to the parts they have
                pl = x.dh;
                if (n != x.piece) {
                    rc = plan_product(rows, dim, n, x.ldg, ldw, 0, 0, false, false, false, 0, 0, 0, ncu, &pl);
                    if (rc != TGEMM_OK) return rc;
                    if (pl.splits > x.dh.splits) {
                        rc = plan_product(rows, dim, n, x.ldg, ldw, 0, 0, false, true, false, 0, 0, 0, ncu, &pl);
                        if (rc != TGEMM_OK) return rc;
                    }
                }
                a.C = sums;
                a.ldc = dim;
                a.res = q ? sums : nullptr;
                a.ldres = q ? dim : 0;
                rc = launch_tile(a, ab, kEndAcc32, kActNone, 0, 0, pl, ncu, stream);
            }
            if (rc != TGEMM_OK) return rc;
        }
        if (dW) {
            rc = plan_product(n, dim, rows, x.ldg, ldh, 0, 1, true, false, false, 0, 0, 0, ncu, &pl);
            if (rc != TGEMM_OK) return rc;
            OpArgs a = op_args();
            a.A = G;
            a.B = static_cast<const uint16_t*>(H);
            a.C = static_cast<uint16_t*>(dW) + v0 * lddw;
            a.lda = x.ldg;
            a.ldb = ldh;
            a.ldc = lddw;
            a.M = (int)n;
            a.N = (int)dim;
            a.K = (int)rows;
            a.alpha_dev = scale;
            rc = run_tn(a, ab, false, pl, ncu, ws + x.off_dw, stream);
            if (rc != TGEMM_OK) return rc;
        }
    }
    if (dH && x.dh_sums) {
        OpArgs a = op_args();
        a.C = dH;
        a.ldc = lddh;
        a.M = (int)rows;
        a.N = (int)dim;
        a.alpha_dev = scale;
        return launch_join(a, ab, sums, x.dh.splits, false, false, stream);
    }
    return TGEMM_OK;
}

extern "C" int64_t tgemm_xent_both_workspace(int64_t rows, int64_t vocab, int64_t dim, int type, int64_t ldh, int64_t ldw,
                                             int64_t lddh, int64_t lddw) {
    XentBothPlan x;
    int ncu;
    const int rc = plan_xent_both(rows, vocab, dim, type, ldh, ldw, lddh, lddw, &ncu, &x);
    return rc != TGEMM_OK ? rc : x.ws;
}

extern "C" int tgemm_xent_both(int64_t rows, int64_t vocab, int64_t dim, int type, const void* H, int64_t ldh, const void* W,
                               int64_t ldw, const int64_t* target, int64_t ignore, int reduction, float* lse, float* loss,
                               float* total, float* count, void* dH, int64_t lddh, void* dW, int64_t lddw, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    if (check_dims(rows, vocab, dim) != TGEMM_OK || !is16(type) || dim < 8 || vocab < 1 || vocab > kMaxDim / 4 || rows < 1)
        return TGEMM_ERR_INVALID;
    if ((reduction != TGEMM_REDUCE_SUM && reduction != TGEMM_REDUCE_MEAN) || !total || !count) return TGEMM_ERR_INVALID;
    const int64_t rl = rows > 1 ? rows : 1;
    Mem in[3], out[6] = {};
    if (!array_ok(H, rows, dim, ldh, 2, &in[0]) || !array_ok(W, vocab, dim, ldw, 2, &in[1]) ||
        !array_ok(target, 1, rows, rl, 8, &in[2]) || !array_ok(lse, 1, rows, rl, 4, &out[0]) ||
        !array_ok(loss, 1, rows, rl, 4, &out[1]) || !array_ok(total, 1, 1, 1, 4, &out[2]) ||
        !array_ok(count, 1, 1, 1, 4, &out[3]))
        return TGEMM_ERR_INVALID;
    if (dH && !array_ok(dH, rows, dim, lddh, 2, &out[4])) return TGEMM_ERR_INVALID;
    if (dW && !array_ok(dW, vocab, dim, lddw, 2, &out[5])) return TGEMM_ERR_INVALID;
    if (outputs_meet(in, 3, out, 6)) return TGEMM_ERR_INVALID;
    XentBothPlan x;
    int ncu;
    int rc = plan_xent_both(rows, vocab, dim, type, ldh, ldw, dH ? lddh : dim, dW ? lddw : dim, &ncu, &x);
    if (rc != TGEMM_OK) return rc;
    if (!ws_ok(workspace, workspace_bytes, x.ws)) return TGEMM_ERR_INVALID;
    const Mem mws{workspace, (uint64_t)x.ws};
    if (outputs_meet(in, 3, &mws, 1) || outputs_meet(out, 6, &mws, 1)) return TGEMM_ERR_INVALID;
    const int ab = type == TGEMM_BF16;
    char* ws = static_cast<char*>(workspace);
    uint16_t* G = reinterpret_cast<uint16_t*>(ws + x.off_g);
    XentRow* recs = reinterpret_cast<XentRow*>(ws + x.off_recs);
    float* scale = reinterpret_cast<float*>(ws + x.off_scale);
    OpArgs a = op_args();
    a.A = static_cast<const uint16_t*>(H);
    a.B = static_cast<const uint16_t*>(W);
    a.C = G;
    a.lda = ldh;
    a.ldb = ldw;
    a.ldc = x.ldg;
    a.M = (int)rows;
    a.N = (int)vocab;
    a.K = (int)dim;
    a.target = target;
    a.part = reinterpret_cast<float2*>(ws);
    a.zt = reinterpret_cast<float*>(ws + x.off_zt);
    rc = launch_tile(a, ab, kEndXentExp, kActNone, 1, 0, x.fwd, ncu, stream);
    if (rc == TGEMM_OK) rc = xent_finish(a, x.parts, vocab, ignore, reduction, lse, loss, total, count, recs, scale, stream);
    if (rc != TGEMM_OK || (!dH && !dW)) return rc;
    {
        const float2* part = a.part;
        const float* zt = a.zt;
        const XentRow* crecs = recs;
        int r = (int)rows, v = (int)vocab;
        void* kargs[] = {&G, &x.ldg, &part, &zt, &crecs, &r, &v};
        rc = launch_k((const void*)&tgemm_xent_coef_kernel<1>, ceil_div(rows, 16), ceil_div(vocab, 2048), 256, kargs, stream);
        if (rc != TGEMM_OK) return rc;
    }
    if (dH) {
        OpArgs p = op_args();
        p.A = G;
        p.B = static_cast<const uint16_t*>(W);
        p.C = dH;
        p.lda = x.ldg;
        p.ldb = ldw;
        p.ldc = lddh;
        p.M = (int)rows;
        p.N = (int)dim;
        p.K = (int)vocab;
        p.alpha_dev = scale;
        rc = run_linear(p, ab, 0, false, type, x.dh, ncu, ws + x.off_area, stream);
        if (rc != TGEMM_OK) return rc;
    }
    if (dW) {
        OpArgs p = op_args();
        p.A = G;
        p.B = static_cast<const uint16_t*>(H);
        p.C = dW;
        p.lda = x.ldg;
        p.ldb = ldh;
        p.ldc = lddw;
        p.M = (int)vocab;
        p.N = (int)dim;
        p.K = (int)rows;
        p.alpha_dev = scale;
        rc = run_tn(p, ab, false, x.dw, ncu, ws + x.off_area, stream);
    }
    return rc;
}

extern "C" int tgemm_scale(int type, int64_t n, void* X, int64_t n2, void* X2, const float* factor, void* stream) {
    if (n < 0 || n2 < 0 || !is16(type)) return TGEMM_ERR_INVALID;
    if (n == 0 && n2 == 0) return TGEMM_OK;
    if ((n && !X) || (n2 && !X2) || (uintptr_t)X % 16 || (uintptr_t)X2 % 16) return TGEMM_ERR_INVALID;
    if (!factor || (uintptr_t)factor % 4) return TGEMM_ERR_INVALID;
    const Mem a{X, (uint64_t)n * 2}, b{X2, (uint64_t)n2 * 2}, f{factor, 4};
    if (meet(a, b) || meet(a, f) || meet(b, f)) return TGEMM_ERR_INVALID;
    const int64_t blocks = ceil_div(n > n2 ? n : n2, 2048);
    void* kargs[] = {&X, &n, &X2, &n2, &factor};
    return launch_k(type == TGEMM_BF16 ? (const void*)&tgemm_scale_kernel<1> : (const void*)&tgemm_scale_kernel<0>,
                    blocks < 512 ? blocks : 512, 1, 256, kargs, stream);
}
