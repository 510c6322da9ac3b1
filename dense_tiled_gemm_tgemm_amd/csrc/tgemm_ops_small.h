// Device code of the operators around the product that does not run on the
// tile pipeline: products with few rows, joins of split products and of the
// cross entropy's parts, the activation's gradient with column sums. Included
// by tgemm_ops.hip.
#pragma once

#include "tgemm_ops_kernels.h"

namespace tg {
// ------------------------------------------------------- few rows of A --
// C = act(alpha A B + bias) + residual for blocks of at most 16 MB rows of A and
// a B stored N x K (a token's or a small batch's pass through a layer: one block;
// small products: several). What counts is reading the weight once: a workgroup
// owns 16 columns, its KW waves walk the K axis in turn in pieces of 128 (256
// bytes of 16 weight rows), with the next piece in flight while the current one
// is multiplied, no LDS staging and no barrier on the way. The waves' sums meet
// in LDS and are added in wave order.
//
// v_mfma_f32_16x16x32 wants lane l to hold chunk l / 16 of row l mod 16. Loaded
// that way, each 16 lanes touch 16 rows and the vector L1 serves 16 bytes a
// clock; four neighbouring lanes on 64 bytes of one row (row l / 4, chunk l mod
// 4) are served four times as fast, and ds_bpermute brings the chunks to their
// lanes. 8 x 12288 x 12288: 69.9 -> 58.8 us, 16 x 4096 x 12288: 26.9 -> 21.9
// (with the steps after it 53.6, 5.6 TB/s of weight, and 21.4). A's rows come
// through the caches the same way, or, up to 4 rows (XP = 0), in the operand's
// layout at once.
__device__ __forceinline__ u32x4 load16_lanes(const BufRsrc& rs, unsigned off, int soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)off, soff, 0));
#else
    (void)rs; (void)off; (void)soff;
    return u32x4{};
#endif
}

__device__ __forceinline__ BufRsrc bytes_rsrc(const void* p, int64_t bytes) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(bytes > 0x7fffffff ? 0x7fffffff : bytes),
                                             0x00020000);
#else
    (void)p; (void)bytes;
    return 0;
#endif
}

constexpr int kFewU = 4;                              // 32-deep steps of a piece
constexpr int kFewK = 32 * kFewU;                     // k of a piece

// One piece's fragments: the weight's and A's 16-byte chunks of steps k0 .. , as
// loaded. Chunks that do not end inside K read zeros (a last partial chunk is
// added by few_tail). woff, xoff: byte offsets of the lane's chunk at k = 0.
template <int MB>
struct FewFrags {
    u32x4 w[kFewU], x[MB][kFewU];
};

template <int MB, int XP>
__device__ __forceinline__ void few_load(FewFrags<MB>& f, const BufRsrc& rw, const BufRsrc& rx, unsigned woff,
                                         const unsigned (&xoff)[MB], int k0, int K, int lane) {
    if (k0 + kFewK <= K) {                            // uniform
#pragma unroll
        for (int u = 0; u < kFewU; ++u) {
            f.w[u] = load16_lanes(rw, woff, 2 * (k0 + 32 * u));
#pragma unroll
            for (int m = 0; m < MB; ++m) f.x[m][u] = load16_lanes(rx, xoff[m], 2 * (k0 + 32 * u));
        }
    } else {
        const int cw = lane & 3, cx = XP ? cw : lane >> 4;
#pragma unroll
        for (int u = 0; u < kFewU; ++u) {
            const bool okw = k0 + 32 * u + 8 * cw + 8 <= K, okx = k0 + 32 * u + 8 * cx + 8 <= K;
            f.w[u] = load16_lanes(rw, okw ? woff : kCOob, 2 * (k0 + 32 * u));
#pragma unroll
            for (int m = 0; m < MB; ++m) f.x[m][u] = load16_lanes(rx, okx ? xoff[m] : kCOob, 2 * (k0 + 32 * u));
        }
    }
}

// Offsets of the lane's chunk of 16 weight rows / of A's row block m.
__device__ __forceinline__ unsigned few_woff(int lane, int ncols, int64_t ldb) {
    return (lane >> 2) < ncols ? (unsigned)(lane >> 2) * (unsigned)(ldb * 2) + 16u * (unsigned)(lane & 3) : kCOob;
}
template <int XP>
__device__ __forceinline__ unsigned few_xoff(int lane, int m, int M, int64_t lda) {
    const int row = 16 * m + (XP ? lane >> 2 : lane & 15), c = XP ? lane & 3 : lane >> 4;
    return row < M ? (unsigned)row * (unsigned)(lda * 2) + 16u * (unsigned)c : kCOob;
}

// A chunk from the lane that loaded it: `from` = 4 (4 (l mod 16) + l / 16).
__device__ __forceinline__ half8 few_perm(const u32x4& v, int from) {
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (unsigned)__builtin_amdgcn_ds_bpermute(from, (int)v[e]);
    return __builtin_bit_cast(half8, o);
}

template <int AB, int MB, int XP>
__device__ __forceinline__ void few_mma(f32x4 (&acc)[MB], const FewFrags<MB>& f, int from) {
#pragma unroll
    for (int u = 0; u < kFewU; ++u) {
        const half8 w = few_perm(f.w[u], from);
#pragma unroll
        for (int m = 0; m < MB; ++m)
            acc[m] = mfma16<AB>(w, XP ? few_perm(f.x[m][u], from) : __builtin_bit_cast(half8, f.x[m][u]), acc[m]);
        if (u & 1) __builtin_amdgcn_sched_barrier(0);
    }
}

// The last K mod 8 values, element by element, as one more 32-deep step of
// which only the first chunk (lanes 0-15) is not zero.
template <int AB, int MB>
__device__ __forceinline__ void few_tail(f32x4 (&acc)[MB], const OpArgs& a, int n, int r16, int g) {
    const int kt = a.K & ~7;
    const bool on = g == 0;
    const half8 w = __builtin_bit_cast(half8, load8_elems(a.B + (on && n < a.N ? (int64_t)n * a.ldb + kt : 0),
                                                          on && n < a.N ? a.K - kt : 0));
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const int row = 16 * m + r16;
        const half8 x = __builtin_bit_cast(half8, load8_elems(a.A + (on && row < a.M ? (int64_t)row * a.lda + kt : 0),
                                                              on && row < a.M ? a.K - kt : 0));
        acc[m] = mfma16<AB>(w, x, acc[m]);
    }
}

__device__ __forceinline__ float act_any(int act, float x) {
    switch (act) {
        case kActRelu: return act_fwd<kActRelu>(x);
        case kActSilu: return act_fwd<kActSilu>(x);
        case kActGelu: return act_fwd<kActGelu>(x);
        case kActGeluTanh: return act_fwd<kActGeluTanh>(x);
        default: return x;
    }
}

// One output of the linear epilogue from its sum (c32: fp32 C; rf32: fp32 residual).
template <int AB>
__device__ __forceinline__ void finish_one(const OpArgs& a, float sum, float alpha, int row, int col, bool c32, bool rf32) {
    float v = __builtin_fmaf(alpha, sum, a.biasv ? load_elem<AB>(a.biasv, a.bias_f32, col) : 0.f);
    if (a.pre) static_cast<uint16_t*>(a.pre)[(int64_t)row * a.ldpre + col] = to16<AB>(v);
    v = act_any(a.act, v);
    if (a.res) v += load_elem<AB>(a.res, rf32, (int64_t)row * a.ldres + col);
    if (c32)
        static_cast<float*>(a.C)[(int64_t)row * a.ldc + col] = v;
    else
        static_cast<uint16_t*>(a.C)[(int64_t)row * a.ldc + col] = to16<AB>(v);
}

template <int AB, int MB, int XP, int KW>
__global__ void __launch_bounds__(64 * KW) __attribute__((amdgpu_waves_per_eu(MB == 1 ? 5 : 4)))
tgemm_few_kernel(OpArgs a, int c32) {
    static_assert(XP || MB == 1, "A in the operand's layout: at most 16 rows");
    __shared__ f32x4 red[KW][MB][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int from = 4 * (4 * r16 + g);
    const int n0 = 16 * (int)blockIdx.x;
    const int ncols = a.N - n0 < 16 ? a.N - n0 : 16;
    const int row0 = 16 * MB * (int)blockIdx.y;       // more rows: one workgroup per 16 MB of them
    a.A += (int64_t)row0 * a.lda;
    a.M = a.M - row0 < 16 * MB ? a.M - row0 : 16 * MB;
    const BufRsrc rw = bytes_rsrc(a.B + (int64_t)n0 * a.ldb, ((int64_t)(ncols - 1) * a.ldb + a.K) * 2);
    const BufRsrc rx = bytes_rsrc(a.A, ((int64_t)(a.M - 1) * a.lda + a.K) * 2);
    const unsigned woff = few_woff(lane, ncols, a.ldb);
    unsigned xoff[MB];
    f32x4 acc[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        xoff[m] = few_xoff<XP>(lane, m, a.M, a.lda);
        acc[m] = f32x4{};
    }
    const int np = (a.K + kFewK - 1) / kFewK;
    FewFrags<MB> f0, f1;
    int p = wave;
    if (p < np) few_load<MB, XP>(f0, rw, rx, woff, xoff, p * kFewK, a.K, lane);
    while (p < np) {
        const int p1 = p + KW, p2 = p + 2 * KW;
        if (p1 < np) few_load<MB, XP>(f1, rw, rx, woff, xoff, p1 * kFewK, a.K, lane);
        few_mma<AB, MB, XP>(acc, f0, from);
        if (p1 >= np) break;
        if (p2 < np) few_load<MB, XP>(f0, rw, rx, woff, xoff, p2 * kFewK, a.K, lane);
        few_mma<AB, MB, XP>(acc, f1, from);
        p = p2;
    }
    if ((a.K & 7) && wave == 0) few_tail<AB, MB>(acc, a, n0 + r16, r16, g);
#pragma unroll
    for (int m = 0; m < MB; ++m) red[wave][m][lane] = acc[m];
    __syncthreads();
    if (wave >= MB) return;
    f32x4 s = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < KW; ++w) s += red[w][wave][lane];
    const int row = 16 * wave + r16;
    if (row >= a.M) return;
    const float alpha = a.alpha_dev ? a.alpha * *a.alpha_dev : a.alpha;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int col = n0 + 4 * g + e;
        if (col < a.N) finish_one<AB>(a, s[e], alpha, row0 + row, col, c32 != 0, false);
    }
}

// Cross entropy, forward, for at most 16 MB rows: one wave per workgroup walks
// every grid-th group of 16 vocabulary rows over the whole K axis (the weight is
// read once, as in tgemm_few_kernel) and keeps, per lane, the running maximum
// and sum of its four columns of each row; the lanes of a row are joined once,
// at the end, into one part per wave.
template <int AB, int MB, int XP>
__global__ void __launch_bounds__(64) tgemm_xent_few_kernel(OpArgs a) {
    const int lane = threadIdx.x;
    const int r16 = lane & 15, g = lane >> 4;
    const int from = 4 * (4 * r16 + g);
    const int np = (a.K + kFewK - 1) / kFewK;
    const int groups = (a.N + 15) / 16;
    const BufRsrc rx = bytes_rsrc(a.A, ((int64_t)(a.M - 1) * a.lda + a.K) * 2);
    unsigned xoff[MB];
    float mx[MB], sum[MB];
    int64_t tgt[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const int row = 16 * m + r16;
        xoff[m] = few_xoff<XP>(lane, m, a.M, a.lda);
        tgt[m] = row < a.M ? a.target[row] : -1;
        mx[m] = -__builtin_inff();
        sum[m] = 0.f;
    }
    for (int cg = (int)blockIdx.x; cg < groups; cg += (int)gridDim.x) {
        const int n0 = 16 * cg;
        const int ncols = a.N - n0 < 16 ? a.N - n0 : 16;
        const BufRsrc rw = bytes_rsrc(a.B + (int64_t)n0 * a.ldb, ((int64_t)(ncols - 1) * a.ldb + a.K) * 2);
        const unsigned woff = few_woff(lane, ncols, a.ldb);
        f32x4 acc[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[m] = f32x4{};
        FewFrags<MB> f0, f1;
        few_load<MB, XP>(f0, rw, rx, woff, xoff, 0, a.K, lane);
        for (int p = 0; p < np; p += 2) {
            if (p + 1 < np) few_load<MB, XP>(f1, rw, rx, woff, xoff, (p + 1) * kFewK, a.K, lane);
            few_mma<AB, MB, XP>(acc, f0, from);
            if (p + 1 >= np) break;
            if (p + 2 < np) few_load<MB, XP>(f0, rw, rx, woff, xoff, (p + 2) * kFewK, a.K, lane);
            few_mma<AB, MB, XP>(acc, f1, from);
        }
        if (a.K & 7) few_tail<AB, MB>(acc, a, n0 + r16, r16, g);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            f32x4 z = acc[m];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = n0 + 4 * g + e;
                if (col >= a.N) z[e] = -__builtin_inff();
                else if (tgt[m] == col) a.zt[16 * m + r16] = z[e];
            }
            const float top = fmaxf(mx[m], fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
            const float nm2 = -kLog2e * finite_max(top);
            // (a running maximum of -inf comes with a sum of 0; one of +inf keeps its weight; one
            // that stays keeps 1: taken through nm2, whose product is rounded, every group would
            // multiply the sum by the same factor beside 1, 2e-4 of lse over 600,000 columns)
            const float keep = __builtin_fabsf(mx[m]) == __builtin_inff()
                                   ? 1.f
                                   : __builtin_amdgcn_exp2f(kLog2e * (mx[m] - finite_max(top)));
            float s = sum[m] * keep;
#pragma unroll
            for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(__builtin_fmaf(kLog2e, z[e], nm2));
            mx[m] = top;
            sum[m] = s;
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const float top = max4g(mx[m]);
        const float w = __builtin_fabsf(mx[m]) == __builtin_inff()
                            ? 1.f
                            : __builtin_amdgcn_exp2f(kLog2e * (mx[m] - finite_max(top)));
        const float s = sum4g(sum[m] * w);
        const int row = 16 * m + r16;
        if (g == 0 && row < a.M) a.part[(int64_t)blockIdx.x * a.M + row] = float2{top, s};
    }
}

// Four neighbouring outputs of a row at once (all inside N).
template <int AB>
__device__ __forceinline__ void finish_four(const OpArgs& a, const float (&sum)[4], float alpha, int row, int col, bool c32,
                                            bool rf32) {
    typedef f32x4 __attribute__((aligned(4))) f32x4u;
    typedef u32x2 __attribute__((aligned(2))) u32x2u;
    auto four16 = [](const void* p, int64_t i) {
        const u32x2 w = *reinterpret_cast<const u32x2u*>(static_cast<const uint16_t*>(p) + i);
        return f32x4{lo16<AB>(w[0]), hi16<AB>(w[0]), lo16<AB>(w[1]), hi16<AB>(w[1])};
    };
    auto put16 = [](void* p, int64_t i, const f32x4& v) {
        *reinterpret_cast<u32x2u*>(static_cast<uint16_t*>(p) + i) = u32x2{pack2<AB>(v[0], v[1]), pack2<AB>(v[2], v[3])};
    };
    f32x4 b{}, r{}, v;
    if (a.biasv) b = a.bias_f32 ? *reinterpret_cast<const f32x4u*>(static_cast<const float*>(a.biasv) + col) : four16(a.biasv, col);
    if (a.res) {
        const int64_t i = (int64_t)row * a.ldres + col;
        r = rf32 ? *reinterpret_cast<const f32x4u*>(static_cast<const float*>(a.res) + i) : four16(a.res, i);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(alpha, sum[e], b[e]);
    if (a.pre) put16(a.pre, (int64_t)row * a.ldpre + col, v);
    auto act = [&](auto f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = f(v[e]) + r[e];
    };
    switch (a.act) {
        case kActRelu: act([](float x) { return act_fwd<kActRelu>(x); }); break;
        case kActSilu: act([](float x) { return act_fwd<kActSilu>(x); }); break;
        case kActGelu: act([](float x) { return act_fwd<kActGelu>(x); }); break;
        case kActGeluTanh: act([](float x) { return act_fwd<kActGeluTanh>(x); }); break;
        default: act([](float x) { return x; });
    }
    const int64_t o = (int64_t)row * a.ldc + col;
    if (c32)
        *reinterpret_cast<f32x4u*>(static_cast<float*>(a.C) + o) = v;
    else
        put16(a.C, o, v);
}

// ------------------------------------------------------------- joins --
// The parts of a split product (fp32, splits arrays of M x N) added in order,
// then the linear epilogue. splits == 0: a product over an empty K axis.
template <int AB>
__global__ void __launch_bounds__(256) tgemm_join_kernel(OpArgs a, const float* sums, int c32, int rf32) {
    const int64_t quads = ((int64_t)a.N + 3) / 4;
    const int64_t total = quads * a.M;
    const int64_t mn = (int64_t)a.M * a.N;
    const float alpha = a.alpha_dev ? a.alpha * *a.alpha_dev : a.alpha;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int row = (int)(t / quads);
        const int col = 4 * (int)(t - (int64_t)row * quads);
        const float* p = sums + (int64_t)row * a.N + col;
        const int n = a.N - col < 4 ? a.N - col : 4;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        if (n == 4) {
            typedef f32x4 __attribute__((aligned(4))) f32x4u;
#pragma unroll 4
            for (int q = 0; q < a.splits; ++q) {
                const f32x4 v = *reinterpret_cast<const f32x4u*>(p + q * mn);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += v[e];
            }
            finish_four<AB>(a, s, alpha, row, col, c32 != 0, rf32 != 0);
        } else {
            for (int q = 0; q < a.splits; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < n) s[e] += p[q * mn + e];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) finish_one<AB>(a, s[e], alpha, row, col + e, c32 != 0, rf32 != 0);
        }
    }
}

// C^T-operand product for shapes the tile kernel does not take (fewer than 8
// columns of an operand, row strides past its limit): a workgroup sums one row
// and 32 columns of C, eight parts of the K axis side by side.
template <int AB>
__global__ void __launch_bounds__(256) tgemm_tn_narrow_kernel(OpArgs a, float* sums) {
    __shared__ float red[8][32];
    const int c = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int64_t nb = ((int64_t)a.N + 31) / 32;
    for (int64_t t = blockIdx.x; t < nb * a.M; t += gridDim.x) {
        const int64_t m = t / nb, n = (t - m * nb) * 32 + c;
        float s = 0.f;
        if (n < a.N)
            for (int64_t k = part; k < a.K; k += 8)
                s = __builtin_fmaf(from16<AB>(a.A[k * a.lda + m]), from16<AB>(a.B[k * a.ldb + n]), s);
        red[part][c] = s;
        __syncthreads();
        if (part == 0 && n < a.N) {
#pragma unroll
            for (int q = 1; q < 8; ++q) s += red[q][c];
            sums[m * a.N + n] = s;
        }
        __syncthreads();
    }
}

// ------------------------------------- gradient of bias and activation --
// dp = dy * act'(pre), 16 bits, and the column sums of dp (before its rounding)
// per block of `rows` rows. A workgroup owns 256 columns x `rows` rows: 32
// lanes x 8 columns (16 bytes), 8 rows side by side, so every wave instruction
// reads two whole 512-byte row pieces. Bound by HBM: three arrays of M x N once.
//
// G32: dy is fp32, dp (where it is not null, with any ACT) is rounded once, and
// the column sums are of values that were never rounded. Binary16 holds neither
// the 1e-8 of a mean over a large result nor a gradient past 65504, so dp is
// multiplied there by the power of two that takes the largest |dy| into
// [2^14, 2^15) (no derivative here exceeds 1.13; exact, but for what falls 2^39
// below the largest); `tops` holds ntops maxima of parts of |dy|, `scale`
// receives what undoes the factor after the products. bfloat16 has fp32's range:
// tops is null, the factor 1. dy goes through HBM twice with binary16 (8192 x 8192,
// silu: 150 us, 108 with bfloat16; a cast of dy before the kernel of 16-bit values,
// 155).
__device__ __forceinline__ float largest_exponent_factor(float m, int* shift) {
    int s = m > 0.f ? 15 - __builtin_amdgcn_frexp_expf(m) : 0;
    s = s > 126 ? 126 : s;                            // 2^-s stays normal (s >= 15 - 128)
    *shift = s;
    return ldexpf(1.0f, s);
}

template <int AB, int ACT, bool G32 = false>
__global__ void __launch_bounds__(256)
tgemm_act_grad_kernel(const void* dyv, int64_t lddy, const uint16_t* pre, int64_t ldpre, uint16_t* dp, int64_t lddp,
                      float* part, int M, int N, int rows, const float* tops, int ntops, float* scale) {
    using Dy = std::conditional_t<G32, float, uint16_t>;
    constexpr bool kDp = G32 || ACT != kActNone;
    __shared__ float red[8][32][9];
    const Dy* dy = static_cast<const Dy*>(dyv);
    float up = 1.0f;
    if constexpr (G32) {
        int shift = 0;
        if (tops) {
            __shared__ float rm[4];
            float m = 0.f;
            for (int i = threadIdx.x; i < ntops; i += 256) m = fmaxf(m, tops[i]);
            for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
            if ((threadIdx.x & 63) == 0) rm[threadIdx.x >> 6] = m;
            __syncthreads();
            up = largest_exponent_factor(fmaxf(fmaxf(rm[0], rm[1]), fmaxf(rm[2], rm[3])), &shift);
        }
        if (scale && (blockIdx.x | blockIdx.y | threadIdx.x) == 0) *scale = ldexpf(1.0f, -shift);
    }
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int col = (int)blockIdx.x * 256 + 8 * c;
    const int row0 = (int)blockIdx.y * rows;
    const int n = N - col < 8 ? N - col : 8;          // valid columns (may be <= 0)
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    typedef u32x4 __attribute__((aligned(2))) u32x4u;
    if (n > 0) {
#pragma unroll 4
        for (int q = 0; q < rows / 8; ++q) {
            const int row = row0 + 8 * q + r;
            if (row >= M) break;
            const Dy* gy = dy + (int64_t)row * lddy + col;
            float gv[8];
            u32x4 w{};
            if constexpr (G32) {
                typedef f32x4 __attribute__((aligned(4))) f32x4u;
                if (n == 8) {
                    const f32x4 a = *reinterpret_cast<const f32x4u*>(gy), b = *reinterpret_cast<const f32x4u*>(gy + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        gv[e] = a[e];
                        gv[4 + e] = b[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) gv[e] = e < n ? gy[e] : 0.f;
                }
            } else {
                const u32x4 v = n == 8 ? *reinterpret_cast<const u32x4u*>(gy) : load8_elems(gy, n);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    gv[2 * e] = lo16<AB>(v[e]);
                    gv[2 * e + 1] = hi16<AB>(v[e]);
                }
            }
            if constexpr (ACT != kActNone) {
                const uint16_t* gp = pre + (int64_t)row * ldpre + col;
                w = n == 8 ? *reinterpret_cast<const u32x4u*>(gp) : load8_elems(gp, n);
            }
            u32x4 o{};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo = gv[2 * e], hi = gv[2 * e + 1];
                if constexpr (ACT != kActNone) {
                    lo *= act_grad<ACT>(lo16<AB>(w[e]));
                    hi *= act_grad<ACT>(hi16<AB>(w[e]));
                }
                if constexpr (kDp) o[e] = G32 ? pack2<AB>(lo * up, hi * up) : pack2<AB>(lo, hi);
                s[2 * e] += lo;
                s[2 * e + 1] += hi;
            }
            if (kDp && (!G32 || dp)) {
                uint16_t* go = dp + (int64_t)row * lddp + col;
                if (n == 8) {
                    *reinterpret_cast<u32x4u*>(go) = o;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n) go[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) red[r][c][e] = s[e];
    __syncthreads();
    const int cc = threadIdx.x >> 3, e = threadIdx.x & 7;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += red[q][cc][e];
    const int ccol = (int)blockIdx.x * 256 + 8 * cc + e;
    if (ccol < N) part[(int64_t)blockIdx.y * N + ccol] = t;
}

// The largest finite |dy| of the parts of an fp32 M x N array (G32 above): a
// workgroup takes every gridDim.x-th 256 columns of every gridDim.y-th 8 rows.
// Infinities and NaN do not count: the factor stays that of the other values.
__global__ void __launch_bounds__(256)
tgemm_largest_kernel(const float* dy, int64_t lddy, int M, int N, float* tops) {
    __shared__ float rm[4];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    float m = 0.f;
    auto take = [&](float v) {
        v = __builtin_fabsf(v);
        m = fmaxf(m, v < __builtin_inff() ? v : 0.f);
    };
    for (int64_t row = (int64_t)blockIdx.y * 8 + r; row < M; row += (int64_t)gridDim.y * 8)
        for (int64_t col = (int64_t)blockIdx.x * 256 + 8 * c; col < N; col += (int64_t)gridDim.x * 256) {
            typedef f32x4 __attribute__((aligned(4))) f32x4u;
            const float* p = dy + row * lddy + col;
            if (col + 8 <= N) {
                const f32x4 a = *reinterpret_cast<const f32x4u*>(p), b = *reinterpret_cast<const f32x4u*>(p + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    take(a[e]);
                    take(b[e]);
                }
            } else {
                for (int e = 0; col + e < N; ++e) take(p[e]);
            }
        }
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) rm[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) tops[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = fmaxf(fmaxf(rm[0], rm[1]), fmaxf(rm[2], rm[3]));
}

// Column sums of the row blocks' parts, in row order: four waves take a
// quarter of the blocks each.
template <int AB>
__global__ void __launch_bounds__(256) tgemm_colsum_join_kernel(const float* part, int blocks, int N, void* out, int out_f32) {
    __shared__ float red[4][64];
    const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int per = (blocks + 3) / 4;
    const int b1 = (q + 1) * per < blocks ? (q + 1) * per : blocks;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < N; c0 += (int64_t)gridDim.x * 64) {
        const int64_t col = c0 + c;
        float s = 0.f;
        if (col < N) {
#pragma unroll 8
            for (int b = q * per; b < b1; ++b) s += part[(int64_t)b * N + col];
        }
        red[q][c] = s;
        __syncthreads();
        if (q == 0 && col < N) {
            s = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
            if (out_f32)
                static_cast<float*>(out)[col] = s;
            else
                static_cast<uint16_t*>(out)[col] = to16<AB>(s);
        }
        __syncthreads();
    }
}

// ------------------------------------------------- cross entropy rows --
// lse and loss of each row from its parts: a workgroup joins RW rows, 256 / RW
// threads to a row, whose results meet in LDS by halves (a fixed order). A
// part's weight is exp(m_part - m); parts whose maximum is infinite count as
// they are (their sums are 0 or +inf). RW = 16 reads whole 128-byte lines; few
// rows with thousands of parts take RW = 2 (5 rows of 2048 parts: 39 us with
// RW = 16 in one workgroup). recs, where it is not null: the rows' records of a
// loss gradient of 1 for every row (the scale of a mean is the reduction's).
template <int RW>
__global__ void __launch_bounds__(256)
tgemm_xent_join_kernel(const float2* part, int parts, int rows, const float* zt, const int64_t* target, int64_t V,
                       int64_t ignore, float* lse, float* loss, XentRow* recs) {
    constexpr int kQ = 256 / RW;
    __shared__ float sm[kQ][RW], ss[kQ][RW];
    const int r = threadIdx.x % RW, q = threadIdx.x / RW;
    for (int64_t row0 = (int64_t)blockIdx.x * RW; row0 < rows; row0 += (int64_t)gridDim.x * RW) {
        const int64_t row = row0 + r;
        float m = -__builtin_inff(), s = 0.f;
        auto add = [&](float pm, float ps) {
            const float top = fmaxf(m, pm), f = finite_max(top);
            const float wm = __builtin_fabsf(m) == __builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(kLog2e * (m - f));
            const float wp = __builtin_fabsf(pm) == __builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(kLog2e * (pm - f));
            s = s * wm + ps * wp;
            m = top;
        };
        if (row < rows) {
#pragma unroll 4
            for (int p = q; p < parts; p += kQ) {
                const float2 v = part[(int64_t)p * rows + row];
                add(v.x, v.y);
            }
        }
        sm[q][r] = m;
        ss[q][r] = s;
#pragma unroll
        for (int o = kQ / 2; o; o >>= 1) {
            __syncthreads();
            if (q < o) {
                add(sm[q + o][r], ss[q + o][r]);
                sm[q][r] = m;
                ss[q][r] = s;
            }
        }
        if (q == 0 && row < rows) {
            const float l = finite_max(m) + logf(s);
            lse[row] = l;
            const int64_t t = target[row];
            float v = 0.f;
            const bool live = t != ignore, bad = live && (t < 0 || t >= V);
            if (live) v = bad ? __builtin_nanf("") : l - zt[row];
            loss[row] = v;
            if (recs) {
                XentRow x;
                x.nl2 = -kLog2e * l;
                x.p = bad ? __builtin_nanf("") : (live ? 1.0f : 0.f);
                x.hot = live ? 1.0f : 0.f;
                x.target = live && !bad ? (int)t : -1;
                recs[row] = x;
            }
        }
        __syncthreads();
    }
}

// Sum (mean: divided by the count of rows that are not ignored, at least one) of
// the rows' losses, and that count, in one workgroup and a fixed order. scale,
// where it is not null: the gradient of each row's loss.
__global__ void __launch_bounds__(1024)
tgemm_xent_reduce_kernel(const float* loss, const int64_t* target, int64_t ignore, int rows, int mean, float* out,
                         float* count, float* scale) {
    __shared__ double rs[16];
    __shared__ int rc[16];
    double s = 0.0;
    int n = 0;
    for (int i = threadIdx.x; i < rows; i += 1024) {
        s += (double)loss[i];
        n += target[i] != ignore ? 1 : 0;
    }
    for (int o = 32; o; o >>= 1) {
        s += __shfl_xor(s, o);
        n += __shfl_xor(n, o);
    }
    if ((threadIdx.x & 63) == 0) {
        rs[threadIdx.x >> 6] = s;
        rc[threadIdx.x >> 6] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) {
            s += rs[i];
            n += rc[i];
        }
        const int c = n > 1 ? n : 1;
        *out = (float)(mean ? s / c : s);
        *count = (float)c;
        if (scale) *scale = mean ? 1.0f / (float)c : 1.0f;
    }
}

// The gradient's per-row records. With g the gradient of the row's loss
// (divided by the count for a mean) and e that of its lse, the coefficient of
// column v is (g + e) softmax(z)_v - g [v == target], e softmax(z)_v for an
// ignored row. Everything is divided by the largest of |g|, |g + e| and |e|, so
// that no coefficient exceeds 1, and multiplied by 2^15 with binary16
// coefficients, whose small probabilities would otherwise fall into its
// subnormal range; `scale` undoes both after the products. (With a power of two
// instead, a mean's common factor 1/count stayed a value such as 0.526 that the
// 16 bits round the same way in every row: its error, up to half a step, came
// out whole in both gradients, 0.36% where the rounding of the output is 0.17%.)
// A target outside the vocabulary that is not the ignored label makes the row
// NaN. One workgroup: the largest comes first.
__global__ void __launch_bounds__(1024)
tgemm_xent_rows_kernel(const float* lse, const int64_t* target, int64_t V, int64_t ignore, const float* gloss,
                       int gstride, const float* count, const float* glse, int rows, int shift, XentRow* out,
                       float* scale) {
    __shared__ float rm[16];
    const float inv = count ? 1.0f / *count : 1.0f;
    auto coef = [&](int i, float* p, float* h) {
        const int64_t t = target[i];
        const float g = gloss ? gloss[(int64_t)i * gstride] * inv : 0.f;
        const float e = glse ? glse[i] : 0.f;
        *p = t == ignore ? e : g + e;
        *h = t == ignore ? 0.f : g;
    };
    float m = 0.f;
    for (int i = threadIdx.x; i < rows; i += 1024) {
        float p, h;
        coef(i, &p, &h);
        m = fmaxf(m, fmaxf(fmaxf(__builtin_fabsf(p), __builtin_fabsf(h)), __builtin_fabsf(p - h)));
    }
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) rm[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int i = 0; i < 16; ++i) m = fmaxf(m, rm[i]);
    m = m > 0.f && m < __builtin_inff() ? fmaxf(m, 0x1p-90f) : 1.0f;
    const float up = ldexpf(1.0f / m, shift);
    if (threadIdx.x == 0) *scale = ldexpf(m, -shift);
    for (int i = threadIdx.x; i < rows; i += 1024) {
        const int64_t t = target[i];
        float p, h;
        coef(i, &p, &h);
        const bool bad = t != ignore && (t < 0 || t >= V);
        XentRow r;
        r.nl2 = -kLog2e * lse[i];
        r.p = bad ? __builtin_nanf("") : p * up;
        r.hot = h * up;
        r.target = t == ignore || bad ? -1 : (int)t;
        out[i] = r;
    }
}

// The exponentials of the forward pass become the gradient's coefficients, in
// place: E = exp(z - m) of a 128-column group with maximum m turns into
// p exp(m - lse) E - hot [v == target]. The target's own coefficient is taken
// from its fp32 logit (p - 1 of a probability near 1 would not survive E's 16
// bits); the others are rounded twice, as E and here. A workgroup owns 2048
// columns of 16 rows. Bound by HBM: 4 bytes an element.
template <int AB>
__global__ void __launch_bounds__(256)
tgemm_xent_coef_kernel(uint16_t* G, int64_t ldg, const float2* part, const float* zt, const XentRow* recs, int rows, int V) {
    const int col = (int)blockIdx.y * 2048 + 8 * (int)threadIdx.x;
    if (col >= V) return;
    const int row0 = (int)blockIdx.x * 16;
    const int n = rows - row0 < 16 ? rows - row0 : 16;
    const float2* pt = part + (int64_t)(col >> 7) * rows + row0;
    uint16_t* g = G + (int64_t)row0 * ldg + col;
#pragma unroll 4
    for (int r = 0; r < n; ++r) {
        const XentRow xr = recs[row0 + r];
        const float m = pt[r].x;
        u32x4 v = *reinterpret_cast<const u32x4*>(g + (int64_t)r * ldg);
        const bool dead = xr.p == 0.f && xr.hot == 0.f;
        // (a group of -inf has E = 0 against finite_max = 0, whatever lse is)
        const float f = m == -__builtin_inff() ? xr.p * 0.f
                                               : xr.p * __builtin_amdgcn_exp2f(__builtin_fmaf(kLog2e, finite_max(m), xr.nl2));
        const int rel = xr.target - col;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = dead ? 0u : pack2<AB>(f * lo16<AB>(v[e]), f * hi16<AB>(v[e]));
        if ((unsigned)rel < 8u) {
            const float c = xr.p * __builtin_amdgcn_exp2f(__builtin_fmaf(kLog2e, zt[row0 + r], xr.nl2)) - xr.hot;
            const unsigned b = (unsigned)to16<AB>(c) << (16 * (rel & 1)), keep = 0xffff0000u >> (16 * (rel & 1));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if ((rel >> 1) == e) v[e] = (v[e] & keep) | b;
        }
        *reinterpret_cast<u32x4*>(g + (int64_t)r * ldg) = v;
    }
}

// Two arrays, 16 bits, multiplied by *factor in place; nothing is touched where
// the factor is 1.
template <int AB>
__global__ void __launch_bounds__(256) tgemm_scale_kernel(uint16_t* x0, int64_t n0, uint16_t* x1, int64_t n1, const float* factor) {
    const float f = *factor;
    if (f == 1.0f) return;
    auto run = [&](uint16_t* x, int64_t n) {
        for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
            if (i + 8 <= n) {
                u32x4 v = *reinterpret_cast<const u32x4*>(x + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = pack2<AB>(f * lo16<AB>(v[e]), f * hi16<AB>(v[e]));
                *reinterpret_cast<u32x4*>(x + i) = v;
            } else {
                for (int64_t k = i; k < n; ++k) x[k] = to16<AB>(f * from16<AB>(x[k]));
            }
        }
    };
    run(x0, n0);
    run(x1, n1);
}

}  // namespace tg
