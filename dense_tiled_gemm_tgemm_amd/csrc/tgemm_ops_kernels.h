// Device code of the operators around the product (gfx950): the linear layer
// C = act(alpha * A * B + bias) + residual, the product with a transposed left
// operand, the linear cross entropy (softmax cross entropy of H * W^T without
// keeping the logits) and the small kernels that join their parts.
//
// The large products run on the direct-to-LDS pipeline of tgemm_kernels.h
// (its K loop, LDS layouts, load stream and raster as they are) with another
// end of tile: tgemm_op_kernel below. The accumulators hold C transposed, so
// a lane owns four consecutive columns of one row per 16 x 16 block: a row's
// 128 columns of a wave lie in four lanes (l, l ^ 16, l ^ 32, l ^ 48), and a
// row reduction is 31 in-lane steps and two exchanges.
#pragma once

#include "tgemm_kernels.h"

namespace tg {

// What a tile's sums turn into.
enum : int {
    kEndLin16 = 0,   // linear epilogue, C of the operands' type
    kEndLin32 = 1,   // linear epilogue, fp32 C
    kEndAcc32 = 3,   // fp32 C with an fp32 residual (running sums); also the parts of a split K axis
    kEndXentFwd = 4, // per row: maximum and sum of exponentials of the tile's columns
    kEndXentBwd = 5, // coefficients of the loss gradient, 16 bits
    kEndXentExp = 6  // kEndXentFwd, and the exponentials themselves, 16 bits
};

enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// One row of the cross entropy's gradient: column v's coefficient is
// p * exp2(log2(e) z_v + nl2) - hot * [v == target], zero throughout for an
// ignored row (p == 0 and hot == 0).
struct XentRow {
    float nl2, p, hot;
    int target;
};

struct OpArgs : Args {
    const void* biasv;            // N values of the operands' type or fp32, or null
    int bias_f32;
    const float* alpha_dev;       // null, or a device value alpha is multiplied by
    int act;
    void* pre;                    // null, or M x N of the operands' type: alpha * A * B + bias
    int64_t ldpre;
    const void* res;              // null, or the M x N residual (operands' type; kEndAcc32: fp32)
    int64_t ldres;
    int splits, kper;             // parts of the K axis and k of each (a multiple of 64)
    float2* part;                 // kEndXentFwd, -Exp: [part][row] (maximum, sum of exp(z - finite_max(maximum)))
    float* zt;                    // kEndXentFwd, -Exp: the target's logit per row
    const int64_t* target;
    const XentRow* rows;          // kEndXentBwd
    int v0;                       // kEndXentBwd: vocabulary index of B's row 0
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The normal distribution's lower tail F(-u) = erfc(u / sqrt 2) / 2 =
// exp(-u^2 / 2) t P(t), t = 1 / (1 + 0.375 u / sqrt 2), u >= 0: the factor of the
// exponential is smooth and bounded in t, and P (degree 6) was fitted to it with
// equal relative error over 0 <= u <= 13.4 (6.8e-7; half a step of binary16 is
// 4.9e-4), so the negative tail of gelu keeps its relative accuracy too.
__device__ __forceinline__ float tail_factor(float u) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.375f * 0.7071067811865476f, u, 1.0f));
    float p = 0.5f * -0.13508586034923598f;
    p = __builtin_fmaf(p, t, 0.5f * 0.3879001385194335f);
    p = __builtin_fmaf(p, t, 0.5f * -0.12953986109067597f);
    p = __builtin_fmaf(p, t, 0.5f * 0.28301614073587816f);
    p = __builtin_fmaf(p, t, 0.5f * 0.16668415019859276f);
    p = __builtin_fmaf(p, t, 0.5f * 0.21568481999428807f);
    p = __builtin_fmaf(p, t, 0.5f * 0.21133983897864692f);
    return p * t;
}
// exp(-x^2 / 2)
__device__ __forceinline__ float bell(float x) {
    const float y = 0.8493218002880191f * x;          // sqrt(log2(e) / 2)
    return __builtin_amdgcn_exp2f(-(y * y));
}

// Activations and their derivatives in fp32 (v_exp_f32 and v_rcp_f32, one
// step each); a NaN stays NaN.
//   silu      x s(x), s the logistic function       s (1 + x (1 - s))
//   gelu      x F(x) = max(x, 0) - |x| F(-|x|)     F + x exp(-x^2 / 2) / sqrt(2 pi)
//   gelu_tanh x s(2u), u = sqrt(2/pi)(x + c x^3)    s + x s (1 - s) 2 u'
// (x/2 (1 + tanh u) = x s(2u)).
template <int ACT>
__device__ __forceinline__ float act_fwd(float x) {
    if constexpr (ACT == kActRelu) {
        return x < 0.f ? 0.f : x;
    } else if constexpr (ACT == kActSilu) {
        return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
    } else if constexpr (ACT == kActGelu) {
        // (the bound keeps infinity times a vanished tail at zero; a NaN comes back through the bell)
        const float u = __builtin_fminf(__builtin_fabsf(x), 1e30f);
        const float h = tail_factor(u) * bell(x);
        return __builtin_fmaf(-u, h, __builtin_fmaxf(x, 0.f));
    } else if constexpr (ACT == kActGeluTanh) {
        const float u2 = x * __builtin_fmaf(2.0f * 0.7978845608028654f * 0.044715f, x * x, 2.0f * 0.7978845608028654f);
        return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * u2));
    } else {
        return x;
    }
}

// The derivatives are 0 below -1000 and 1 above 1000 in fp32, and are taken
// there: a pre-activation past 65504 is kept as an infinity in binary16, and the
// square of one past 1.8e19 is one in bfloat16, where 0 * inf would come out.
template <int ACT>
__device__ __forceinline__ float act_grad(float x) {
    if constexpr (ACT == kActSilu || ACT == kActGelu || ACT == kActGeluTanh)
        x = __builtin_fabsf(x) > 1000.0f ? __builtin_copysignf(1000.0f, x) : x;   // (a NaN stays)
    if constexpr (ACT == kActRelu) {
        return x > 0.f ? 1.0f : (x <= 0.f ? 0.f : x);
    } else if constexpr (ACT == kActSilu) {
        // far below zero exp2 overflows and s and s x both vanish
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
        return s * __builtin_fmaf(x, 1.0f - s, 1.0f);
    } else if constexpr (ACT == kActGelu) {
        const float e = bell(x);
        const float h = tail_factor(__builtin_fabsf(x)) * e;
        return __builtin_fmaf(x, 0.3989422804014327f * e, x < 0.f ? h : 1.0f - h);
    } else if constexpr (ACT == kActGeluTanh) {
        const float x2 = x * x;
        const float u2 = x * __builtin_fmaf(2.0f * 0.7978845608028654f * 0.044715f, x2, 2.0f * 0.7978845608028654f);
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * u2));
        const float du = __builtin_fmaf(6.0f * 0.7978845608028654f * 0.044715f, x2, 2.0f * 0.7978845608028654f);
        return __builtin_fmaf(x * s * (1.0f - s), du, s);
    } else {
        return 1.0f;
    }
}

// 16 bits (AB: 0 binary16, 1 bfloat16) to fp32; lo / hi half of a word.
template <int AB>
__device__ __forceinline__ float from16(uint16_t b) {
    if constexpr (AB == 0)
        return (float)__builtin_bit_cast(_Float16, b);
    else
        return __builtin_bit_cast(float, (unsigned)b << 16);
}
template <int AB>
__device__ __forceinline__ float lo16(unsigned w) { return from16<AB>((uint16_t)w); }
template <int AB>
__device__ __forceinline__ float hi16(unsigned w) { return from16<AB>((uint16_t)(w >> 16)); }

// Element i of an array of the operands' type or fp32.
template <int AB>
__device__ __forceinline__ float load_elem(const void* p, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : from16<AB>(static_cast<const uint16_t*>(p)[i]);
}

template <int AB>
__device__ __forceinline__ uint16_t to16(float v) { return (uint16_t)pack2<AB>(v, 0.f); }

// ------------------------------------------------------------ stores --
// Where a wave's 16-byte pieces go in an M x N array of 16-bit or fp32
// elements: the resource starts at the wave's first row, `lane` is the lane's
// byte offset (row rl of the block's 8, its first column), `ld8` the bytes of 8
// rows. Offsets stay below 2^31 (host stride limit).
struct Dest {
    BufRsrc rs;
    char* base;                 // first byte of the wave's first row
    unsigned lane;
    int ld8;
};

__device__ __forceinline__ Dest dest(void* p, int64_t ld, int es, int mrow, int rl, int col) {
    Dest d;
    d.base = static_cast<char*>(p) + (int64_t)mrow * ld * es;
    d.rs = c_rows_rsrc(d.base, 0);
    d.lane = (unsigned)rl * (unsigned)(ld * es) + (unsigned)col * (unsigned)es;
    d.ld8 = (int)(ld * es * 8);
    return d;
}

// The pieces d[0], d[1] of rows rl and rl + 8 of 16-row block i (as store_c of
// tgemm_kernels.h leaves them), columns col .. of the row; `cb` is the
// column's byte distance from the lane's first. `roff` (the block's byte
// offset) is uniform and rides in the scalar offset.
template <int ES>
__device__ __forceinline__ void store_pieces(const u32x4 (&d)[2], const Dest& t, int rows_left, int N, int roff, int col,
                                             int cb, bool whole, bool stream) {
    constexpr int kN = 16 / ES;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool rok = 8 * h < rows_left;           // rows_left: M minus the lane's row of the block's first 8
        const bool ok16 = rok & (col + kN <= N);
        unsigned o = ok16 ? t.lane + (unsigned)cb : kCOob;
        asm volatile("" : "+v"(o));
        const int so = roff + h * t.ld8;
#if defined(__HIP_DEVICE_COMPILE__)
        if (stream)
            __builtin_amdgcn_raw_buffer_store_b128(d[h], t.rs, (int)o, so, kCStorePolicy);
        else
            __builtin_amdgcn_raw_buffer_store_b128(d[h], t.rs, (int)o, so, 0);
#endif
        if (__builtin_expect(!whole, 0)) {
            asm volatile("");
            if (!ok16 && rok && col < N) {
                char* dst = t.base + (unsigned)so + (t.lane + (unsigned)cb);
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    if (col + e < N) {
                        if constexpr (ES == 4)
                            reinterpret_cast<unsigned*>(dst)[e] = d[h][e];
                        else
                            reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(d[h][e >> 1] >> (16 * (e & 1)));
                    }
            }
        }
    }
}

// Trade of 16-byte pieces between lanes l and l + 8 of each 16-lane row.
__device__ __forceinline__ void trade8(u32x4 (&d)[2], const u32x4 (&vs)[2], bool hi) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const unsigned u = hi ? vs[0][e] : vs[1][e];
        const unsigned w = (unsigned)__builtin_amdgcn_mov_dpp((int)u, 0x128, 0xf, 0xf, false);
        d[0][e] = hi ? w : vs[0][e];
        d[1][e] = hi ? vs[1][e] : w;
    }
}

// Two blocks' four columns each, 16 bits, as the 8 consecutive columns that
// the lane stores.
template <int AB>
__device__ __forceinline__ u32x4 swap_pack(const f32x4& x, const f32x4& y) {
    const auto s0 = __builtin_amdgcn_permlane16_swap(pack2<AB>(x[0], x[1]), pack2<AB>(y[0], y[1]), false, false);
    const auto s1 = __builtin_amdgcn_permlane16_swap(pack2<AB>(x[2], x[3]), pack2<AB>(y[2], y[3]), false, false);
    return u32x4{s0[0], s1[0], s0[1], s1[1]};
}

// Four consecutive values col .. col + 3 of a row vector of N >= 4 elements
// (bias), without a branch: a lane whose columns straddle N reads the four that
// end at N and shifts them down, one past N reads zeros, so no byte outside the
// array is touched. Any element alignment.
template <int AB, bool F32>
__device__ __forceinline__ f32x4 load_row4(const BufRsrc& rs, int col, int N) {
    f32x4 v{};
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr unsigned kEs = F32 ? 4 : 2;
    const int c = col <= N - 4 ? col : N - 4;
    const unsigned o = col < N ? (unsigned)c * kEs : kCOob;
    const int sh = col - c;
    if constexpr (F32) {
        const f32x4 w = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)o, 0, 0));
        v[0] = sh <= 0 ? w[0] : (sh == 1 ? w[1] : (sh == 2 ? w[2] : w[3]));
        v[1] = sh <= 0 ? w[1] : (sh == 1 ? w[2] : w[3]);
        v[2] = sh <= 0 ? w[2] : w[3];
        v[3] = w[3];
    } else {
        const uint64_t w = __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(rs, (int)o, 0, 0)) >>
                           (16 * (sh & 3));
        v = f32x4{lo16<AB>((unsigned)w), hi16<AB>((unsigned)w), lo16<AB>((unsigned)(w >> 32)), hi16<AB>((unsigned)(w >> 32))};
    }
#endif
    return v;
}

// The residual as the 16-byte pieces that the stores write (store_pieces' rows
// and columns; whole 128-byte row pieces per instruction, where a lane's own
// four columns would take 32 bytes of sixteen rows). A lane outside M x N
// presents an offset past the range and reads zeros; one whose columns straddle
// N reads those that end at N (the host keeps N >= 8 here), which shift_piece
// moves down when they are used.
template <int ES>
__device__ __forceinline__ void load_pieces(u32x4 (&d)[2], const Dest& t, int rows_left, int N, int roff, int col, int cb) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int kN = 16 / ES;
    const int over = col > N - kN ? col - (N - kN) : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        unsigned o = (8 * h < rows_left && col < N) ? t.lane + (unsigned)cb - (unsigned)(over * ES) : kCOob;
        asm volatile("" : "+v"(o));
        d[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(t.rs, (int)o, roff + h * t.ld8, 0));
    }
#endif
}

// A piece that was read `over` elements early (over > 7: no column, zeros).
template <int ES>
__device__ __forceinline__ u32x4 shift_piece(u32x4 v, int over) {
    const int b = over * ES;                          // bytes
    if (b & 8) v = u32x4{v[2], v[3], 0u, 0u};
    if (b & 4) v = u32x4{v[1], v[2], v[3], 0u};
    if (b & 2) v = u32x4{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16), v[3] >> 16};
    return v;
}

// End of a tile of the linear layer: v = alpha * sum + bias (one rounding),
// optionally stored as `pre`, then act(v) + residual, rounded once to C's type.
// RF32: the residual is fp32 (running sums; without `pre`).
// The residual arrives in the store's layout and takes the store's exchanges
// backwards (both are their own inverses); its loads run kAhead 16-row blocks
// before their use, so the memory latency is met about once per tile and not
// once per block.
// In-place use (C is the residual) is safe: a lane stores the very pieces it
// has loaded, after it has used them.
// MORE: there is a residual or `pre` (tested per use); POL: C's store policy
// (1 streamed, 0 default, -1 by a.c_stream). end_tile picks the copy once per
// tile: with every test inside one copy the plain layer's end of tile had twice
// the branches.
template <int AB, bool C32, bool RF32, int ACT, bool MORE, int POL, int NI>
__device__ __forceinline__ void end_linear(const f32x4 (&acc)[NI][8], const OpArgs& a, int m0, int n0, int wm, int wn,
                                           int lane) {
    constexpr int kWr = 16 * NI;
    constexpr int kEs = C32 ? 4 : 2;
    constexpr int kRes = RF32 ? 4 : 2;
    constexpr int kNp = RF32 ? 4 : 2;                 // pairs of pieces in a 16-row block of the residual
    constexpr int kAhead = (RF32 || NI <= 4) ? 2 : 4;
    const int r16 = lane & 15, g = lane >> 4;
    const int mrow = m0 + wm * kWr, ncol = n0 + wn * 128;
    const bool hi = r16 >= 8;
    const int rl = r16 & 7;
    const int col16 = ncol + (g & 1) * 16 + (g >> 1) * 8 + (hi ? 32 : 0);
    const int col32 = ncol + 4 * g + (hi ? 16 : 0);
    const int colc = C32 ? col32 : col16;
    const int colr = RF32 ? col32 : col16;
    const bool has_res = MORE && a.res != nullptr, has_pre = MORE && !RF32 && a.pre != nullptr;
    const bool whole = __builtin_amdgcn_readfirstlane((int)(mrow + kWr <= a.M && ncol + 128 <= a.N)) != 0;
    const bool edge = __builtin_amdgcn_readfirstlane((int)(ncol + 128 > a.N)) != 0;
    const bool stream = POL < 0 ? __builtin_amdgcn_readfirstlane(a.c_stream) != 0 : POL == 1;
    u32x4 rp[NI][kNp][2];
    const Dest dr = dest(const_cast<void*>(a.res), a.ldres, kRes, mrow, rl, colr);
    auto request = [&](int i, int rb) {
#pragma unroll
        for (int q = 0; q < kNp; ++q)
            load_pieces<kRes>(rp[i][q], dr, a.M - mrow - 16 * rb - rl, a.N, 2 * rb * dr.ld8, colr + (128 / kNp) * q,
                              (128 / kNp) * kRes * q);
    };
    if (has_res) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) request(i, i);
    }
    const Dest dc = dest(a.C, a.ldc, kEs, mrow, rl, colc);
    Dest dp;
    if constexpr (!RF32) dp = dest(a.pre, a.ldpre, 2, mrow, rl, col16);
    float alpha = a.alpha;
    if (a.alpha_dev) alpha *= *a.alpha_dev;
    f32x4 bv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) bv[j] = f32x4{};
    if (a.biasv) {
        const BufRsrc brs = c_rows_rsrc(const_cast<void*>(a.biasv), 0);
        if (a.bias_f32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) bv[j] = load_row4<AB, true>(brs, ncol + 16 * j + 4 * g, a.N);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) bv[j] = load_row4<AB, false>(brs, ncol + 16 * j + 4 * g, a.N);
        }
    }
    int rb = 0;                                       // 16-row block (uniform; opaque, so that no offset is hoisted)
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+s"(rb));
        const int rows_left = a.M - mrow - 16 * rb - rl;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            f32x4 v[4], rv[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) rv[b] = f32x4{};
            if (has_res) {
#pragma unroll
                for (int p = 0; p < kNp / 2; ++p) {
                    const int qq = q * (kNp / 2) + p;
                    u32x4 d[2] = {rp[i][qq][0], rp[i][qq][1]}, vs[2];
                    if (__builtin_expect(edge, 0)) {
                        const int c = colr + (128 / kNp) * qq, over = c - (a.N - 16 / kRes);
#pragma unroll
                        for (int h = 0; h < 2; ++h) d[h] = shift_piece<kRes>(d[h], over > 0 ? over : 0);
                    }
                    trade8(vs, d, hi);
                    if constexpr (RF32) {
                        rv[2 * p] = __builtin_bit_cast(f32x4, vs[0]);
                        rv[2 * p + 1] = __builtin_bit_cast(f32x4, vs[1]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const auto s0 = __builtin_amdgcn_permlane16_swap(vs[h][0], vs[h][2], false, false);
                            const auto s1 = __builtin_amdgcn_permlane16_swap(vs[h][1], vs[h][3], false, false);
                            rv[2 * h] = f32x4{lo16<AB>(s0[0]), hi16<AB>(s0[0]), lo16<AB>(s1[0]), hi16<AB>(s1[0])};
                            rv[2 * h + 1] = f32x4{lo16<AB>(s0[1]), hi16<AB>(s0[1]), lo16<AB>(s1[1]), hi16<AB>(s1[1])};
                        }
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int j = 4 * q + b;
                f32x4 x = acc[i][j];
                asm volatile("" : "+v"(x));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[b][e] = __builtin_fmaf(alpha, x[e], bv[j][e]);
            }
            if (has_pre) {
                u32x4 vs[2] = {swap_pack<AB>(v[0], v[1]), swap_pack<AB>(v[2], v[3])};
                u32x4 d[2];
                trade8(d, vs, hi);
                store_pieces<2>(d, dp, rows_left, a.N, 2 * rb * dp.ld8, col16 + 64 * q, 128 * q, whole, stream);
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[b][e] = act_fwd<ACT>(v[b][e]) + rv[b][e];
            if constexpr (C32) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    u32x4 vs[2] = {__builtin_bit_cast(u32x4, v[2 * p]), __builtin_bit_cast(u32x4, v[2 * p + 1])};
                    u32x4 d[2];
                    trade8(d, vs, hi);
                    const int qq = 2 * q + p;
                    store_pieces<4>(d, dc, rows_left, a.N, 2 * rb * dc.ld8, col32 + 32 * qq, 128 * qq, whole, stream);
                }
            } else {
                u32x4 vs[2] = {swap_pack<AB>(v[0], v[1]), swap_pack<AB>(v[2], v[3])};
                u32x4 d[2];
                trade8(d, vs, hi);
                store_pieces<2>(d, dc, rows_left, a.N, 2 * rb * dc.ld8, col16 + 64 * q, 128 * q, whole, stream);
            }
        }
        if (i + kAhead < NI) {
            if (has_res) request(i + kAhead < NI ? i + kAhead : 0, rb + kAhead);
        }
        ++rb;
    }
}

// Maximum / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max4g(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const float m = fmaxf(__builtin_bit_cast(float, (unsigned)s[0]), __builtin_bit_cast(float, (unsigned)s[1]));
    const unsigned w = __builtin_bit_cast(unsigned, m);
    const auto t = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return fmaxf(__builtin_bit_cast(float, (unsigned)t[0]), __builtin_bit_cast(float, (unsigned)t[1]));
}
__device__ __forceinline__ float sum4g(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const float m = __builtin_bit_cast(float, (unsigned)s[0]) + __builtin_bit_cast(float, (unsigned)s[1]);
    const unsigned w = __builtin_bit_cast(unsigned, m);
    const auto t = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return __builtin_bit_cast(float, (unsigned)t[0]) + __builtin_bit_cast(float, (unsigned)t[1]);
}

// A maximum that exponentials can be taken against: of a row of -inf, or one
// that holds +inf, the differences would be NaN; against zero their
// exponentials are 0 and +inf, whose logarithms are what the row has.
__device__ __forceinline__ float finite_max(float m) { return __builtin_fabsf(m) == __builtin_inff() ? 0.f : m; }

// End of a tile of the cross entropy's forward pass: per row of the wave's
// 128 columns the maximum m and the sum of exp(z - m), and the target's logit
// where it lies here. Columns at or past N count as -inf. EXP: the exponentials
// also go to C, rounded to 16 bits (their sum is taken before).
template <int AB, bool EXP, int NI>
__device__ __forceinline__ void end_xent_fwd(const f32x4 (&acc)[NI][8], const OpArgs& a, int m0, int n0, int wm, int wn,
                                             int lane) {
    constexpr int kWr = 16 * NI;
    const int r16 = lane & 15, g = lane >> 4;
    const int mrow = m0 + wm * kWr, ncol = n0 + wn * 128;
    const bool inside = __builtin_amdgcn_readfirstlane((int)(ncol + 128 <= a.N)) != 0;
    const bool whole = __builtin_amdgcn_readfirstlane((int)(mrow + kWr <= a.M && ncol + 128 <= a.N)) != 0;
    const bool stream = EXP && __builtin_amdgcn_readfirstlane(a.c_stream) != 0;
    if (ncol >= a.N) return;                          // uniform: the group has no column
    float2* part = a.part + (int64_t)(ncol >> 7) * a.M;
    const bool hi = r16 >= 8;
    const int rl = r16 & 7;
    const int col16 = ncol + (g & 1) * 16 + (g >> 1) * 8 + (hi ? 32 : 0);
    Dest dc;
    if constexpr (EXP) dc = dest(a.C, a.ldc, 2, mrow, rl, col16);
    int rb = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+s"(rb));
        const int row = mrow + 16 * rb + r16;
        f32x4 z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[j] = acc[i][j];
            asm volatile("" : "+v"(z[j]));
        }
        const int64_t t = row < a.M ? a.target[row] : -1;
        const int64_t rel = t - ncol;
        if (rel >= 0 && rel < 128 && t < a.N && (((int)rel >> 2) & 3) == g) {
            float zt = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((int)rel == 16 * j + 4 * g + e) zt = z[j][e];
            a.zt[row] = zt;
        }
        if (!inside) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (ncol + 16 * j + 4 * g + e >= a.N) z[j][e] = -__builtin_inff();
        }
        float m = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[0][2], z[0][3]));
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, fmaxf(fmaxf(z[j][0], z[j][1]), fmaxf(z[j][2], z[j][3])));
        m = max4g(m);
        const float nm2 = -kLog2e * finite_max(m);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[j][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(kLog2e, z[j][e], nm2));
                s[e] += z[j][e];
            }
        const float sum = sum4g((s[0] + s[1]) + (s[2] + s[3]));
        if (g == 0 && row < a.M) part[row] = float2{m, sum};
        if constexpr (EXP) {
            const int rows_left = a.M - mrow - 16 * rb - rl;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                u32x4 vs[2] = {swap_pack<AB>(z[4 * q], z[4 * q + 1]), swap_pack<AB>(z[4 * q + 2], z[4 * q + 3])};
                u32x4 d[2];
                trade8(d, vs, hi);
                store_pieces<2>(d, dc, rows_left, a.N, 2 * rb * dc.ld8, col16 + 64 * q, 128 * q, whole, stream);
            }
        }
        ++rb;
    }
}

// End of a tile of the cross entropy's backward pass: the recomputed logits
// become the gradient's coefficients, 16 bits, in C (one piece of the
// vocabulary).
template <int AB, int NI>
__device__ __forceinline__ void end_xent_bwd(const f32x4 (&acc)[NI][8], const OpArgs& a, int m0, int n0, int wm, int wn,
                                             int lane) {
    constexpr int kWr = 16 * NI;
    const int r16 = lane & 15, g = lane >> 4;
    const int mrow = m0 + wm * kWr, ncol = n0 + wn * 128;
    const bool whole = __builtin_amdgcn_readfirstlane((int)(mrow + kWr <= a.M && ncol + 128 <= a.N)) != 0;
    const bool hi = r16 >= 8;
    const int rl = r16 & 7;
    const int col16 = ncol + (g & 1) * 16 + (g >> 1) * 8 + (hi ? 32 : 0);
    const Dest dc = dest(a.C, a.ldc, 2, mrow, rl, col16);
    int rb = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+s"(rb));
        const int row = mrow + 16 * rb + r16;
        const int rows_left = a.M - mrow - 16 * rb - rl;
        const XentRow xr = a.rows[row < a.M ? row : a.M - 1];
        const int rel = xr.target - a.v0 - ncol - 4 * g;
        const bool dead = xr.p == 0.f && xr.hot == 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            f32x4 v[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int j = 4 * q + b;
                f32x4 x = acc[i][j];
                asm volatile("" : "+v"(x));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[b][e] = dead ? 0.f : xr.p * __builtin_amdgcn_exp2f(__builtin_fmaf(kLog2e, x[e], xr.nl2));
            }
            if ((unsigned)(rel - 64 * q) < 64u) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (rel == 64 * q + 16 * b + e) v[b][e] -= xr.hot;
            }
            u32x4 vs[2] = {swap_pack<AB>(v[0], v[1]), swap_pack<AB>(v[2], v[3])};
            u32x4 d[2];
            trade8(d, vs, hi);
            store_pieces<2>(d, dc, rows_left, a.N, 2 * rb * dc.ld8, col16 + 64 * q, 128 * q, whole, false);
        }
        ++rb;
    }
}

template <int AB, int END, int ACT, int NI>
__device__ __forceinline__ void end_tile(const f32x4 (&acc)[NI][8], const OpArgs& a, int m0, int n0, int wm, int wn,
                                         int lane) {
    if constexpr (END == kEndXentFwd || END == kEndXentExp) {
        end_xent_fwd<AB, END == kEndXentExp, NI>(acc, a, m0, n0, wm, wn, lane);
    } else if constexpr (END == kEndXentBwd) {
        end_xent_bwd<AB, NI>(acc, a, m0, n0, wm, wn, lane);
    } else {
        constexpr bool kC32 = END != kEndLin16, kR32 = END == kEndAcc32;
        if constexpr (NI < 8) {
            end_linear<AB, kC32, kR32, ACT, true, -1, NI>(acc, a, m0, n0, wm, wn, lane);
        } else if (a.res || (!kR32 && a.pre)) {
            end_linear<AB, kC32, kR32, ACT, true, -1, NI>(acc, a, m0, n0, wm, wn, lane);
        } else if (a.c_stream && !kR32) {
            end_linear<AB, kC32, kR32, ACT, false, 1, NI>(acc, a, m0, n0, wm, wn, lane);
        } else {
            end_linear<AB, kC32, kR32, ACT, false, 0, NI>(acc, a, m0, n0, wm, wn, lane);
        }
    }
}

// The direct-to-LDS tile kernel (tgemm_dma_kernel: same K loop, load stream,
// wait counts and tile walk) with an operator's end of tile. AKM: A is stored
// K x M, so C = A^T B over both operands' rows. A tile changes every nk steps
// without draining the load stream; inside a tile the stream is kept by
// additions (StepCursor; 8192 x 4096 x 8192 in bfloat16: 389 -> 372 us for a B
// stored K x N, 397 -> 377 for A^T B, whose steps spent 80 of 330 instructions
// on 64-bit products and comparisons). 256-row tiles are bound by the matrix
// cores at the clock the card's power leaves them (8192^3: 1623 TFLOP/s, the
// library product 1632), 128- and 64-row ones by LDS traffic, 40 KiB a step
// and compute unit at 64 rows. kEndAcc32 with splits > 1
// (grid W * splits): a workgroup computes one part of the K axis of one tile,
// into that part of C (splits arrays of M x ldc, one after another).
template <int AB, int NXK, int AKM, int KS, int S, int I, int END, int ACT = kActNone>
__global__ void __launch_bounds__(NTHREADS)
__attribute__((amdgpu_waves_per_eu(I == 8 || KS == 64 ? 1 : 2, I == 8 || KS == 64 ? 1 : 2)))
tgemm_op_kernel(OpArgs a) {
    using Ctx = DmaCtx<KS, NXK, S, I>;
    static_assert(KS == 64 || KS == 32, "K step");
    static_assert(KS == 32 || S == 2 || I < 8, "64-deep steps of 256-row tiles use a 2-stage ring");
    static_assert(I == 8 || KS == 64 || Ctx::kSlots * 16 <= 80 * 1024, "two workgroups per compute unit");
    constexpr int kL = Ctx::kLa + KS / 8;
    constexpr int kBm = 32 * I;
    __shared__ u32x4 smem[Ctx::kSlots];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int wid = (int)blockIdx.x;
    if constexpr (END == kEndAcc32) {
        if (a.splits > 1) {
            // each die takes one contiguous range of (part, tile), so that the
            // tiles it runs side by side share panels of the same part (as the
            // raster's first step does for the tiles of a product in one part)
            const int total = a.W * a.splits, x = wid % a.num_xcd, i = wid / a.num_xcd;
            const int q = total / a.num_xcd, r = total % a.num_xcd;
            wid = x < r ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;
            a.num_xcd = 1;
            const int s = wid / a.W;
            wid -= s * a.W;
            const int k0 = s * a.kper;
            a.A += AKM ? (int64_t)k0 * a.lda : (int64_t)k0;
            a.B += NXK ? (int64_t)k0 : (int64_t)k0 * a.ldb;
            a.K = a.K - k0 < a.kper ? a.K - k0 : a.kper;
            const int64_t part = (int64_t)s * a.M * a.ldc;
            a.C = static_cast<float*>(a.C) + part;
            if (a.res) a.res = static_cast<const float*>(a.res) + part;
        }
    }
    const int nkd = (a.K + KS - 1) / KS;
    const int lead = KS == 32 ? (nkd & 1) : 0;
    const int nk = nkd + lead;

    Tile tc = make_tile<NXK, kBm, AB, AKM>(a, wid);
    bool has_next = wid + a.grid < a.W;
    Tile tn = has_next ? make_tile<NXK, kBm, AB, AKM>(a, wid + a.grid) : tc;
    f32x4 acc[I][8];
    if (KS == 32) zero_acc_mma<AB, I>(acc);

    Ctx c;
    c.p = lane_loads<KS, NXK, Ctx::kLa, AB, AKM>(a, tid);
    c.bstep = (unsigned)(KS * 2);
    c.nk = nk;
    c.lead = lead;
    c.klast = (nkd - 1) * KS;
    c.fixup = (a.K % KS) != 0 || (!NXK && (a.N % 8) != 0) || (AKM && (a.M % 8) != 0);
    c.tid = tid;
    c.wave = wave;
    c.lane = lane;
    c.smem = smem;
    c.fp = frag_ptrs<KS, NXK, I, AB, AKM>(c.a_blk(0), c.b_blk(0), wm, wn, lane);
    half8 fa[2][I], fb[2][8];
    for (int t = 0; t < S; ++t) {
        const int d = t - lead;
        const bool live = d >= 0 && t < nk;
        for (int idx = 0; idx < kL; ++idx)
            issue_load<KS, NXK>(a_step_rsrc<KS, AKM>(tc, live ? d : 0, a.lda),
                                b_step_rsrc<KS, NXK, AB>(tc, live ? d : 0, a.ldb), c.p, idx,
                                live ? (AKM ? 0u : (unsigned)d * (unsigned)(KS * 2)) : kOob,
                                live ? (NXK ? (unsigned)d * c.bstep : 0u) : kOob, c.a_blk(t), c.b_blk(t), wave);
    }
    wait_vmcnt<(S - 1) * kL>();
    if (c.fixup && nk == 1)
        fix_last_step<KS, NXK, Ctx::kLa, AB, AKM>(c.a_blk(0), c.b_blk(0), c.p, a, tc.m0, tc.n0, c.klast, tid, wave, lane);
    block_barrier();
    read_frags<KS, NXK, I, AB, AKM>(fa[0], fb[0], c.fp, 0);
    FragPtrs<KS, NXK> cur = c.fp;
    if constexpr (KS == 64) {
        int st = 0;
        auto next = [&] { st = S == 2 ? st ^ 1 : (st + 1 == S ? 0 : st + 1); };
        for (;;) {
            dma_step<AB, NXK, KS, S, 0, true, false, I, false, AKM>(acc, fa, fb, st, 0, a, c, cur, tc, tn, has_next);
            next();
            if constexpr (S == 2) {
                if (nk > 2) {
                    StepCursor<KS, NXK, AKM> mid;
                    mid.set(tc, 1 + S, a.lda, a.ldb);
                    for (int t = 1; t + S < nk; ++t) {
                        dma_step<AB, NXK, KS, S, 0, false, false, I, false, AKM, true>(acc, fa, fb, st, t, a, c, cur, tc, tn,
                                                                                       has_next, &mid);
                        next();
                    }
                    dma_step<AB, NXK, KS, S, 0, false, false, I, false, AKM>(acc, fa, fb, st, nk - 2, a, c, cur, tc, tn,
                                                                             has_next);
                    next();
                }
            } else {
                int t = 1;
                if (nk > S) {
                    StepCursor<KS, NXK, AKM> mid;
                    mid.set(tc, 1 + S, a.lda, a.ldb);
                    for (; t + S < nk; ++t) {
                        dma_step<AB, NXK, KS, S, 0, false, false, I, false, AKM, true>(acc, fa, fb, st, t, a, c, cur, tc, tn,
                                                                                       has_next, &mid);
                        next();
                    }
                }
                for (; t + 1 < nk; ++t) {
                    dma_step<AB, NXK, KS, S, 0, false, false, I, false, AKM>(acc, fa, fb, st, t, a, c, cur, tc, tn, has_next);
                    next();
                }
            }
            dma_step<AB, NXK, KS, S, 0, false, true, I, false, AKM>(acc, fa, fb, st, nk - 1, a, c, cur, tc, tn, has_next);
            next();
            end_tile<AB, END, ACT, I>(acc, a, tc.m0, tc.n0, wm, wn, lane);
            if (!has_next) break;
            read_frags<KS, NXK, I, AB, AKM>(fa[0], fb[0], cur, 0);
            wid += a.grid;
            tc = tn;
            has_next = wid + a.grid < a.W;
            if (has_next) tn = make_tile<NXK, kBm, AB, AKM>(a, wid + a.grid);
        }
    } else {
        step_pairs<AB, NXK, S, I, false, AKM>(acc, fa, fb, a, c, cur, tc);
        end_tile<AB, END, ACT, I>(acc, a, tc.m0, tc.n0, wm, wn, lane);
    }
    wait_vmcnt<0>();
}


// The tile kernel for an operand type, an end of tile, an activation (the
// linear ends), B's and A's layout, tile rows and K step, or null where the
// combination is not built. Each (type, end, activation) is instantiated in a
// translation unit of its own.
template <int AB, int END, int ACT>
const void* op_kernel(int nxk, int akm, int tile_m, int k_step);

}  // namespace tg
