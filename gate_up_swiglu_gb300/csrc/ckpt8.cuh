// ckpt8.cuh -- device code of the 8-bit activation checkpoint: e4m3 codes with
// one power-of-two scale per block of 32 columns (the format of swiglu_moe.h).
#pragma once

#include <stdint.h>

#include "swiglu_kernels.cuh"

namespace ckpt8 {

constexpr int kBlock = 32;

// Largest finite |v| of a thread's values.  fmaxf drops NaN; infinities are
// rare enough to be looked for only once one has turned up.
template <int N>
__device__ __forceinline__ float finite_amax(const float *v) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
    if (m == INFINITY) {
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]) == INFINITY ? 0.0f : fabsf(v[i]));
    }
    return m;
}

// The smallest code c >= 0 with amax <= 448 * 2^(c - 127), 448 = 1.75 * 2^8:
// with amax = m 2^k (1 <= m < 2), c = k - 8 + 127, one more when m > 1.75.
// Adding 0x1fffff to the bits carries into the exponent exactly for mantissas
// above .75.
__device__ __forceinline__ uint32_t scale_code(float amax) {
    const int c = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;
    return (uint32_t)max(c, 0);
}

// 2^(127 - c) and 2^(c - 127), exact (c <= 247; 2^-127 is a subnormal).
__device__ __forceinline__ float encode_factor(uint32_t c) { return __uint_as_float((254u - c) << 23); }
__device__ __forceinline__ float decode_factor(uint32_t c) {
    return __uint_as_float(c == 0 ? 1u << 22 : c << 23);
}

// Two values to e4m3, nearest even; `lo` in the low byte.  The conversion
// saturates, so an infinity is made a NaN first (finite values of a block are
// at most 448 after scaling).
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    unsigned short h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
    return h;
}

// N values (N = 1 or a multiple of 2) scaled by `f` to N codes.  The largest
// values of fp32 would round up to 256 * 2^120 = 2^128, which fp32 cannot hold:
// they keep the code of 240.  One test of the largest value tells whether any
// of this, or an infinity, has to be looked at; kCare: it has.
template <int N, bool kCare>
__device__ __forceinline__ void encode_values(const float *v, float f, uint32_t *out) {
    const float top = f == 7.52316384526264e-37f ? 240.0f : 448.0f;  // 2^-120: the largest scale
    const auto one = [&](int i) {
        float t = __fmul_rn(v[i], f);
        if (kCare)
            t = fabsf(v[i]) == INFINITY ? __uint_as_float(0x7fc00000u) : t > top ? top : t < -top ? -top : t;
        return t;
    };
    if (N == 1) {
        out[0] = codes2(one(0), 0.0f) & 0xffu;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint32_t h = codes2(one(i), one(i + 1));
            if (i % 4 == 0)
                out[i / 4] = h;
            else
                out[i / 4] |= h << 16;
        }
    }
}

template <int N>
__device__ __forceinline__ void encode(const float *v, float f, uint32_t *out) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
    if (m <= 2.97747071e38f)  // 1.75 * 2^127
        encode_values<N, false>(v, f, out);
    else
        encode_values<N, true>(v, f, out);
}

// N codes to the values they stand for (e4m3 is exact in fp16 and fp32).
template <int N>
__device__ __forceinline__ void decode(const uint32_t *q, float f, float *v) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const unsigned short h = (unsigned short)(q[i / 4] >> (i % 4 * 8));
        uint32_t pair;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(pair) : "h"(h));
        float lo, hi;
        asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}\n"
            : "=f"(lo), "=f"(hi)
            : "r"(pair));
        v[i] = __fmul_rn(lo, f);
        if (i + 1 < N) v[i + 1] = __fmul_rn(hi, f);
    }
}

// VEC codes.
template <int VEC>
__device__ __forceinline__ void load_codes(const uint8_t *p, uint32_t *q) {
    if constexpr (VEC == 1)
        q[0] = __ldg(p);
    else
        swiglu::Ld<VEC, swiglu::kLdNC>::run(p, q);
}

template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t *p, const uint32_t *q) {
    if constexpr (VEC == 1)
        *p = (uint8_t)q[0];
    else
        swiglu::St<VEC, swiglu::kStStream>::run(p, q);
}

// ---------------------------------------------------------------- kernels ---
// Both are one pass over the data: the forward reads x (2 elements a pair) and
// writes y, two codes and 2/32 scale bytes; the backward reads dy, the codes
// and scales and writes dx (and y).  In bf16 that is 8.06 bytes a pair either
// way for about 15 (forward) and 20 (backward) instructions, so both are bound
// by HBM: [8192, 2 x 14336] bf16 forward 136 us (1.04 of the 6680 GB/s copy),
// backward without weights 140 us (1.01; 169 us with y, 1.04), fp32
// [8192, 2 x 4096] 69 / 71 us (1.02 / 0.99).
//
// A pack is VEC elements of one half; a block of 32 columns is 32 / VEC
// neighbouring lanes, so the forward's block maximum is a shuffle inside that
// lane group.  Rows are padded to whole blocks in the pack index (rows *
// blocks * 32 / VEC packs in all), which keeps a block's lanes together in one
// warp whatever n is.

struct FwdParams {
    const char *x;
    const float *w;  // [rows], or null
    char *y;
    uint8_t *q;
    uint8_t *scales;
    int64_t rows, n;
    int64_t x_stride, y_stride;  // bytes
    int64_t q_stride, s_stride;
    int64_t packs;               // rows * packs per row
    swiglu::FastDiv div;         // by the packs per row
    int32_t row_packs;
    int32_t blocks;              // per half
};

// U packs per thread, T packs apart, all loaded first: 1 for 32-byte packs (two:
// 140 us against 136 for [8192, 2 x 14336] bf16), 2 for 16-byte packs (one: 164 us
// against 153 for [8192, 2 x 14344]).  CTAs of 256 or 64 threads were no faster.
template <typename E, int VEC, int U, int T>
__global__ void __launch_bounds__(T) ckpt8_fwd_kernel(const FwdParams p) {
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    constexpr int B = E::kBytes * VEC;
    constexpr int NW = (B + 3) / 4;
    constexpr int kLanes = kBlock / VEC;  // lanes of a block
    constexpr int QW = (VEC + 3) / 4;
    // the loop's condition is the same for a whole warp: the shuffles need it
    for (int64_t v0 = (int64_t)blockIdx.x * (U * T) + (threadIdx.x & ~31); v0 < p.packs;
         v0 += (int64_t)gridDim.x * (U * T)) {
        uint32_t gw[U][NW], uw[U][NW];
        int64_t row[U];
        int32_t col[U];  // first column (n <= 2^30); -1: no pack
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t v = v0 + (threadIdx.x & 31) + k * T;
            row[k] = swiglu::fast_div(v, p.div);
            const int32_t c = (int32_t)(v - row[k] * p.row_packs);
            col[k] = v < p.packs && (int64_t)c * VEC < p.n ? c * VEC : -1;
#pragma unroll
            for (int i = 0; i < NW; ++i) gw[k][i] = uw[k][i] = 0u;
            if (col[k] >= 0) {
                const char *xr = p.x + row[k] * p.x_stride + (int64_t)col[k] * E::kBytes;
                swiglu::Ld<B, swiglu::kLdNC>::run(xr, gw[k]);
                swiglu::Ld<B, swiglu::kLdNC>::run(xr + p.n * E::kBytes, uw[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float g[VEC], u[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                g[i] = E::get(gw[k], i);
                u[i] = E::get(uw[k], i);
            }
            float mg = finite_amax<VEC>(g), mu = finite_amax<VEC>(u);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) {
                mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
                mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
            }
            if (col[k] >= 0) {
                const uint32_t cg = scale_code(mg), cu = scale_code(mu);
                uint32_t qg[QW], qu[QW];
                encode<VEC>(g, encode_factor(cg), qg);
                encode<VEC>(u, encode_factor(cu), qu);
                uint8_t *qr = p.q + row[k] * p.q_stride + col[k];
                store_codes<VEC>(qr, qg);
                store_codes<VEC>(qr + p.n, qu);
                if (col[k] % kBlock == 0) {
                    uint8_t *sr = p.scales + row[k] * p.s_stride + col[k] / kBlock;
                    sr[0] = (uint8_t)cg;
                    sr[p.blocks] = (uint8_t)cu;
                }
                const float wr = p.w != nullptr ? __ldg(p.w + row[k]) : 1.0f;
                float yv[VEC];
                if (swiglu::pack_has_deep<E, VEC>(gw[k]))
                    swiglu::fwd_pack<E, VEC, swiglu::kWeight, true>(gw[k], uw[k], nullptr, nullptr, wr, yv);
                else
                    swiglu::fwd_pack<E, VEC, swiglu::kWeight, false>(gw[k], uw[k], nullptr, nullptr, wr, yv);
                uint32_t o[NW] = {};
                swiglu::store_pack<E, VEC>(o, yv);
                swiglu::St<B, swiglu::kStStream>::run(p.y + row[k] * p.y_stride + (int64_t)col[k] * E::kBytes, o);
            }
        }
    }
}

// --------------------------------------------------------- narrow packs ---
// Widths, strides or addresses that allow packs of at most 8 bytes, down to single
// elements (odd n, or rows misaligned to one another).  A warp takes K chunks of
// 32 VEC columns of one row, one pack per lane and chunk, so a block is 32 / VEC
// lanes (single elements: the warp, whose maximum is one reduction), each lane
// forms its row pointers once for K packs, and all loads are issued before the
// first is used (one pack per thread over the flattened index, as for wide packs,
// was 1.2 to 2.3 times slower).  Forward and backward without weights, of the 6680
// GB/s copy: packs of 8 bytes bf16 [8192, 2 x 5460] 66 us (0.82) and 62 us (0.87),
// fp32 [8192, 2 x 2730] 61 us (0.77) and 57 us (0.83); of 4 bytes [8192, 2 x 10922]
// 164 us (0.66) and 147 us (0.73); elements bf16 [8192, 2 x 5503] 126 us (0.43) and
// 108 us (0.50), fp32 [3000, 2 x 5503] 51.6 us (0.67) and 50.8 us (0.68).  Packs
// of 4 bytes keep the issue slots 76 - 78 % busy; single elements are bound by their
// memory instructions (taking arithmetic out of them gained 1 %).

template <typename E, int VEC>
constexpr bool kNarrow = E::kBytes * VEC <= 8;

// Chunks of 32 packs a warp takes at a time (4-byte packs forward: 6 chunks 164 us, 4
// 181 us, 8 165 us; backward: 6 147 us, 4 150 us, 8 142 us, but 73 against 65 us for
// weighted packs of 8 bytes).
template <int VEC>
constexpr int kFwdChunks = VEC == 1 ? 8 : VEC == 2 ? 6 : 4;
constexpr int kBwdChunks = 6;

// Positions of a warp: its row and the first column of its lane.
struct Segment {
    int64_t row, col;
};

template <int VEC, int K>
__device__ __forceinline__ Segment segment_at(int64_t seg, int32_t chunks, const swiglu::FastDiv &div) {
    const int64_t r = swiglu::fast_div(seg, div);
    return {r, (seg - r * chunks) * (32 * VEC * K) + (threadIdx.x & 31) * VEC};
}

// Packs of this lane (<= 0: none).
template <int VEC, int K>
__device__ __forceinline__ int live_packs(const Segment &at, int64_t n) {
    return (int)min((int64_t)K, (n - at.col + 32 * VEC - 1) / (32 * VEC));
}

// The largest of the lanes of a block, for the gates and the ups (bits of |v|; those
// of bf16 values are 16 and travel together).
template <typename E, int VEC>
__device__ __forceinline__ void block_max(uint32_t &g, uint32_t &u) {
    if (VEC == 1) {
        g = __reduce_max_sync(0xffffffffu, g);
        u = __reduce_max_sync(0xffffffffu, u);
    } else if (E::kBytes == 2) {
        uint32_t both = (g >> 16) | u;
#pragma unroll
        for (int o = 16 / VEC; o > 0; o >>= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, o));
        g = both << 16;
        u = both & 0xffff0000u;
    } else {
#pragma unroll
        for (int o = 16 / VEC; o > 0; o >>= 1) {
            g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
            u = max(u, __shfl_xor_sync(0xffffffffu, u, o));
        }
    }
}

// The scale codes of a block, from the bits of |v|, which order like the values.
// True: no value of the warp is infinite, NaN or above 1.75 * 2^127, so that encoding
// needs no care.
template <typename E, int VEC>
__device__ __forceinline__ bool block_codes(const float *g, const float *u, uint32_t &cg, uint32_t &cu) {
    constexpr uint32_t kAbs = 0x7fffffffu, kInf = 0x7f800000u;
    uint32_t mg = 0u, mu = 0u;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        mg = max(mg, __float_as_uint(g[i]) & kAbs);
        mu = max(mu, __float_as_uint(u[i]) & kAbs);
    }
    block_max<E, VEC>(mg, mu);
    const bool plain = !__any_sync(0xffffffffu, max(mg, mu) > 0x7f600000u);
    if (!plain) {
        mg = mu = 0u;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint32_t a = __float_as_uint(g[i]) & kAbs, b = __float_as_uint(u[i]) & kAbs;
            mg = max(mg, a < kInf ? a : 0u);
            mu = max(mu, b < kInf ? b : 0u);
        }
        block_max<E, VEC>(mg, mu);
    }
    cg = scale_code(__uint_as_float(mg));
    cu = scale_code(__uint_as_float(mu));
    return plain;
}

// p.row_packs: warps (segments of 32 VEC K columns) per row; p.packs: in all.
template <typename E, int VEC, int K, int T>
__global__ void __launch_bounds__(T) ckpt8_fwd_narrow_kernel(const FwdParams p) {
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    constexpr int EB = E::kBytes, B = EB * VEC, NW = (B + 3) / 4, W = 32 * VEC;
    const int lane = threadIdx.x & 31;
    for (int64_t seg = (int64_t)blockIdx.x * (T / 32) + (threadIdx.x >> 5); seg < p.packs;
         seg += (int64_t)gridDim.x * (T / 32)) {
        const Segment at = segment_at<VEC, K>(seg, p.row_packs, p.div);
        const char *xr = p.x + at.row * p.x_stride + at.col * EB;
        const char *ur = xr + p.n * EB;
        const int live = live_packs<VEC, K>(at, p.n);
        uint32_t gw[K][NW], uw[K][NW];
#pragma unroll
        for (int i = 0; i < K; ++i) {
#pragma unroll
            for (int k = 0; k < NW; ++k) gw[i][k] = uw[i][k] = 0u;
            if (i < live) {
                swiglu::Ld<B, swiglu::kLdNC>::run(xr + i * W * EB, gw[i]);
                swiglu::Ld<B, swiglu::kLdNC>::run(ur + i * W * EB, uw[i]);
            }
        }
        const float wr = p.w != nullptr ? __ldg(p.w + at.row) : 1.0f;
        char *yr = p.y + at.row * p.y_stride + at.col * EB;
        uint8_t *qr = p.q + at.row * p.q_stride + at.col;
        uint8_t *sr = p.scales + at.row * p.s_stride + at.col / kBlock;
        const int64_t first = at.col - lane * VEC;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if (first + W * i >= p.n) break;  // the same for the whole warp
            float g[VEC], u[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                g[k] = E::get(gw[i], k);
                u[k] = E::get(uw[i], k);
            }
            uint32_t cg, cu;
            const bool plain = block_codes<E, VEC>(g, u, cg, cu);
            const float fg = encode_factor(cg), fu = encode_factor(cu);
            if (i < live) {
                uint32_t qg, qu;
                if (VEC == 1 && plain) {
                    qg = codes2(__fmul_rn(g[0], fg), __fmul_rn(u[0], fu));
                    qu = qg >> 8;
                } else if (plain) {
                    encode_values<VEC, false>(g, fg, &qg);
                    encode_values<VEC, false>(u, fu, &qu);
                } else {
                    encode_values<VEC, true>(g, fg, &qg);
                    encode_values<VEC, true>(u, fu, &qu);
                }
                store_codes<VEC>(qr + i * W, &qg);
                store_codes<VEC>(qr + p.n + i * W, &qu);
                float yv[VEC];
                if (E::kDeepScale && (swiglu::pack_has_deep<E, VEC>(gw[i])))
                    swiglu::fwd_pack<E, VEC, swiglu::kWeight, true>(gw[i], uw[i], nullptr, nullptr, wr, yv);
                else
                    swiglu::fwd_pack<E, VEC, swiglu::kWeight, false>(gw[i], uw[i], nullptr, nullptr, wr, yv);
                uint32_t o[NW] = {};
                swiglu::store_pack<E, VEC>(o, yv);
                swiglu::St<B, swiglu::kStStream>::run(yr + i * W * EB, o);
                if (lane * VEC % kBlock == 0) {
                    sr[i * VEC] = (uint8_t)cg;
                    sr[i * VEC + p.blocks] = (uint8_t)cu;
                }
            }
        }
    }
}

struct BwdParams {
    const char *dy;
    const uint8_t *q;
    const uint8_t *scales;
    const float *w;  // [rows], or null
    char *dx;
    float *dw;       // [rows], or null
    char *y;         // or null
    int64_t rows, n;
    int64_t dy_stride, dx_stride, y_stride;  // bytes
    int64_t q_stride, s_stride;
    int64_t packs;
    swiglu::FastDiv div;
    int32_t row_packs;  // ceil(n / VEC)
    int32_t blocks;
};

// One pack: dg, du, y (all with the row weight) and the dw terms added up.
template <typename E, int VEC, int MODE, bool kMayDeep>
__device__ __forceinline__ void bwd_values(const uint32_t *d, const float *g, const float *u, float wr, float &acc,
                                           float *dg, float *du, float *yv) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float df = E::get(d, i);
        const swiglu::Act act = swiglu::activation<E, true, kMayDeep>(g[i]);
        float y = __fmul_rn(act.silu, u[i]);
        float dd = df;
        if (MODE & swiglu::kWeight) {
            float term = __fmul_rn(df, y);
            if (kMayDeep) term = __fmul_rn(term, act.scale);
            acc = __fadd_rn(acc, term);
            dd = __fmul_rn(df, wr);
            y = __fmul_rn(y, wr);
        }
        dg[i] = __fmul_rn(dd, __fmul_rn(u[i], act.dsilu));
        du[i] = __fmul_rn(dd, act.silu);
        if (kMayDeep) {
            dg[i] = __fmul_rn(dg[i], act.scale);
            du[i] = __fmul_rn(du[i], act.scale);
            y = __fmul_rn(y, act.scale);
        }
        yv[i] = y;
    }
}

// What a pack reads.  It lies `at` packs (whole blocks, known to the compiler) behind
// column col of row r.  (Pointers formed once for both halves of the work held 7 more
// registers and were 3 % slower with one pack per thread.)
template <typename E, int VEC>
struct BwdPack {
    static constexpr int B = E::kBytes * VEC;
    uint32_t d[(B + 3) / 4], qg[(VEC + 3) / 4], qu[(VEC + 3) / 4], cg, cu;

    __device__ __forceinline__ void load(const BwdParams &p, int64_t r, int64_t col, int at) {
        const uint8_t *qr = p.q + r * p.q_stride + col;
        const uint8_t *sr = p.scales + r * p.s_stride + col / kBlock;
        swiglu::Ld<B, swiglu::kLdNC>::run(p.dy + r * p.dy_stride + col * E::kBytes + at * B, d);
        load_codes<VEC>(qr + at * VEC, qg);
        load_codes<VEC>(qr + p.n + at * VEC, qu);
        cg = __ldg(sr + at * VEC / kBlock);
        cu = __ldg(sr + p.blocks + at * VEC / kBlock);
    }

    template <int MODE>
    __device__ __forceinline__ void finish(const BwdParams &p, int64_t r, int64_t col, int at, float wr,
                                           float &acc) const {
        float g[VEC], u[VEC], dg[VEC], du[VEC], yv[VEC];
        decode<VEC>(qg, decode_factor(cg), g);
        decode<VEC>(qu, decode_factor(cu), u);
        float gmin = g[0];
#pragma unroll
        for (int i = 1; i < VEC; ++i) gmin = fminf(gmin, g[i]);
        if (E::kDeepScale && (gmin < -64.0f))
            bwd_values<E, VEC, MODE, true>(d, g, u, wr, acc, dg, du, yv);
        else
            bwd_values<E, VEC, MODE, false>(d, g, u, wr, acc, dg, du, yv);
        const auto store = [](char *to, const float *v) {
            uint32_t o[(B + 3) / 4] = {};
            swiglu::store_pack<E, VEC>(o, v);
            swiglu::St<B, swiglu::kStStream>::run(to, o);
        };
        char *dxr = p.dx + r * p.dx_stride + col * E::kBytes;
        store(dxr + at * B, dg);
        store(dxr + p.n * E::kBytes + at * B, du);
        if (p.y != nullptr) store(p.y + r * p.y_stride + col * E::kBytes + at * B, yv);
    }
};

// Without weights: the flattened pack index, one pack per thread.
template <typename E, int VEC, int T>
__global__ void __launch_bounds__(T) ckpt8_bwd_kernel(const BwdParams p) {
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    float acc = 0.0f;
    for (int64_t v = (int64_t)blockIdx.x * T + threadIdx.x; v < p.packs; v += (int64_t)gridDim.x * T) {
        const int64_t r = swiglu::fast_div(v, p.div);
        const int32_t c = (int32_t)(v - r * p.row_packs);
        BwdPack<E, VEC> pack;
        pack.load(p, r, (int64_t)c * VEC, 0);
        pack.template finish<swiglu::kPlain>(p, r, (int64_t)c * VEC, 0, 1.0f, acc);
    }
}

// K packs of one lane (columns col, col + 32 VEC, ...), all loads first.
template <typename E, int VEC, int K, int MODE>
__device__ __forceinline__ void bwd_packs(const BwdParams &p, const Segment &at, float wr, float &acc) {
    const int live = live_packs<VEC, K>(at, p.n);
    BwdPack<E, VEC> pack[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < live) pack[i].load(p, at.row, at.col, 32 * i);
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < live) pack[i].template finish<MODE>(p, at.row, at.col, 32 * i, wr, acc);
}

template <typename E, int VEC, int K, int T>
__global__ void __launch_bounds__(T) ckpt8_bwd_narrow_kernel(const BwdParams p) {
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    float acc = 0.0f;
    for (int64_t seg = (int64_t)blockIdx.x * (T / 32) + (threadIdx.x >> 5); seg < p.packs;
         seg += (int64_t)gridDim.x * (T / 32))
        bwd_packs<E, VEC, K, swiglu::kPlain>(p, segment_at<VEC, K>(seg, p.row_packs, p.div), 1.0f, acc);
}

// With weights a row's dw is one sum, in an order that the sizes fix.  ROWS = 4:
// a warp takes a row (rows of few packs; T = 128).  ROWS = 1: a CTA does, or a
// cluster of them when there are too few rows for the SMs; each CTA then leaves
// its sum in shared memory and the first one adds them in rank order.
//
// Times (bf16, with y where it says so, of the 6680 GB/s copy): [8192, 2 x 4096]
// 44.7 us 0.91, with y 52.5 us 0.96; [8192, 2 x 14336] 143 us 0.99.  Registers held
// to 8 CTAs of 128 threads for 32-byte packs (45.9 us unbound, 62.9 us at 10; measured
// with a CTA per row, the warp per row takes the same bound).
template <typename E, int VEC, int T, int ROWS>
__global__ void __launch_bounds__(T, E::kBytes * VEC == 32 && T == 128 ? 8 : 0) ckpt8_bwd_weighted_kernel(const BwdParams p) {
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    static_assert(ROWS == 1 || ROWS == T / 32, "a row per CTA or per warp");
    __shared__ float red[T / 32 + 1];
    uint32_t rank, size;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t threads = ROWS == 1 ? (int32_t)size * T : 32;  // of a row
    const int32_t id = ROWS == 1 ? (int32_t)rank * T + (int32_t)threadIdx.x : lane;
    const int64_t rows_at_once = (int64_t)(gridDim.x / size) * ROWS;
    for (int64_t r = (int64_t)(blockIdx.x / size) * ROWS + (ROWS == 1 ? 0 : warp); r < p.rows; r += rows_at_once) {
        const float wr = __ldg(p.w + r);
        float acc = 0.0f;
        if constexpr (kNarrow<E, VEC>) {
            constexpr int K = kBwdChunks;
            for (int64_t c = (int64_t)(id >> 5) * (32 * VEC * K); c < p.n; c += (int64_t)threads * (VEC * K))
                bwd_packs<E, VEC, K, swiglu::kWeight>(p, {r, c + lane * VEC}, wr, acc);
        } else {
            // (two packs in flight held 96 registers and were 5-13 % slower in bf16)
            for (int32_t c = id; c < p.row_packs; c += threads) {
                BwdPack<E, VEC> pack;
                pack.load(p, r, (int64_t)c * VEC, 0);
                pack.template finish<swiglu::kWeight>(p, r, (int64_t)c * VEC, 0, wr, acc);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, o));
        if constexpr (ROWS > 1) {
            if (lane == 0) p.dw[r] = acc;
        } else {
            __syncthreads();  // red may still be read for the previous row
            if (lane == 0) red[warp] = acc;
            __syncthreads();
            float t = 0.0f;
            if (threadIdx.x == 0) {
#pragma unroll
                for (int k = 0; k < T / 32; ++k) t = __fadd_rn(t, red[k]);
            }
            if (size > 1) {
                if (threadIdx.x == 0) red[T / 32] = t;
                asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
                if (rank == 0 && threadIdx.x == 0) {
                    const uint32_t own = (uint32_t)__cvta_generic_to_shared(red + T / 32);
                    t = 0.0f;
                    for (uint32_t k = 0; k < size; ++k) {
                        uint32_t at;
                        float v;
                        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(own), "r"(k));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
                        t = __fadd_rn(t, v);
                    }
                }
                // no CTA goes on to its next row, or leaves, before its sum is read
                asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
            }
            if (rank == 0 && threadIdx.x == 0) p.dw[r] = t;
        }
    }
}

}  // namespace ckpt8
