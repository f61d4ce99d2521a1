// mx4.cuh -- device code of the 4-bit format of swiglu_mx4.h: E2M1 codes with
// one power-of-two scale per block of 32 columns, scales in tiles of 128 rows
// by 4 blocks.
#pragma once

#include <stdint.h>

#include "load_after.cuh"
#include "swiglu_kernels.cuh"

namespace mx4 {

constexpr int kBlock = 32;       // columns per scale
constexpr int kTileRows = 128;   // rows and
constexpr int kTileBlocks = 4;   // blocks of a scale tile
constexpr int kTileBytes = kTileRows * kTileBlocks;

// The bits of |v|: their order is that of the values, infinities and NaN on top.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale byte of a block whose largest magnitude has these bits: the smallest
// c >= 0 with amax <= 6 * 2^(c - 127), 6 = 1.5 * 2^2.  With amax = m 2^k (1 <= m
// < 2), c = k - 2 + 127, one more when m > 1.5; adding 0x3fffff to the bits
// carries into the exponent exactly for mantissas above .5.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255;
    return (uint32_t)max((int)((amax + 0x3fffffu) >> 23) - 2, 0);
}

// 2^(127 - c), exact for c <= 253.  A NaN block (c = 255) takes the factor 0 (which leaves
// NaN and infinities NaN: scale_values puts zeros for the whole block).
__device__ __forceinline__ float encode_factor(uint32_t c) {
    return c == 255 ? 0.0f : __uint_as_float((254u - c) << 23);
}

// 2^(c - 127), exact (2^-127 is a subnormal); 255 is NaN.
__device__ __forceinline__ float decode_factor(uint32_t c) {
    return __uint_as_float(c == 0 ? 1u << 22 : c == 255 ? 0x7fc00000u : c << 23);
}

// Two values to codes, nearest even, `lo` in the low half of the byte.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    uint32_t r;
    asm("{\n.reg .b8 t;\ncvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\nmov.b32 %0, {t, t, t, t};\n}\n"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r & 0xffu;
}

// Eight values to 32 bits of codes, v[0] in the lowest four.
__device__ __forceinline__ uint32_t codes8(const float *v) {
    uint32_t r;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// N values of a block under the scale c, ready for the conversion.  NaN blocks give
// zeros; under the largest scale values stay at 3 (see swiglu_mx4.h): one test a block
// tells both from the rest.
template <int N>
__device__ __forceinline__ void scale_values(float *v, uint32_t c) {
    const float f = encode_factor(c);
    const uint64_t f2 = swiglu::x2(f, f);
#pragma unroll
    for (int k = 0; k < N; k += 2) swiglu::x2_split(swiglu::mul_x2(swiglu::x2(v[k], v[k + 1]), f2), v[k], v[k + 1]);
    if (c >= 253)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = c == 255 ? 0.0f : fminf(fmaxf(v[k], -3.0f), 3.0f);
}

// The byte of row i, block b of a part whose tiles start at `tile`.
__device__ __forceinline__ int64_t scale_offset(int64_t tile, int64_t i, int32_t b, int32_t chunks) {
    const int64_t t = tile + (i >> 7);
    const int32_t r = (int32_t)(i & 127);
    return (t * chunks + (b >> 2)) * kTileBytes + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
}

// ---------------------------------------------------------------- kernels ---
// Quantising and its inverse are one pass over the data: 2 (4) bytes an element on the
// one side, 17/32 on the other, a few instructions an element: HBM bound.  [28672, 4096]
// bf16 46.5 us (94 % of the copy rate), the inverse 44.9 us (98 %).  Rows at any address pay
// for their shifts and their ends: [8192, 4095] bf16 31 us (40 %) and 39 us (32 %).
//
// A thread takes eight or sixteen neighbouring elements (a pack) of kRows rows below
// each other, so that what it costs to find its place comes once; 32 / VEC neighbouring
// lanes hold a block.  The index space covers the scale tiles: padded rows (whole tiles a
// part) and padded blocks (whole chunks), so that every scale byte is written; and so every
// thread of a CTA has a place, and all lanes of a warp take part in its shuffles.

constexpr int kRows = 4;
constexpr int kPlaces = kTileRows / kRows * (kTileBlocks * kBlock / 16);  // of a scale tile, in the longer packs

struct ConvParams {
    const char *x;   // the tensor: source of quantising,
    char *y;         // or result of the inverse
    uint8_t *q;
    uint8_t *scales;
    int64_t rows;         // a part
    int64_t padded_rows;  // a part
    int64_t stride;       // of x or y, bytes
    int64_t n;
    uint64_t lo, hi;      // x's bytes, rounded inwards to 16 (see load_any)
    int32_t nb, chunks;
    int32_t row_units;    // packs a padded row
    swiglu::FastDiv div_row, div_part;  // by row_units, by padded rows / kRows
};

// The pack of a thread: row group `i` of the part that starts at row `first` of the tensor
// and scale tile `tile`, pack `c` of the row.
struct Place {
    int64_t tile, i, first;
    int32_t c;
};

__device__ __forceinline__ Place locate(const ConvParams &p, int64_t unit) {
    const int64_t pr = swiglu::fast_div(unit, p.div_row), part = swiglu::fast_div(pr, p.div_part);
    Place at;
    at.c = (int32_t)(unit - pr * p.row_units);
    at.i = pr * kRows - part * p.padded_rows;
    at.tile = part * (p.padded_rows >> 7);
    at.first = part * p.rows;
    return at;
}

// Eight elements from any address: the aligned 16-byte pieces around them, shifted into
// place.  A piece that reaches out of the tensor (of its first or last bytes) is not read:
// there the elements come one by one.
template <typename E>
__device__ __forceinline__ void load_any(const char *src, uint64_t lo, uint64_t hi, uint32_t (&w)[2 * E::kBytes]) {
    constexpr int NW = 2 * E::kBytes, V = NW / 4 + 1;  // words of the result, pieces
    const uint64_t a = reinterpret_cast<uint64_t>(src), base = a & ~(uint64_t)15;
    if (base >= lo && base + 16 * V <= hi) {
        uint32_t r[4 * V];
#pragma unroll
        for (int k = 0; k < V; ++k) swiglu::load_after<16, true>(reinterpret_cast<const char *>(base) + 16 * k, r + 4 * k);
        const uint32_t off = (uint32_t)(a & 15);
#pragma unroll
        for (int k = 0; k < NW + 2; ++k) r[k] = off & 8 ? r[k + 2 < 4 * V ? k + 2 : k] : r[k];
#pragma unroll
        for (int k = 0; k < NW + 1; ++k) r[k] = off & 4 ? r[k + 1] : r[k];
#pragma unroll
        for (int k = 0; k < NW; ++k) w[k] = E::kBytes == 4 ? r[k] : __funnelshift_r(r[k], r[k + 1], (off & 2) * 8);
    } else {
#pragma unroll
        for (int k = 0; k < NW; ++k) w[k] = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t e[1];
            swiglu::load_after<E::kBytes, true>(src + k * E::kBytes, e);
            if constexpr (E::kBytes == 4)
                w[k] = e[0];
            else
                w[k / 2] |= e[0] << (k % 2 * 16);
        }
    }
}

// ANY: rows at any address, of any length (VEC = 8); else packs are aligned and whole.
template <typename E, int VEC, bool ANY, int T>
__global__ void __launch_bounds__(T) mx4_quantize_kernel(const __grid_constant__ ConvParams p) {
    constexpr int L = kBlock / VEC, B = E::kBytes * VEC, NW = B / 4;
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    const int64_t unit = (int64_t)blockIdx.x * T + threadIdx.x;
    const Place at = locate(p, unit);
    const int32_t b = at.c / L;
    const int64_t col = (int64_t)at.c * VEC;
    const int left = p.n - col < VEC ? (int)(p.n - col) : VEC;  // elements of the pack inside the row
    uint32_t w[kRows][NW];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
        for (int k = 0; k < NW; ++k) w[r][k] = 0;
        if (left > 0 && at.i + r < p.rows) {
            const char *src = p.x + (at.first + at.i + r) * p.stride + col * E::kBytes;
            if constexpr (!ANY) {
                swiglu::load_after<B, false>(src, w[r]);
            } else if (left == VEC) {
                load_any<E>(src, p.lo, p.hi, w[r]);
            } else {
                for (int k = 0; k < VEC; ++k)
                    if (k < left) {
                        uint32_t e[1];
                        swiglu::load_after<E::kBytes, true>(src + k * E::kBytes, e);
#pragma unroll
                        for (int j = 0; j < VEC; ++j)
                            if (j == k) w[r][j * E::kBytes / 4] |= E::kBytes == 4 ? e[0] : e[0] << (j % 2 * 16);
                    }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        // the bits of the largest |x|: their order is that of the values
        uint32_t m = 0;
        if constexpr (E::kBytes == 4) {
#pragma unroll
            for (int k = 0; k < NW; ++k) m = max(m, w[r][k] & 0x7fffffffu);
        } else {
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const uint32_t v = w[r][k] & 0x7fff7fffu;
                asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(v));
            }
            m = max(m & 0xffff0000u, m << 16);
        }
#pragma unroll
        for (int d = 1; d < L; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const uint32_t sc = scale_byte(m);
        const bool live = at.i + r < p.rows;
        if (live && b < p.nb) {
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = E::get(w[r], k);
            scale_values<VEC>(v, sc);
            uint32_t o[VEC / 8];
#pragma unroll
            for (int k = 0; k < VEC; k += 8) o[k / 8] = codes8(v + k);
            swiglu::St<VEC / 2, swiglu::kStPlain>::run(p.q + (at.first + at.i + r) * ((int64_t)p.nb * 16) + col / 2, o);
        }
        if (at.c % L == 0) p.scales[scale_offset(at.tile, at.i + r, b, p.chunks)] = live ? (uint8_t)sc : 0;
    }
}

__device__ __forceinline__ uint32_t load_byte(const uint8_t *p) {
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// The value of a code: e2m1 is exact in fp16 and fp32.
__device__ __forceinline__ void values2(uint32_t byte, float f, float &lo, float &hi) {
    uint32_t pair;
    asm("{\n.reg .b8 t, u, v, w;\nmov.b32 {t, u, v, w}, %1;\ncvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(pair) : "r"(byte));
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}\n"
        : "=f"(lo), "=f"(hi)
        : "r"(pair));
    lo = __fmul_rn(lo, f);
    hi = __fmul_rn(hi, f);
}

// Element e (8 a pack) of a pack's words.
template <typename E>
__device__ __forceinline__ void store_element(char *dst, const uint32_t (&w)[2 * E::kBytes], int e) {
    uint32_t v[1] = {0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j == e) v[0] = E::kBytes == 4 ? w[j * E::kBytes / 4] : w[j * E::kBytes / 4] >> (j % 2 * 16) & 0xffffu;
    swiglu::St<E::kBytes, swiglu::kStPlain>::run(dst + e * E::kBytes, v);
}

// Packs of eight elements to any address, by lanes that hold neighbouring packs of a row:
// each lane puts the end of its left neighbour's pack (`before`, in a warp's first lane)
// in front of its own and stores aligned 16-byte pieces.  What is left over goes element
// by element: the start of a row's first pack, the end of its last whole one, and a pack
// that the row's end cuts (left < 8).
template <typename E>
__device__ __forceinline__ void store_any(char *dst, const uint32_t (&w)[2 * E::kBytes], const uint32_t (&before)[4],
                                          bool first, bool last, int left) {
    constexpr int NW = 2 * E::kBytes;
    const uint32_t off = (uint32_t)(reinterpret_cast<uint64_t>(dst) & 15);
    uint32_t r[4 + NW];  // the neighbour's last 16 bytes, then the pack
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        r[k] = __shfl_up_sync(0xffffffffu, w[NW - 4 + k], 1);
        if ((threadIdx.x & 31) == 0) r[k] = before[k];
    }
#pragma unroll
    for (int k = 0; k < NW; ++k) r[4 + k] = w[k];
    if (left < 8) {
        for (int e = 0; e < left; ++e) store_element<E>(dst, w, e);
        return;
    }
    // words from `off` bytes before the pack on, in steps of 8, 4 and 2 bytes
    uint32_t a[2 + NW], t[1 + NW], o[NW];
#pragma unroll
    for (int k = 0; k < 2 + NW; ++k) a[k] = off & 8 ? r[k] : r[k + 2];
#pragma unroll
    for (int k = 0; k < 1 + NW; ++k) t[k] = off & 4 ? a[k] : a[k + 1];
#pragma unroll
    for (int k = 0; k < NW; ++k) o[k] = E::kBytes == 2 && (off & 2) ? __funnelshift_r(t[k], t[k + 1], 16) : t[k + 1];
    const bool head = first && off != 0;
#pragma unroll
    for (int k = 0; k < NW / 4; ++k)
        if (k > 0 || !head) swiglu::St<16, swiglu::kStPlain>::run(dst - off + 16 * k, o + 4 * k);
    if (head)
        for (int e = 0; e < (int)(16 - off) / E::kBytes; ++e) store_element<E>(dst, w, e);
    if (last)
        for (int e = 8 - (int)off / E::kBytes; e < 8; ++e) store_element<E>(dst, w, e);
}

template <typename E, int VEC, bool ANY, int T>
__global__ void __launch_bounds__(T) mx4_dequantize_kernel(const __grid_constant__ ConvParams p) {
    constexpr int L = kBlock / VEC, B = E::kBytes * VEC, NW = B / 4;
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    const int64_t unit = (int64_t)blockIdx.x * T + threadIdx.x;
    const Place at = locate(p, unit);
    const int32_t b = at.c / L;
    const int64_t col = (int64_t)at.c * VEC;
    const int left = p.n - col < VEC ? (int)(p.n - col) : VEC;  // elements of the pack inside the row
    // the last eight codes of the pack to the left, for a warp's first lane (see store_any)
    const bool reach = ANY && (threadIdx.x & 31) == 0 && at.c > 0 && left > 0;
    uint32_t q[kRows][VEC / 8], sc[kRows], qb[kRows], scb[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        sc[r] = qb[r] = scb[r] = 0;
#pragma unroll
        for (int k = 0; k < VEC / 8; ++k) q[r][k] = 0;
        if (left > 0 && at.i + r < p.rows) {
            const uint8_t *src = p.q + (at.first + at.i + r) * ((int64_t)p.nb * 16) + col / 2;
            swiglu::load_after<VEC / 2, false>(src, q[r]);
            sc[r] = load_byte(p.scales + scale_offset(at.tile, at.i + r, b, p.chunks));
            if (reach) {
                swiglu::load_after<4, false>(src - 4, qb + r);
                scb[r] = load_byte(p.scales + scale_offset(at.tile, at.i + r, (at.c - 1) / L, p.chunks));
            }
        }
    }
    const auto decode = [](const uint32_t *codes, uint32_t scale, uint32_t *w, int n) {
        const float f = decode_factor(scale);
#pragma unroll
        for (int k = 0; k < n; k += 2) {
            float lo, hi;
            values2(codes[k / 8] >> (k % 8 * 4) & 0xffu, f, lo, hi);
            E::put2(w, k, lo, hi);
        }
    };
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        uint32_t w[NW];
        decode(q[r], sc[r], w, VEC);
        char *dst = p.y + (at.first + at.i + r) * p.stride + col * E::kBytes;
        const bool live = at.i + r < p.rows;  // of all lanes of a row
        if constexpr (ANY) {
            uint32_t before[4] = {0, 0, 0, 0};
            if (reach) {
                uint32_t all[NW];
                decode(qb + r, scb[r], all, 8);
#pragma unroll
                for (int k = 0; k < 4; ++k) before[k] = all[NW - 4 + k];
            }
            store_any<E>(dst, w, before, at.c == 0, p.n - col < 16, live ? left : 0);
        } else if (live && left > 0) {
            swiglu::St<B, swiglu::kStStream>::run(dst, w);
        }
    }
}

}  // namespace mx4
