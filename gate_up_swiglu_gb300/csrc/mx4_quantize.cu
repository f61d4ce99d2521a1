// mx4_quantize.cu -- host side of the 4-bit format's conversions: argument checks,
// pack width and launches.  The contract is in include/swiglu_mx4.h, the kernels
// are in mx4.cuh.
#include "fast_div.h"
#include "mx4.cuh"
#include "mx4_host.h"

namespace mx4 {

namespace {

using moe::Span;

constexpr int kT = 256;

int elem_bytes(swiglu_dtype_t dt) { return dt == SWIGLU_F32 ? 4 : dt == SWIGLU_BF16 ? 2 : 0; }

// Whether every row holds whole packs of 32 bytes at aligned addresses.
bool whole_packs(int eb, int64_t n, int64_t stride, const void *p) {
    const int vec = 32 / eb;
    return n % vec == 0 && stride % vec == 0 && (uintptr_t)p % 32 == 0;
}

// The parameters of a tensor of `rows` rows in `parts` parts; `data`: x or y.
ConvParams params(const void *data, const void *q, const void *scales, int64_t rows, int64_t n, int64_t parts,
                  int64_t stride, int eb) {
    ConvParams p{};
    p.x = static_cast<const char *>(data);
    p.y = const_cast<char *>(p.x);
    p.q = static_cast<uint8_t *>(const_cast<void *>(q));
    p.scales = static_cast<uint8_t *>(const_cast<void *>(scales));
    p.rows = rows / parts;
    p.padded_rows = tiles_of(p.rows) * 128;
    p.stride = stride * eb;
    p.n = n;
    p.nb = (int32_t)blocks_of(n);
    p.chunks = (int32_t)chunks_of(n);
    const uint64_t a = (uint64_t)(uintptr_t)data, z = a + (uint64_t)(((rows - 1) * stride + n) * eb);
    p.lo = (a + 15) & ~(uint64_t)15;
    p.hi = z & ~(uint64_t)15;
    return p;
}

template <typename K>
swiglu_status_t launch(K kernel, ConvParams p, int vec, int64_t parts, swiglu_stream_t stream) {
    p.row_units = p.chunks * (kTileBlocks * kBlock / vec);
    p.div_row = swiglu::make_fast_div((uint64_t)p.row_units);
    p.div_part = swiglu::make_fast_div((uint64_t)(p.padded_rows / kRows));
    static_assert(kPlaces % kT == 0, "no CTA is cut: a warp's shuffles have all its lanes");
    const int64_t ctas = parts * (p.padded_rows / kRows) * p.row_units / kT;
    if (ctas > INT32_MAX) return SWIGLU_ERR_SHAPE;
    const cudaError_t e = moe::launch(kernel, dim3((unsigned)ctas), kT, 0, stream, 0, p);
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

}  // namespace

swiglu_status_t launch_quantize(const void *x, void *q, void *scales, int64_t rows, int64_t n, int64_t parts,
                                int64_t x_row_stride, swiglu_dtype_t dtype, swiglu_stream_t stream) {
    const int eb = elem_bytes(dtype);
    const ConvParams p = params(x, q, scales, rows, n, parts, x_row_stride, eb);
    const bool whole = whole_packs(eb, n, x_row_stride, x);
    if (dtype == SWIGLU_BF16)
        return whole ? launch(mx4_quantize_kernel<swiglu::BF16, 16, false, kT>, p, 16, parts, stream)
                     : launch(mx4_quantize_kernel<swiglu::BF16, 8, true, kT>, p, 8, parts, stream);
    return whole ? launch(mx4_quantize_kernel<swiglu::F32, 8, false, kT>, p, 8, parts, stream)
                 : launch(mx4_quantize_kernel<swiglu::F32, 8, true, kT>, p, 8, parts, stream);
}

}  // namespace mx4

extern "C" {

swiglu_status_t swiglu_mx4_scales_size(int64_t rows, int64_t n, int64_t parts, size_t *bytes) {
    if (bytes == nullptr) return SWIGLU_ERR_NULL;
    if (!mx4::sizes_ok(rows, n) || parts < 1 || rows % parts != 0) return SWIGLU_ERR_SHAPE;
    *bytes = (size_t)mx4::scale_bytes(rows, n, parts);
    return SWIGLU_OK;
}

swiglu_status_t swiglu_mx4_quantize(const void *x, void *q, void *scales, int64_t rows, int64_t n, int64_t parts,
                                    int64_t x_row_stride, swiglu_dtype_t dtype, swiglu_stream_t stream) {
    using namespace mx4;
    const int eb = elem_bytes(dtype);
    if (eb == 0) return SWIGLU_ERR_DTYPE;
    if (!sizes_ok(rows, n) || parts < 1 || rows % parts != 0) return SWIGLU_ERR_SHAPE;
    if (rows == 0 || n == 0) return SWIGLU_OK;
    if (x == nullptr || q == nullptr || scales == nullptr) return SWIGLU_ERR_NULL;
    if (x_row_stride < n) return SWIGLU_ERR_STRIDE;
    Span sx, sq, ss;
    if (!moe::span_of(x, rows, n, x_row_stride, eb, sx) || !span_bytes(q, q_bytes(rows, n), sq) ||
        !span_bytes(scales, scale_bytes(rows, n, parts), ss))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sq, ss}, {sx})) return SWIGLU_ERR_ALIAS;
    if ((uintptr_t)x % eb != 0 || ((uintptr_t)q | (uintptr_t)scales) % 16 != 0) return SWIGLU_ERR_STRIDE;
    return launch_quantize(x, q, scales, rows, n, parts, x_row_stride, dtype, stream);
}

swiglu_status_t swiglu_mx4_dequantize(const void *q, const void *scales, void *y, int64_t rows, int64_t n,
                                      int64_t parts, int64_t y_row_stride, swiglu_dtype_t dtype,
                                      swiglu_stream_t stream) {
    using namespace mx4;
    const int eb = elem_bytes(dtype);
    if (eb == 0) return SWIGLU_ERR_DTYPE;
    if (!sizes_ok(rows, n) || parts < 1 || rows % parts != 0) return SWIGLU_ERR_SHAPE;
    if (rows == 0 || n == 0) return SWIGLU_OK;
    if (q == nullptr || scales == nullptr || y == nullptr) return SWIGLU_ERR_NULL;
    if (y_row_stride < n) return SWIGLU_ERR_STRIDE;
    Span sy, sq, ss;
    if (!moe::span_of(y, rows, n, y_row_stride, eb, sy) || !span_bytes(q, q_bytes(rows, n), sq) ||
        !span_bytes(scales, scale_bytes(rows, n, parts), ss))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sy}, {sq, ss})) return SWIGLU_ERR_ALIAS;
    if ((uintptr_t)y % eb != 0 || ((uintptr_t)q | (uintptr_t)scales) % 16 != 0) return SWIGLU_ERR_STRIDE;
    const ConvParams p = params(y, q, scales, rows, n, parts, y_row_stride, eb);
    const bool whole = whole_packs(eb, n, y_row_stride, y);
    if (dtype == SWIGLU_BF16)
        return whole ? launch(mx4_dequantize_kernel<swiglu::BF16, 16, false, kT>, p, 16, parts, stream)
                     : launch(mx4_dequantize_kernel<swiglu::BF16, 8, true, kT>, p, 8, parts, stream);
    return whole ? launch(mx4_dequantize_kernel<swiglu::F32, 8, false, kT>, p, 8, parts, stream)
                 : launch(mx4_dequantize_kernel<swiglu::F32, 8, true, kT>, p, 8, parts, stream);
}

}  // extern "C"
