// ckpt8.cu -- host side of the 8-bit activation checkpoint: argument checks,
// pack width and launches.  The contract is in include/swiglu_moe.h, the
// kernels are in ckpt8.cuh.
#include <climits>

#include "ckpt8.cuh"
#include "moe_host.h"

namespace {

using moe::Span;

int elem_bytes(swiglu_dtype_t dt) { return dt == SWIGLU_F32 ? 4 : dt == SWIGLU_BF16 ? 2 : 0; }

// Far beyond any memory; keeps rows * packs per row inside int64.
constexpr int64_t kMaxRows = (int64_t)1 << 32;

// Multiplier and shift of swiglu::fast_div for the divisor d >= 1 (the
// smallest l with 2^l >= d, m = ceil(2^(63 + l) / d)).
swiglu::FastDiv make_fast_div(uint64_t d) {
    if (d <= 1) return {0, -1};
    int l = 0;
    while (l < 63 && ((uint64_t)1 << l) < d) ++l;
    const unsigned __int128 num = (unsigned __int128)1 << (63 + l);
    return {(uint64_t)((num + d - 1) / d), l - 1};
}

bool multiple(int64_t by, std::initializer_list<int64_t> v) {
    for (int64_t x : v)
        if (x % by != 0) return false;
    return true;
}

// Packs a thread of the forward takes at once, by the pack's bytes.
template <int BYTES>
constexpr int kFwdPacks = BYTES >= 32 ? 1 : 2;

// The weighted backward: packs (or groups of narrow ones) of a row that one
// warp takes ([16384, 2 x 256] bf16 22 -> 12 us against a CTA per row), and the
// CTAs up to which rows are shared by clusters (one row of n = 28008 fp32 23 -> 9 us).
// 16-byte packs take CTAs of 256 threads ([8192, 2 x 14344] bf16 175 -> 153 us; 32-byte
// packs of n = 14336 were slower that way, 144 -> 159 us).
constexpr int64_t kWarpRow = 64;
constexpr int64_t kClusterCtas = 152 * 8;

// CTAs of T threads for `packs` packs, one pack a thread (the kernels' grid
// stride covers what the launch limit leaves).
unsigned one_pass(int64_t packs, int T) {
    const int64_t need = (packs + T - 1) / T;
    return (unsigned)(need < INT32_MAX ? need : INT32_MAX);
}

template <typename E, int VEC>
swiglu_status_t launch_fwd(ckpt8::FwdParams p, swiglu_stream_t stream) {
    constexpr int T = 128;
    cudaError_t e;
    if constexpr (ckpt8::kNarrow<E, VEC>) {
        constexpr int K = ckpt8::kFwdChunks<VEC>;
        p.row_packs = (int32_t)((p.n + 32 * VEC * K - 1) / (32 * VEC * K));
        p.packs = p.rows * p.row_packs;
        p.div = make_fast_div((uint64_t)p.row_packs);
        e = moe::launch(ckpt8::ckpt8_fwd_narrow_kernel<E, VEC, K, T>, dim3(one_pass(p.packs, T / 32)), T, 0, stream, 0, p);
    } else {
        p.row_packs = p.blocks * (ckpt8::kBlock / VEC);
        p.packs = p.rows * p.row_packs;
        p.div = make_fast_div((uint64_t)p.row_packs);
        constexpr int U = kFwdPacks<E::kBytes * VEC>;
        e = moe::launch(ckpt8::ckpt8_fwd_kernel<E, VEC, U, T>, dim3(one_pass(p.packs, U * T)), T, 0, stream, 0, p);
    }
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

template <typename E, int VEC>
swiglu_status_t launch_bwd(ckpt8::BwdParams p, swiglu_stream_t stream) {
    constexpr int T = 128;
    p.row_packs = (int32_t)((p.n + VEC - 1) / VEC);
    p.packs = p.rows * p.row_packs;
    p.div = make_fast_div((uint64_t)p.row_packs);
    cudaError_t e;
    if (p.dw != nullptr) {
        // a warp per row of up to kWarpRow packs, else a CTA, or a cluster while that
        // gives the SMs more to do
        const int64_t packs =
            ckpt8::kNarrow<E, VEC> ? (p.row_packs + ckpt8::kBwdChunks - 1) / ckpt8::kBwdChunks : p.row_packs;
        if (packs <= kWarpRow) {
            const int64_t ctas = (p.rows + T / 32 - 1) / (T / 32);
            e = moe::launch(ckpt8::ckpt8_bwd_weighted_kernel<E, VEC, T, T / 32>,
                            dim3((unsigned)(ctas < INT32_MAX ? ctas : INT32_MAX)), T, 0, stream, 0, p);
        } else {
            int size = 1;
            while (size < 8 && p.rows * size * 2 <= kClusterCtas && packs > (int64_t)T * size) size *= 2;
            const int64_t ctas = p.rows < (1 << 27) ? p.rows : (1 << 27);
            constexpr int TR = E::kBytes * VEC == 16 ? 256 : T;
            e = moe::launch(ckpt8::ckpt8_bwd_weighted_kernel<E, VEC, TR, 1>, dim3((unsigned)(ctas * size)), TR, 0,
                            stream, size, p);
        }
    } else if constexpr (ckpt8::kNarrow<E, VEC>) {
        constexpr int K = ckpt8::kBwdChunks;
        p.row_packs = (int32_t)((p.n + 32 * VEC * K - 1) / (32 * VEC * K));
        p.packs = p.rows * p.row_packs;
        p.div = make_fast_div((uint64_t)p.row_packs);
        e = moe::launch(ckpt8::ckpt8_bwd_narrow_kernel<E, VEC, K, T>, dim3(one_pass(p.packs, T / 32)), T, 0, stream, 0, p);
    } else {
        e = moe::launch(ckpt8::ckpt8_bwd_kernel<E, VEC, T>, dim3(one_pass(p.packs, T)), T, 0, stream, 0, p);
    }
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

// Elements of the widest pack (32 to 4 bytes, two elements at least) that n, the tensors' strides
// (elements) and addresses and the codes' stride and address allow, else 1.
int pick_vec(int eb, int64_t n, std::initializer_list<int64_t> strides, std::initializer_list<int64_t> addresses,
             int64_t q_stride, const void *q) {
    for (int bytes = 32; bytes >= 2 * eb; bytes /= 2) {
        const int vec = bytes / eb;
        if (n % vec == 0 && multiple(vec, strides) && multiple(bytes, addresses) && q_stride % vec == 0 &&
            (uintptr_t)q % (uintptr_t)vec == 0)
            return vec;
    }
    return 1;
}

}  // namespace

extern "C" {

swiglu_status_t swiglu_ckpt8_fwd(const void *x, const float *w, void *y, void *q, void *scales, int64_t rows,
                                 int64_t n, int64_t x_row_stride, int64_t y_row_stride, int64_t q_row_stride,
                                 int64_t scale_row_stride, swiglu_dtype_t dtype, swiglu_stream_t stream) {
    const int eb = elem_bytes(dtype);
    if (eb == 0) return SWIGLU_ERR_DTYPE;
    if (rows < 0 || rows > kMaxRows || n < 0 || n > SWIGLU_MAX_N) return SWIGLU_ERR_SHAPE;
    if (rows == 0 || n == 0) return SWIGLU_OK;
    if (x == nullptr || y == nullptr || q == nullptr || scales == nullptr) return SWIGLU_ERR_NULL;
    const int64_t nb = (n + SWIGLU_CKPT8_BLOCK - 1) / SWIGLU_CKPT8_BLOCK;
    if (x_row_stride < 2 * n || y_row_stride < n || q_row_stride < 2 * n || scale_row_stride < 2 * nb)
        return SWIGLU_ERR_STRIDE;
    Span sx, sw, sy, sq, ss;
    if (!moe::span_of(x, rows, 2 * n, x_row_stride, eb, sx) || !moe::span_of(w, rows, 1, 1, 4, sw) ||
        !moe::span_of(y, rows, n, y_row_stride, eb, sy) || !moe::span_of(q, rows, 2 * n, q_row_stride, 1, sq) ||
        !moe::span_of(scales, rows, 2 * nb, scale_row_stride, 1, ss))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sy, sq, ss}, {sx, sw})) return SWIGLU_ERR_ALIAS;
    if ((uintptr_t)x % eb != 0 || (uintptr_t)y % eb != 0 || (uintptr_t)w % 4 != 0) return SWIGLU_ERR_STRIDE;

    ckpt8::FwdParams p{};
    p.x = static_cast<const char *>(x);
    p.w = w;
    p.y = static_cast<char *>(y);
    p.q = static_cast<uint8_t *>(q);
    p.scales = static_cast<uint8_t *>(scales);
    p.rows = rows;
    p.n = n;
    p.x_stride = x_row_stride * eb;
    p.y_stride = y_row_stride * eb;
    p.q_stride = q_row_stride;
    p.s_stride = scale_row_stride;
    p.blocks = (int32_t)nb;
    const int vec = pick_vec(eb, n, {x_row_stride, y_row_stride}, {(int64_t)(uintptr_t)x, (int64_t)(uintptr_t)y},
                             q_row_stride, q);
    if (dtype == SWIGLU_BF16) {
        if (vec == 16) return launch_fwd<swiglu::BF16, 16>(p, stream);
        if (vec == 8) return launch_fwd<swiglu::BF16, 8>(p, stream);
        if (vec == 4) return launch_fwd<swiglu::BF16, 4>(p, stream);
        if (vec == 2) return launch_fwd<swiglu::BF16, 2>(p, stream);
        return launch_fwd<swiglu::BF16, 1>(p, stream);
    }
    if (vec == 8) return launch_fwd<swiglu::F32, 8>(p, stream);
    if (vec == 4) return launch_fwd<swiglu::F32, 4>(p, stream);
    if (vec == 2) return launch_fwd<swiglu::F32, 2>(p, stream);
    return launch_fwd<swiglu::F32, 1>(p, stream);
}

swiglu_status_t swiglu_ckpt8_bwd(const void *dy, const void *q, const void *scales, const float *w, void *dx,
                                 float *dw, void *y, int64_t rows, int64_t n, int64_t dy_row_stride,
                                 int64_t q_row_stride, int64_t scale_row_stride, int64_t dx_row_stride,
                                 int64_t y_row_stride, swiglu_dtype_t dtype, swiglu_stream_t stream) {
    const int eb = elem_bytes(dtype);
    if (eb == 0) return SWIGLU_ERR_DTYPE;
    if (rows < 0 || rows > kMaxRows || n < 0 || n > SWIGLU_MAX_N) return SWIGLU_ERR_SHAPE;
    if (rows == 0) return SWIGLU_OK;
    Span sdw;
    if (!moe::span_of(dw, rows, 1, 1, 4, sdw)) return SWIGLU_ERR_SHAPE;
    if (n == 0) {  // dw is a sum over no columns
        if (dw == nullptr) return SWIGLU_OK;
        if ((uintptr_t)dw % 4 != 0) return SWIGLU_ERR_STRIDE;
        const cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)rows * 4, reinterpret_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
    }
    if (dy == nullptr || q == nullptr || scales == nullptr || dx == nullptr || (w == nullptr) != (dw == nullptr))
        return SWIGLU_ERR_NULL;
    const int64_t nb = (n + SWIGLU_CKPT8_BLOCK - 1) / SWIGLU_CKPT8_BLOCK;
    if (dy_row_stride < n || q_row_stride < 2 * n || scale_row_stride < 2 * nb || dx_row_stride < 2 * n ||
        (y != nullptr && y_row_stride < n))
        return SWIGLU_ERR_STRIDE;
    Span sdy, sq, ss, sw, sdx, sy;
    if (!moe::span_of(dy, rows, n, dy_row_stride, eb, sdy) || !moe::span_of(q, rows, 2 * n, q_row_stride, 1, sq) ||
        !moe::span_of(scales, rows, 2 * nb, scale_row_stride, 1, ss) || !moe::span_of(w, rows, 1, 1, 4, sw) ||
        !moe::span_of(dx, rows, 2 * n, dx_row_stride, eb, sdx) ||
        (y != nullptr && !moe::span_of(y, rows, n, y_row_stride, eb, sy)))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sdx, sdw, sy}, {sdy, sq, ss, sw})) return SWIGLU_ERR_ALIAS;
    if ((uintptr_t)dy % eb != 0 || (uintptr_t)dx % eb != 0 || (uintptr_t)y % eb != 0 || (uintptr_t)w % 4 != 0 ||
        (uintptr_t)dw % 4 != 0)
        return SWIGLU_ERR_STRIDE;

    ckpt8::BwdParams p{};
    p.dy = static_cast<const char *>(dy);
    p.q = static_cast<const uint8_t *>(q);
    p.scales = static_cast<const uint8_t *>(scales);
    p.w = w;
    p.dx = static_cast<char *>(dx);
    p.dw = dw;
    p.y = static_cast<char *>(y);
    p.rows = rows;
    p.n = n;
    p.dy_stride = dy_row_stride * eb;
    p.dx_stride = dx_row_stride * eb;
    p.y_stride = y != nullptr ? y_row_stride * eb : 0;
    p.q_stride = q_row_stride;
    p.s_stride = scale_row_stride;
    p.blocks = (int32_t)nb;
    const int64_t ys = y != nullptr ? y_row_stride : 0;
    const int vec = pick_vec(eb, n, {dy_row_stride, dx_row_stride, ys},
                             {(int64_t)(uintptr_t)dy, (int64_t)(uintptr_t)dx, (int64_t)(uintptr_t)y}, q_row_stride, q);
    if (dtype == SWIGLU_BF16) {
        if (vec == 16) return launch_bwd<swiglu::BF16, 16>(p, stream);
        if (vec == 8) return launch_bwd<swiglu::BF16, 8>(p, stream);
        if (vec == 4) return launch_bwd<swiglu::BF16, 4>(p, stream);
        if (vec == 2) return launch_bwd<swiglu::BF16, 2>(p, stream);
        return launch_bwd<swiglu::BF16, 1>(p, stream);
    }
    if (vec == 8) return launch_bwd<swiglu::F32, 8>(p, stream);
    if (vec == 4) return launch_bwd<swiglu::F32, 4>(p, stream);
    if (vec == 2) return launch_bwd<swiglu::F32, 2>(p, stream);
    return launch_bwd<swiglu::F32, 1>(p, stream);
}

}  // extern "C"
