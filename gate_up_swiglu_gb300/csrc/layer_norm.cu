// layer_norm.cu -- host side of the layer norm: argument checks, the plan (pack
// width, threads a row, row groups) and the launches.  The contract is in
// include/swiglu_norm.h, the kernels are in layer_norm.cuh.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "layer_norm.cuh"
#include "moe_host.h"
#include "swiglu_norm.h"

namespace {

using moe::Span;

int elem_bytes(swiglu_dtype_t dt) { return dt == SWIGLU_F32 ? 4 : dt == SWIGLU_BF16 ? 2 : 0; }

swiglu_status_t status_of(cudaError_t e) { return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e); }

// Elements of an aligned pack: 16 bytes if n, the strides (elements) and the addresses
// allow it in every row (parameters: the same columns, aligned for it), else one.
int pick_vec(int eb, int pb, int64_t n, std::initializer_list<int64_t> strides, std::initializer_list<const void *> data,
             std::initializer_list<const void *> params) {
    const int vec = 16 / eb;
    bool ok = n % vec == 0;
    for (int64_t s : strides) ok = ok && s % vec == 0;
    for (const void *p : data) ok = ok && (uintptr_t)p % 16 == 0;
    for (const void *p : params) ok = ok && (uintptr_t)p % (uintptr_t)(vec * pb) == 0;
    return ok ? vec : 1;
}

// Elements of a row that a thread holds; the backward has two sums a column beside.
constexpr int held_fwd(int eb, int vec) { return eb == 2 && vec > 1 ? 32 : 16; }
constexpr int kHeldBwd = 16;

constexpr int kMaxDevices = 64;

cudaError_t device(int &dev, int &sms) {
    static std::atomic<int> known[kMaxDevices];
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && (sms = known[dev].load()) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) known[dev].store(sms);
    return e;
}

// The most dynamic shared memory that any launch of the kernel asks for, allowed once
// per device.
template <auto kernel>
cudaError_t allow_smem(int dev, int bytes) {
    static std::atomic<bool> done[kMaxDevices];
    if (dev >= 0 && dev < kMaxDevices && done[dev].load()) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true);
    return e;
}

// Shared memory of an SM for rings (of 228 KB; a CTA has 1 KB and its barriers beside).
constexpr int kRingBytes = 212 * 1024;

// A ring slot for a row of n elements at any address, in whole 16-byte pieces.  `any`:
// with the piece behind the row that a shifted pack may touch.
int64_t slot_of(int64_t n, int eb, bool any) { return (n * eb + 30) / 16 * 16 + (any ? 16 : 0); }

// The number of rows after which rows with these strides (elements) lie as before within
// 16 bytes: a power of two, 16 / eb at most.
int period_of(int eb, std::initializer_list<int64_t> strides) {
    int period = 1;
    for (int64_t s : strides)
        while (s * eb * period % 16 != 0) period *= 2;
    return period;
}

lnorm::Rows rows_of(const void *p, int64_t rows, int64_t n, int64_t stride, int eb) {
    const uint64_t a = (uint64_t)(uintptr_t)p, z = a + (uint64_t)(((rows - 1) * stride + n) * eb);
    return {(a + 15) & ~15ull, z & ~15ull};
}

// ----------------------------------------------------------------- forward ---

// bf16, and fp32 rows that are not aligned: through the ring.
template <typename E, typename P, int VEC, bool ANY, int G, int kHeld>
swiglu_status_t run_ring(lnorm::FwdParams p, int dev, int sms, swiglu_stream_t stream) {
    constexpr int T = G < 128 ? 128 : G, R = T / G, kPerSm = T >= 512 ? 1 : 512 / T;
    constexpr bool kHold = G < 1024 && P::kBytes * kHeld <= 64;  // registers for the parameters
    constexpr auto kernel = lnorm::layer_norm_fwd_kernel<E, P, VEC, kHeld / VEC, G, T, kHold, ANY>;
    constexpr int kRing = kRingBytes / kPerSm;
    const cudaError_t e = allow_smem<kernel>(dev, kRing);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    p.slot_bytes = (int32_t)slot_of(p.n, E::kBytes, ANY);
    p.slots = (int32_t)std::min<int64_t>(lnorm::kMaxSlots, kRing / (R * (int64_t)p.slot_bytes));
    int64_t ctas = std::min<int64_t>((p.rows + R - 1) / R, (int64_t)sms * kPerSm);
    // a group's rows lie alike within 16 bytes
    if (ANY && ctas * R < p.rows) ctas = std::max<int64_t>(p.period, ctas - ctas % p.period);
    return status_of(moe::launch(kernel, dim3((unsigned)ctas), T, (size_t)R * p.slots * p.slot_bytes, stream, 0, p));
}

// Aligned fp32 rows: two rows a group once that still leaves every SM several groups.
template <typename E, typename P, int VEC, int G, int kHeld>
swiglu_status_t run_rows(const lnorm::FwdParams &p, int sms, swiglu_stream_t stream) {
    constexpr int T = G < 128 ? 128 : G, R = T / G;
    if constexpr (G <= 512)
        if (p.rows >= (int64_t)8 * sms * R)
            return status_of(moe::launch(lnorm::layer_norm_fwd_rows_kernel<E, P, VEC, kHeld / VEC, G, T, 2>,
                                         dim3((unsigned)((p.rows + 2 * R - 1) / (2 * R))), T, 0, stream, 0, p));
    return status_of(moe::launch(lnorm::layer_norm_fwd_rows_kernel<E, P, VEC, kHeld / VEC, G, T, 1>,
                                 dim3((unsigned)((p.rows + R - 1) / R)), T, 0, stream, 0, p));
}

template <typename E, typename P, int VEC, bool ANY, int G, int kHeld = held_fwd(E::kBytes, VEC)>
swiglu_status_t run_fwd(const lnorm::FwdParams &p, int dev, int sms, swiglu_stream_t stream) {
    if constexpr (E::kBytes == 2 || ANY)
        return run_ring<E, P, VEC, ANY, G, kHeld>(p, dev, sms, stream);
    else
        return run_rows<E, P, VEC, G, kHeld>(p, sms, stream);
}

// Threads a row: the fewest that hold it (a warp at least, which then holds less).  ANY:
// packs of rows that start anywhere.
template <typename E, typename P, int VEC, bool ANY>
swiglu_status_t run_fwd_groups(const lnorm::FwdParams &p, int dev, int sms, swiglu_stream_t stream) {
    constexpr int k = held_fwd(E::kBytes, VEC);
    const int64_t n = p.n;
    // fp32 parameters of bf16 rows stay in registers where a thread holds half as much
    // ([8192, 4096] 35.0 us, [8192, 1024] 9.1 us; read again for every row 36.1 and 11.1 us)
    if constexpr (P::kBytes > E::kBytes) {
        constexpr int h = k / 2;
        if (n <= 32 * h / 2) return run_fwd<E, P, VEC, ANY, 32, h / 2>(p, dev, sms, stream);
        if (n <= 32 * h) return run_fwd<E, P, VEC, ANY, 32, h>(p, dev, sms, stream);
        if (n <= 64 * h) return run_fwd<E, P, VEC, ANY, 64, h>(p, dev, sms, stream);
        if (n <= 128 * h) return run_fwd<E, P, VEC, ANY, 128, h>(p, dev, sms, stream);
        if (n <= 256 * h) return run_fwd<E, P, VEC, ANY, 256, h>(p, dev, sms, stream);
        if (n <= 512 * h) return run_fwd<E, P, VEC, ANY, 512, h>(p, dev, sms, stream);
        if (ANY || n <= 512 * k) return run_fwd<E, P, VEC, ANY, 512>(p, dev, sms, stream);
        return run_fwd<E, P, VEC, ANY, 1024>(p, dev, sms, stream);
    }
    if (n <= 32 * k / 4) return run_fwd<E, P, VEC, ANY, 32, k / 4>(p, dev, sms, stream);
    if (n <= 32 * k / 2) return run_fwd<E, P, VEC, ANY, 32, k / 2>(p, dev, sms, stream);
    if (n <= 32 * k) return run_fwd<E, P, VEC, ANY, 32>(p, dev, sms, stream);
    if (n <= 64 * k) return run_fwd<E, P, VEC, ANY, 64>(p, dev, sms, stream);
    if (n <= 128 * k) return run_fwd<E, P, VEC, ANY, 128>(p, dev, sms, stream);
    if (n <= 256 * k) return run_fwd<E, P, VEC, ANY, 256>(p, dev, sms, stream);
    if (n <= 512 * k) return run_fwd<E, P, VEC, ANY, 512>(p, dev, sms, stream);
    return run_fwd<E, P, VEC, ANY, 1024>(p, dev, sms, stream);
}

template <typename E, typename P, int VEC>
swiglu_status_t launch_fwd(const lnorm::FwdParams &p, int dev, int sms, swiglu_stream_t stream) {
    constexpr int kPack = 16 / E::kBytes;
    if constexpr (VEC > 1) {
        if (p.n <= 1024 * held_fwd(E::kBytes, VEC)) return run_fwd_groups<E, P, VEC, false>(p, dev, sms, stream);
    } else {
        // (fp32 parameters of long bf16 rows would be read one by one for every row: [1000,
        // 32761] 89 us, in three passes 67 us)
        constexpr int kMost = P::kBytes > E::kBytes ? 512 : 1024;
        if (p.n <= kMost * held_fwd(E::kBytes, kPack)) return run_fwd_groups<E, P, kPack, true>(p, dev, sms, stream);
    }
    return status_of(moe::launch(lnorm::layer_norm_fwd_long_kernel<E, P, VEC, 1024>, dim3((unsigned)p.rows), 1024, 0, stream,
                                 0, p));
}

// ---------------------------------------------------------------- backward ---

// Threads a CTA, one CTA an SM.  With 16 columns a thread, 512 threads have the registers
// they need ([8192, 4096] bf16 41 us and the sums of the groups; 768 threads spill, 67 us;
// 1024 threads of 8 columns 61 us: what a row costs each thread comes more often).
constexpr int kBwdThreads = 512;

constexpr int kMaxCluster = 8;
constexpr int kClusterGroup = 256;  // threads a row of a CTA of a cluster
constexpr int kTileThreads = 128;

struct Plan {
    int G;        // threads a row of a CTA; 0: long rows, in three kernels
    int ctas;     // CTAs a row (a cluster)
    int groups;   // partial rows of column sums, at most
    bool any;     // packs of rows that start anywhere
};

// vec: elements of an aligned pack, or 1 where there are none.  Rows that lie anywhere go in
// packs too, by CTAs that take every period-th row each, unless one CTA takes them all: its
// rows do not lie alike, and it takes them element by element.
Plan plan_bwd(int64_t rows, int64_t n, int vec, int period, int sms) {
    const int k = kHeldBwd;
    const bool any = vec == 1;
    const auto whole = [&](int64_t groups, int most) {
        if (!any) return (int)std::min<int64_t>(groups, most);
        groups = std::min<int64_t>((groups + period - 1) / period * period, most / period * period);
        return (int)std::max<int64_t>(groups, period);
    };
    for (int g : {32, 64, 128, 256, kBwdThreads}) {
        const int64_t per_cta = kBwdThreads / g;  // rows that a CTA takes at a time
        // few rows: one CTA, which needs nobody to add up the column sums
        if (n > (int64_t)g * k) continue;
        if (rows <= 4 * per_cta) return {g, 1, 1, false};
        return {g, 1, whole((rows + per_cta - 1) / per_cta, sms), any};
    }
    // a cluster of 4 or 8 CTAs, with two rows at a time (what two could hold, one does; three
    // would take the room of four)
    // Of eight CTAs too few clusters run at a time to share every eighth row: there rows that
    // lie anywhere go element by element ([1000, 32761] bf16 102 us, in packs 138 us).
    for (int c = 4; c <= kMaxCluster; c *= 2) {
        const int64_t groups = (rows + 1) / 2;
        const int most = std::max(1, sms / c);
        if (n <= (int64_t)kClusterGroup * k * c)
            return c < 8 ? Plan{kClusterGroup, c, whole(groups, most), any}
                         : Plan{kClusterGroup, c, (int)std::min<int64_t>(groups, most), false};
    }
    const int64_t tiles = (n + (int64_t)kTileThreads * vec - 1) / ((int64_t)kTileThreads * vec);
    return {0, 1, (int)std::min<int64_t>(rows, std::max<int64_t>(1, ((int64_t)sms * 8 + tiles - 1) / tiles)), false};
}

int64_t pitch_of(int64_t n) { return (n + 7) / 8 * 8; }

int64_t partial_bytes(const Plan &p, int64_t n) { return p.groups > 1 ? (int64_t)p.groups * 2 * pitch_of(n) * 4 : 0; }

// Of any alignment.
int64_t workspace_bound(int64_t rows, int64_t n, int eb, int sms) {
    int64_t most = 0;
    for (int vec : {16 / eb, 1}) {
        Plan p = plan_bwd(rows, n, vec, 1, sms);
        if (p.any) p.groups = (p.groups + 16 / eb - 1) / (16 / eb) * (16 / eb);  // of any period
        most = std::max(most, partial_bytes(p, n) + (p.G == 0 ? rows * 8 : 0));
    }
    return most;
}

// Clusters of `size` CTAs of the kernel that run at the same time (once per device).
template <auto kernel>
cudaError_t active_clusters(int dev, int size, int smem, int &clusters) {
    static std::atomic<int> known[kMaxDevices][kMaxCluster + 1];
    if (dev >= 0 && dev < kMaxDevices && (clusters = known[dev][size].load()) > 0) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kBwdThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    clusters = std::max(clusters, 1);
    if (dev >= 0 && dev < kMaxDevices) known[dev][size].store(clusters);
    return cudaSuccess;
}

template <typename E, typename P, int VEC, bool ANY, int G, bool CLUSTER>
cudaError_t run_bwd(lnorm::BwdParams &p, const Plan &plan, int dev, swiglu_stream_t stream) {
    constexpr int T = kBwdThreads, kHeld = kHeldBwd, R = T / G, kCols = G * kHeld;
    constexpr auto kernel = lnorm::layer_norm_bwd_kernel<E, P, VEC, kHeld / VEC, G, T, CLUSTER, ANY>;
    static_assert(2 * 2 * (kCols * E::kBytes + 78) * R <= kRingBytes, "two rows a group fit the ring");
    cudaError_t e = allow_smem<kernel>(dev, kRingBytes);
    if (e != cudaSuccess) return e;
    p.slot_bytes = (int32_t)(2 * slot_of(std::min<int64_t>(p.n, kCols + (CLUSTER && ANY ? VEC - 1 : 0)), E::kBytes, ANY));
    p.slots = (int32_t)std::min<int64_t>(lnorm::kMaxSlots, kRingBytes / (R * (int64_t)p.slot_bytes));
    const int64_t fold = (int64_t)(R - 1) * (kCols + (ANY ? G : 0)) * 4, ring = (int64_t)R * p.slots * p.slot_bytes;
    int groups = plan.groups;
    if (CLUSTER) {
        int clusters = 1;
        if ((e = active_clusters<kernel>(dev, plan.ctas, kRingBytes, clusters)) != cudaSuccess) return e;
        groups = std::min(groups, ANY ? std::max(p.period, clusters / p.period * p.period) : clusters);
        p.groups = groups;
    }
    return moe::launch(kernel, dim3((unsigned)(groups * plan.ctas)), T, (size_t)std::max(fold, ring), stream,
                       CLUSTER ? plan.ctas : 0, p);
}

template <typename E, typename P, int VEC, bool ANY>
cudaError_t run_bwd_groups(lnorm::BwdParams &p, const Plan &plan, int dev, swiglu_stream_t stream) {
    if (plan.ctas > 1) return run_bwd<E, P, VEC, ANY, kClusterGroup, true>(p, plan, dev, stream);
    if (plan.G == 32) return run_bwd<E, P, VEC, ANY, 32, false>(p, plan, dev, stream);
    if (plan.G == 64) return run_bwd<E, P, VEC, ANY, 64, false>(p, plan, dev, stream);
    if (plan.G == 128) return run_bwd<E, P, VEC, ANY, 128, false>(p, plan, dev, stream);
    if (plan.G == 256) return run_bwd<E, P, VEC, ANY, 256, false>(p, plan, dev, stream);
    return run_bwd<E, P, VEC, ANY, kBwdThreads, false>(p, plan, dev, stream);
}

template <typename E, typename P, int VEC>
swiglu_status_t launch_bwd(lnorm::BwdParams p, const Plan &plan, int dev, swiglu_stream_t stream) {
    cudaError_t e;
    p.groups = plan.groups;
    if (plan.G == 0) {
        e = moe::launch(lnorm::layer_norm_bwd_sums_kernel<E, P, VEC, 512>, dim3((unsigned)p.rows), 512, 0, stream, 0, p);
        if (e != cudaSuccess) return moe::cuda_fail(e);
        const int64_t tiles = (p.n + (int64_t)kTileThreads * VEC - 1) / ((int64_t)kTileThreads * VEC);
        const dim3 grid((unsigned)tiles, (unsigned)plan.groups);
        e = p.rows > (int64_t)lnorm::kSegment * plan.groups
                ? moe::launch(lnorm::layer_norm_bwd_tile_kernel<E, P, VEC, kTileThreads, true>, grid, kTileThreads, 0, stream, 0, p)
                : moe::launch(lnorm::layer_norm_bwd_tile_kernel<E, P, VEC, kTileThreads, false>, grid, kTileThreads, 0, stream, 0, p);
    } else {
        constexpr int kPack = 16 / E::kBytes;
        if constexpr (VEC == 1)
            e = plan.any ? run_bwd_groups<E, P, kPack, true>(p, plan, dev, stream) : run_bwd_groups<E, P, 1, false>(p, plan, dev, stream);
        else
            e = run_bwd_groups<E, P, VEC, false>(p, plan, dev, stream);
    }
    if (e != cudaSuccess || p.partial == nullptr) return status_of(e);
    return status_of(moe::launch(lnorm::layer_norm_reduce_kernel<P, 16>, dim3((unsigned)((p.n + 31) / 32), 2), 512, 0, stream,
                                 0, p.partial, p.dw, p.db, p.n, p.pitch, p.groups));
}

// Calls f with the types of the data and the parameters and the pack width.
#define NORM_DISPATCH(F, ...)                                                                        \
    (dtype == SWIGLU_F32                                                                             \
         ? (vec > 1 ? F<swiglu::F32, swiglu::F32, 4>(__VA_ARGS__) : F<swiglu::F32, swiglu::F32, 1>(__VA_ARGS__)) \
     : param_dtype == SWIGLU_F32                                                                     \
         ? (vec > 1 ? F<swiglu::BF16, swiglu::F32, 8>(__VA_ARGS__) : F<swiglu::BF16, swiglu::F32, 1>(__VA_ARGS__)) \
         : (vec > 1 ? F<swiglu::BF16, swiglu::BF16, 8>(__VA_ARGS__) : F<swiglu::BF16, swiglu::BF16, 1>(__VA_ARGS__)))

bool types_ok(swiglu_dtype_t dtype, swiglu_dtype_t param_dtype) {
    return elem_bytes(dtype) != 0 && (param_dtype == dtype || param_dtype == SWIGLU_F32);
}

bool sizes_ok(int64_t rows, int64_t n) {
    return rows >= 0 && rows <= SWIGLU_NORM_MAX_ROWS && n >= 0 && n <= SWIGLU_MAX_N;
}

}  // namespace

extern "C" {

swiglu_status_t swiglu_layer_norm_fwd(const void *x, const void *w, const void *b, void *y, float *mean, float *rstd,
                                      int64_t rows, int64_t n, int64_t x_row_stride, int64_t y_row_stride, float eps,
                                      swiglu_dtype_t dtype, swiglu_dtype_t param_dtype, swiglu_stream_t stream) {
    if (!types_ok(dtype, param_dtype)) return SWIGLU_ERR_DTYPE;
    const int eb = elem_bytes(dtype), pb = elem_bytes(param_dtype);
    if (!sizes_ok(rows, n) || !(eps >= 0.0f) || std::isinf(eps)) return SWIGLU_ERR_SHAPE;
    if (rows == 0 || n == 0) return SWIGLU_OK;
    if (x == nullptr || y == nullptr) return SWIGLU_ERR_NULL;
    if (x_row_stride < n || y_row_stride < n) return SWIGLU_ERR_STRIDE;
    Span sx, sw, sb, sy, sm, sr;
    if (!moe::span_of(x, rows, n, x_row_stride, eb, sx) || !moe::span_of(y, rows, n, y_row_stride, eb, sy) ||
        !moe::span_of(w, 1, n, n, pb, sw) || !moe::span_of(b, 1, n, n, pb, sb) ||
        !moe::span_of(mean, rows, 1, 1, 4, sm) || !moe::span_of(rstd, rows, 1, 1, 4, sr))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sy, sm, sr}, {sx, sw, sb})) return SWIGLU_ERR_ALIAS;
    if (((uintptr_t)x | (uintptr_t)y) % eb != 0 || ((uintptr_t)w | (uintptr_t)b) % pb != 0 ||
        ((uintptr_t)mean | (uintptr_t)rstd) % 4 != 0)
        return SWIGLU_ERR_STRIDE;
    lnorm::FwdParams p{};
    p.x = static_cast<const char *>(x);
    p.w = static_cast<const char *>(w);
    p.b = static_cast<const char *>(b);
    p.y = static_cast<char *>(y);
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.n = n;
    p.x_stride = x_row_stride * eb;
    p.y_stride = y_row_stride * eb;
    p.eps = eps;
    p.inv_n = (float)(1.0 / (double)n);
    p.period = period_of(eb, {x_row_stride, y_row_stride});
    p.rows_x = rows_of(x, rows, n, x_row_stride, eb);
    int dev = 0, sms = 0;
    const cudaError_t e = device(dev, sms);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    const int vec = pick_vec(eb, pb, n, {x_row_stride, y_row_stride}, {x, y}, {w, b});
    return NORM_DISPATCH(launch_fwd, p, dev, sms, stream);
}

swiglu_status_t swiglu_layer_norm_bwd_workspace_size(int64_t rows, int64_t n, swiglu_dtype_t dtype, size_t *bytes) {
    if (bytes == nullptr) return SWIGLU_ERR_NULL;
    const int eb = elem_bytes(dtype);
    if (eb == 0) return SWIGLU_ERR_DTYPE;
    if (!sizes_ok(rows, n)) return SWIGLU_ERR_SHAPE;
    *bytes = 0;
    if (rows == 0 || n == 0) return SWIGLU_OK;
    int dev = 0, sms = 0;
    const cudaError_t e = device(dev, sms);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    *bytes = (size_t)workspace_bound(rows, n, eb, sms);
    return SWIGLU_OK;
}

swiglu_status_t swiglu_layer_norm_bwd(const void *dy, const void *x, const float *mean, const float *rstd, const void *w,
                                      void *dx, void *dw, void *db, void *workspace, size_t workspace_bytes, int64_t rows,
                                      int64_t n, int64_t dy_row_stride, int64_t x_row_stride, int64_t dx_row_stride,
                                      swiglu_dtype_t dtype, swiglu_dtype_t param_dtype, swiglu_stream_t stream) {
    if (!types_ok(dtype, param_dtype)) return SWIGLU_ERR_DTYPE;
    const int eb = elem_bytes(dtype), pb = elem_bytes(param_dtype);
    if (!sizes_ok(rows, n)) return SWIGLU_ERR_SHAPE;
    if (n == 0) return SWIGLU_OK;
    if (((uintptr_t)w | (uintptr_t)dw | (uintptr_t)db) % pb != 0) return SWIGLU_ERR_STRIDE;
    if (rows == 0) {  // sums over no rows
        for (void *p : {dw, db})
            if (p != nullptr) {
                const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)n * pb, reinterpret_cast<cudaStream_t>(stream));
                if (e != cudaSuccess) return moe::cuda_fail(e);
            }
        return SWIGLU_OK;
    }
    if (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr) return SWIGLU_ERR_NULL;
    if (dy_row_stride < n || x_row_stride < n || dx_row_stride < n) return SWIGLU_ERR_STRIDE;
    Span sdy, sx, sm, sr, sw, sdx, sdw, sdb, sws;
    if (!moe::span_of(dy, rows, n, dy_row_stride, eb, sdy) || !moe::span_of(x, rows, n, x_row_stride, eb, sx) ||
        !moe::span_of(dx, rows, n, dx_row_stride, eb, sdx) || !moe::span_of(w, 1, n, n, pb, sw) ||
        !moe::span_of(dw, 1, n, n, pb, sdw) || !moe::span_of(db, 1, n, n, pb, sdb) ||
        !moe::span_of(mean, rows, 1, 1, 4, sm) || !moe::span_of(rstd, rows, 1, 1, 4, sr))
        return SWIGLU_ERR_SHAPE;
    if (((uintptr_t)dy | (uintptr_t)x | (uintptr_t)dx) % eb != 0 || ((uintptr_t)mean | (uintptr_t)rstd) % 4 != 0)
        return SWIGLU_ERR_STRIDE;
    if (moe::any_alias({sdx, sdw, sdb}, {sdy, sx, sm, sr, sw})) return SWIGLU_ERR_ALIAS;
    int dev = 0, sms = 0;
    const cudaError_t e = device(dev, sms);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    const int64_t need = workspace_bound(rows, n, eb, sms);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < (size_t)need || (uintptr_t)workspace % 16 != 0)
            return SWIGLU_ERR_WORKSPACE;
        if (!moe::span_of(workspace, 1, need, need, 1, sws)) return SWIGLU_ERR_SHAPE;
        if (moe::any_alias({sws}, {sdy, sx, sm, sr, sw, sdx, sdw, sdb})) return SWIGLU_ERR_ALIAS;
    }
    const int vec = pick_vec(eb, pb, n, {dy_row_stride, x_row_stride, dx_row_stride}, {dy, x, dx}, {w});
    lnorm::BwdParams p{};
    p.period = period_of(eb, {dy_row_stride, x_row_stride, dx_row_stride});
    const Plan plan = plan_bwd(rows, n, vec, p.period, sms);
    p.dy = static_cast<const char *>(dy);
    p.x = static_cast<const char *>(x);
    p.w = static_cast<const char *>(w);
    p.mean = mean;
    p.rstd = rstd;
    p.dx = static_cast<char *>(dx);
    p.dw = static_cast<char *>(dw);
    p.db = static_cast<char *>(db);
    p.rows = rows;
    p.n = n;
    p.pitch = pitch_of(n);
    p.dy_stride = dy_row_stride * eb;
    p.x_stride = x_row_stride * eb;
    p.dx_stride = dx_row_stride * eb;
    p.inv_n = (float)(1.0 / (double)n);
    char *at = static_cast<char *>(workspace);
    if (plan.groups > 1 && (dw != nullptr || db != nullptr)) p.partial = reinterpret_cast<float *>(at);
    if (plan.G == 0) p.sums = reinterpret_cast<float *>(at + partial_bytes(plan, n));
    p.rows_x = rows_of(x, rows, n, x_row_stride, eb);
    p.rows_dy = rows_of(dy, rows, n, dy_row_stride, eb);
    return NORM_DISPATCH(launch_bwd, p, plan, dev, stream);
}

swiglu_status_t swiglu_layer_norm_timeout_flag(int *flag) {
    if (flag == nullptr) return SWIGLU_ERR_NULL;
    const cudaError_t e = cudaMemcpyFromSymbol(flag, lnorm::g_norm_timeout, sizeof(int));
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

}  // extern "C"
