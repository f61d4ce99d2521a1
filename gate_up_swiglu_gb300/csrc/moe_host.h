// moe_host.h -- host-side helpers of the routed experts' translation units
// (ckpt8.cu, grouped_mm.cu): byte spans for the overlap checks and the launch.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <utility>

#include "abi_internal.h"
#include "swiglu_moe.h"

namespace moe {

inline swiglu_status_t cuda_fail(cudaError_t e) {
    swiglu_abi::record_cuda_error((int)e);
    return SWIGLU_ERR_CUDA;
}

// Byte extent [lo, hi) of a [rows, cols] tensor (rows, cols >= 1); `p` NULL
// gives the empty span, which overlaps nothing.
struct Span {
    uintptr_t lo = 0, hi = 0;
};

inline bool span_of(const void *p, int64_t rows, int64_t cols, int64_t stride, int eb, Span &s) {
    s = {};
    int64_t last, elems, bytes;
    if (__builtin_mul_overflow(rows - 1, stride, &last)) return false;
    if (__builtin_add_overflow(last, cols, &elems)) return false;
    if (__builtin_mul_overflow(elems, (int64_t)eb, &bytes)) return false;
    if (p == nullptr) return true;
    const uintptr_t lo = (uintptr_t)p;
    if (lo + (uintptr_t)bytes < lo) return false;
    s = {lo, lo + (uintptr_t)bytes};
    return true;
}

inline bool overlaps(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }

// True when an output overlaps an input or another output.
inline bool any_alias(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span *a = outs.begin(); a != outs.end(); ++a) {
        for (const Span &b : ins)
            if (overlaps(*a, b)) return true;
        for (const Span *b = a + 1; b != outs.end(); ++b)
            if (overlaps(*a, *b)) return true;
    }
    return false;
}

// Launch with programmatic stream serialization: the kernel may launch while
// the previous kernel in the stream finishes, and waits for that kernel's
// completion itself before its first global memory access.  cluster > 0: in
// clusters of that many CTAs (0: as the kernel is declared).
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem, swiglu_stream_t stream,
                   int cluster, Args &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace moe
