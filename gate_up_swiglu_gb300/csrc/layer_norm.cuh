// layer_norm.cuh -- device code of the layer norm in front of linear_fc1 and of
// its backward pass (the contract is in swiglu_norm.h).
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   xhat = (x - mean) rstd,  y = xhat w + b
//   h = dy w,  dx = rstd (h - mean(h) - xhat mean(h xhat))
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// The forward reads x and writes y, the backward reads dy and x and writes dx: 2 and 3
// elements of HBM traffic for some 13 and 21 instructions an element (bf16), so both are bound
// by HBM as long as a row is read once and the memory never waits for a row's sums.  So a
// group of G threads (a warp up to a CTA) holds a row in registers, and in the backward
// and the bf16 forward the CTAs are persistent and rows come by bulk copies into a ring in
// shared memory, issued several rows ahead by one thread of the group.
//
// Backward, [8192, 4096]: bf16 42 us (71 % of the copy rate; what is left is the time that
// two rows an SM leave its schedulers idle at their sums), fp32 66 us (89 %).
//
// Rows of any length, stride and address (ANY) go in 16-byte packs too: those that lie
// aligned in the result's row, with single columns in front of them and behind them; x and
// dy are shifted to them on the way from the ring.  Rows a few apart lie alike within 16
// bytes (`period`), and a group takes only such rows, so that its columns, parameters and
// column sums stay the same.  [8192, 4095] bf16: forward 26 us, element by element 54 us;
// backward 49 us, 72 us.  fp32 backward 70 us, 71 us; [8192, 5503] 89 us, 98 us.
#pragma once

#include <stdint.h>

#include "load_after.cuh"
#include "swiglu_kernels.cuh"
#include "tc_pair.cuh"

namespace lnorm {

using swiglu::BF16;
using swiglu::F32;

// Barrier of the G threads of group `g` of a CTA.
template <int G, int T>
__device__ __forceinline__ void group_barrier(int g) {
    if constexpr (G == T)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(G) : "memory");
}

// Sums of N values (1, 2 or 4) over the G threads of group `g`, the same bits in every
// thread.  Within a warp N - 1 exchanges leave each lane with one of the values, so
// that the rest of the tree is one shuffle a level; the warps meet in `at` (N * G / 32
// floats of shared memory, 16-byte aligned where that is a multiple of 4, not used
// again before another barrier of the group).
template <int G, int T, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float *at, int g) {
    const int lane = threadIdx.x & 31;
    float s;
    if constexpr (N == 4) {
        const bool hi = lane & 16;
        float a = hi ? v[2] : v[0], b = hi ? v[3] : v[1];
        a += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
        b += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
        const bool odd = lane & 8;
        s = odd ? b : a;
        s += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
    } else if constexpr (N == 2) {
        const bool hi = lane & 16;
        s = hi ? v[1] : v[0];
        s += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 16);
    } else {
        s = v[0];
        s += __shfl_xor_sync(0xffffffffu, s, 16);
    }
    if constexpr (N < 4) s += __shfl_xor_sync(0xffffffffu, s, 8);
#pragma unroll
    for (int d = 4; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    constexpr int L = 32 / N;  // value k is in lanes k L and on
    if constexpr (G == 32) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = N == 1 ? s : __shfl_sync(0xffffffffu, s, k * L);
    } else {
        constexpr int W = G / 32;
        if (lane % L == 0) at[(lane / L) * W + (threadIdx.x % G >> 5)] = s;
        group_barrier<G, T>(g);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float t = 0.0f;
            if constexpr (W % 4 == 0) {
#pragma unroll
                for (int w = 0; w < W; w += 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(at + k * W + w);
                    t += (q.x + q.y) + (q.z + q.w);
                }
            } else {
#pragma unroll
                for (int w = 0; w < W; ++w) t += at[k * W + w];
            }
            v[k] = t;
        }
    }
}

template <int B>
__device__ __forceinline__ void load_once(const char *p, uint32_t *w) {
    swiglu::load_after<B, false>(p, w);
}

template <int B>
__device__ __forceinline__ void load_words(const char *p, uint32_t *w) {
    constexpr int S = B > 32 ? 32 : B;
#pragma unroll
    for (int k = 0; k < B; k += S) swiglu::load_after<S, true>(p + k, w + k / 4);
}

// VEC parameters (weight or bias, reread by every row: kept in L1).
template <typename P, int VEC>
__device__ __forceinline__ void load_params(const char *p, int64_t col, float *v) {
    constexpr int B = P::kBytes * VEC;
    uint32_t w[B < 4 ? 1 : B / 4];
    load_words<B>(p + col * P::kBytes, w);
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = P::get(w, k);
}

// 1 / sqrt(var + eps) from sum (x - m0)^2 / n and the mean dm of x - m0 (a variance
// is not negative; NaN stays).
__device__ __forceinline__ float inverse_std(float sq, float dm, float eps) {
    const float var = fmaf(-dm, dm, sq);
    return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);
}

// VEC results to `dst`, rounded once.
template <typename E, int VEC>
__device__ __forceinline__ void store_once(char *dst, const float *v) {
    constexpr int B = E::kBytes * VEC;
    uint32_t o[B < 4 ? 1 : B / 4] = {};
    if constexpr (VEC == 1)
        E::put(o, 0, v[0]);
    else
#pragma unroll
        for (int k = 0; k < VEC; k += 2) E::put2(o, k, v[k], v[k + 1]);
    swiglu::St<B, swiglu::kStStream>::run(dst, o);
}

// Element pairs of a row: two lanes of fp32 arithmetic an instruction.
__device__ __forceinline__ uint64_t twice(float v) { return swiglu::x2(v, v); }
__device__ __forceinline__ float both(uint64_t v) {
    float lo, hi;
    swiglu::x2_split(v, lo, hi);
    return lo + hi;
}

// Elements 2 i and 2 i + 1 of C packs of VEC (in the order of packs).
template <typename E, int VEC, int C, int WN>
__device__ __forceinline__ uint64_t pair_of(const uint32_t (&w)[C][WN], int i) {
    return swiglu::x2(E::get(w[2 * i / VEC], 2 * i % VEC), E::get(w[(2 * i + 1) / VEC], (2 * i + 1) % VEC));
}

// ------------------------------------------------------------------- ring ---

__device__ int g_norm_timeout = 0;

constexpr int kMaxSlots = 8;

// A tensor's rows as the ring copies them: bytes [lo, hi) of the whole tensor rounded
// inwards to 16, beyond which no copy reaches.
struct Rows {
    uint64_t lo, hi;
};

// The part of a row (`bytes` from `row` on) that is copied, in whole 16-byte pieces: its
// pieces at the ends too, unless they reach out of the tensor.
__device__ __forceinline__ void copied(const Rows &t, const char *row, int64_t bytes, uint64_t &lo, uint64_t &hi) {
    const uint64_t a = reinterpret_cast<uint64_t>(row), z = a + (uint64_t)bytes;
    lo = a & ~(uint64_t)15;
    hi = (z + 15) & ~(uint64_t)15;
    if (lo < t.lo) lo = t.lo;
    if (hi > t.hi) hi = t.hi;
}

template <int B>
__device__ __forceinline__ void store_shared(uint32_t addr, uint32_t v) {
    if constexpr (B == 4)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
    else
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"((unsigned short)v) : "memory");
}

// The bytes of the row that its copy will bring, which a thread announces on a barrier.
// What the copy leaves out (of the tensor's first and last rows) the thread itself puts to
// `dst` + (address of the row) % 16 before that.
template <typename E>
__device__ __forceinline__ uint32_t prepare_row(const Rows &t, const char *row, int64_t bytes, uint32_t dst) {
    uint64_t lo, hi;
    copied(t, row, bytes, lo, hi);
    const uint64_t a = reinterpret_cast<uint64_t>(row), z = a + (uint64_t)bytes;
    if (lo > a || hi < z) {
        const auto put = [&](uint64_t from, uint64_t to) {
            for (uint64_t e = from; e < to; e += E::kBytes) {
                uint32_t w[1];
                swiglu::load_after<E::kBytes, false>(reinterpret_cast<const char *>(e), w);
                store_shared<E::kBytes>(dst + (uint32_t)(e - (a & ~(uint64_t)15)), w[0]);
            }
        };
        const uint64_t m = max(a, min(lo, z));
        put(a, m);
        put(max(hi, m), z);
        tc::fence_async_shared();
    }
    return hi > lo ? (uint32_t)(hi - lo) : 0u;
}
__device__ __forceinline__ void copy_row(const Rows &t, const char *row, int64_t bytes, uint32_t dst, uint32_t bar) {
    uint64_t lo, hi;
    copied(t, row, bytes, lo, hi);
    if (hi <= lo) return;
    const uint32_t skip = (uint32_t)(lo - (reinterpret_cast<uint64_t>(row) & ~15ull));
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst + skip),
                 "l"(lo), "r"((uint32_t)(hi - lo)), "r"(bar)
                 : "memory");
}

template <int B>
__device__ __forceinline__ void load_shared(uint32_t addr, uint32_t *w) {
    if constexpr (B == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
    else if constexpr (B == 4)
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
    else {
        unsigned short h;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
        w[0] = h;
    }
}

// Packs t, t + G, ... of a row in its slot (zeros past it): 16 bytes of rows that are all
// 16-byte aligned, or one element.
template <typename E, int VEC, int G, int C, int WN>
__device__ __forceinline__ void packs(const char *row, uint32_t slot, int t, const bool (&in)[C], uint32_t (&w)[C][WN]) {
    constexpr int B = E::kBytes * VEC;
    const uint32_t first = slot + (VEC == 1 ? (uint32_t)(reinterpret_cast<uint64_t>(row) & 15) : 0u) + (uint32_t)(t * B);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int k = 0; k < WN; ++k) w[c][k] = 0;
        if (in[c]) load_shared<B>(first + c * G * B, w[c]);
    }
}

// The columns of a thread.  The result's row starts `lead` columns behind 16 bytes; its
// aligned packs go to the threads in turn, and the single columns in front of them and
// behind them one to a thread of the first warp.
template <int VEC, int G>
struct Columns {
    int32_t t, head, packs, single;  // single: -1 for none

    __device__ __forceinline__ Columns(int thread, int lead, int64_t cols) : t(thread) {
        const int n = (int)cols;
        head = min(n, (VEC - lead) & (VEC - 1));
        packs = (n - head) / VEC;
        const int tail = n - head - packs * VEC;
        single = t < head ? t : t - head < tail ? t + packs * VEC : -1;
    }
    __device__ __forceinline__ bool in(int c) const { return t + c * G < packs; }
    __device__ __forceinline__ int32_t col(int c) const { return head + (t + c * G) * VEC; }
};

// A thread's packs of a row that lies anywhere in its slot (`dst` of copy_row), each shifted
// out of two aligned pieces, and its single column (zeros for what it does not have).
template <typename E, int VEC, int G, int C, int WN>
__device__ __forceinline__ float shifted_packs(const char *row, uint32_t slot, const Columns<VEC, G> &cols,
                                               uint32_t (&w)[C][WN]) {
    static_assert(WN == 4, "packs of 16 bytes");
    const uint32_t first = slot + (uint32_t)(reinterpret_cast<uint64_t>(row) & 15);
    const uint32_t start = first + (uint32_t)(cols.col(0) * E::kBytes), off = start & 15;
    uint32_t one[1] = {0};
    if (cols.t < 32 && cols.single >= 0) load_shared<E::kBytes>(first + (uint32_t)(cols.single * E::kBytes), one);
    if (off == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[c][k] = 0;
            if (cols.in(c)) load_shared<16>(start + c * G * 16, w[c]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t r[8] = {};
            if (cols.in(c)) {
                load_shared<16>((start & ~15u) + c * G * 16, r);
                load_shared<16>((start & ~15u) + c * G * 16 + 16, r + 4);
            }
#pragma unroll
            for (int k = 0; k < 6; ++k) r[k] = off & 8 ? r[k + 2] : r[k];
#pragma unroll
            for (int k = 0; k < 5; ++k) r[k] = off & 4 ? r[k + 1] : r[k];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[c][k] = E::kBytes == 2 ? __funnelshift_r(r[k], r[k + 1], (off & 2) * 8) : r[k];
        }
    }
    return E::get(one, 0);
}

// VEC parameters from any column on.
template <typename P, int VEC, int PN>
__device__ __forceinline__ void load_elements(const char *p, int64_t col, uint32_t (&w)[PN]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        uint32_t v[1];
        swiglu::load_after<P::kBytes, true>(p + (col + k) * P::kBytes, v);
        if constexpr (P::kBytes == 4)
            w[k] = v[0];
        else
            w[k / 2] = k % 2 ? w[k / 2] | v[0] << 16 : v[0];
    }
}

template <typename P>
__device__ __forceinline__ float load_param(const char *p, int64_t col) {
    uint32_t v[1];
    swiglu::load_after<P::kBytes, true>(p + col * P::kBytes, v);
    return P::get(v, 0);
}

__device__ __forceinline__ bool row_arrived(uint32_t bar, uint32_t parity) {
    return tc::mbar_wait_or_flag<false>(bar, parity, &g_norm_timeout);
}

struct FwdParams {
    Rows rows_x;
    int32_t slots, slot_bytes;
    int32_t period;  // rows so far apart lie alike within 16 bytes (host)
    const char *x;
    const char *w, *b;  // or NULL
    char *y;
    float *mean, *rstd;  // or NULL
    int64_t rows, n;
    int64_t x_stride, y_stride;  // bytes
    float eps, inv_n;
};

template <typename P, int VEC>
__device__ __forceinline__ void affine(const FwdParams &p, int64_t col, float *v) {
    float q[VEC];
    if (p.w != nullptr) {
        load_params<P, VEC>(p.w, col, q);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] *= q[k];
    }
    if (p.b != nullptr) {
        load_params<P, VEC>(p.b, col, q);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] += q[k];
    }
}

// The mean is found in two steps: m0 = sum x / n as computed, then the mean of x - m0,
// which carries m0's rounding error; so a large common offset costs nothing.
//
// HOLD: the thread's parameters stay in registers over its rows (else they are read
// again for each row, from L2: the ring leaves L1 little).
//
// bf16 rows come this way ([8192, 4096] 23 us, 86 % of the copy rate; read straight to
// registers, as below, 28 us), and fp32 rows that are not aligned ([3000, 5503] 31 us, read
// straight to registers 32 us in packs, 34 us element by element).
template <typename E, typename P, int VEC, int C, int G, int T, bool HOLD, bool ANY>
__global__ void __launch_bounds__(T, T >= 512 ? 1 : 512 / T) layer_norm_fwd_kernel(const __grid_constant__ FwdParams p) {
    constexpr int EB = E::kBytes, B = EB * VEC, WN = B < 4 ? 1 : B / 4, N = C * VEC / 2;  // pairs a row
    constexpr int W = G / 32, R = T / G;
    constexpr int PB = P::kBytes * VEC, PN = PB < 4 ? 1 : PB / 4;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(16) float part[R][3 * W];  // the two sums' own places
    __shared__ __align__(8) uint64_t full[R][kMaxSlots];
    const int t = threadIdx.x % G, g = threadIdx.x / G;
    if (threadIdx.x < R * kMaxSlots) tc::mbar_init(tc::smem_addr(&full[0][0] + threadIdx.x), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    const int64_t step = (int64_t)gridDim.x * R, bytes = p.n * EB;
    int64_t row = (int64_t)blockIdx.x * R + g;
    const uint32_t slot0 = tc::smem_addr(ring) + (uint32_t)g * p.slots * p.slot_bytes, bar0 = tc::smem_addr(&full[g][0]);
    const auto issue = [&](int64_t r, int slot) {
        const char *src = p.x + r * p.x_stride;
        const uint32_t at = slot0 + slot * p.slot_bytes;
        tc::mbar_arrive_expect_tx(bar0 + 8 * slot, prepare_row<E>(p.rows_x, src, bytes, at));
        copy_row(p.rows_x, src, bytes, at, bar0 + 8 * slot);
    };
    if (t == 0)
        for (int k = 0; k < p.slots && row + k * step < p.rows; ++k) issue(row + k * step, k);
    const int lead = ANY ? (int)((reinterpret_cast<uint64_t>(p.y) + (uint64_t)(row * p.y_stride)) & 15) / EB : 0;
    const Columns<VEC, G> cols(t, lead, p.n);
    bool in[C];
    float w1 = 1.0f, b1 = 0.0f;  // of the single column
    if constexpr (ANY) {
        if (cols.single >= 0 && p.w != nullptr) w1 = load_param<P>(p.w, cols.single);
        if (cols.single >= 0 && p.b != nullptr) b1 = load_param<P>(p.b, cols.single);
    }
    uint32_t pw[HOLD ? C : 1][PN], pb[HOLD ? C : 1][PN];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        in[c] = cols.in(c);
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < PN; ++k) {
                pw[c][k] = P::kBytes == 4 ? 0x3f800000u : 0x3f803f80u;  // ones
                pb[c][k] = 0;
            }
            if constexpr (ANY) {
                if (in[c] && p.w != nullptr) load_elements<P, VEC>(p.w, cols.col(c), pw[c]);
                if (in[c] && p.b != nullptr) load_elements<P, VEC>(p.b, cols.col(c), pb[c]);
            } else {
                if (in[c] && p.w != nullptr) load_words<PB>(p.w + (int64_t)(t + c * G) * PB, pw[c]);
                if (in[c] && p.b != nullptr) load_words<PB>(p.b + (int64_t)(t + c * G) * PB, pb[c]);
            }
        }
    }
    const bool whole = in[C - 1];  // no column of this thread lies past the row
    int slot = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (; row < p.rows; row += step) {
        ok = ok && row_arrived(bar0 + 8 * slot, parity);  // one that ran out is not waited for again
        uint32_t raw[C][WN];
        float x1 = 0.0f;  // the single column's
        if constexpr (ANY) {
            x1 = shifted_packs<E>(p.x + row * p.x_stride, slot0 + slot * p.slot_bytes, cols, raw);
        } else {
            packs<E, VEC, G>(p.x + row * p.x_stride, slot0 + slot * p.slot_bytes, t, in, raw);
        }
        uint64_t d[N], a = 0, q = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            d[i] = pair_of<E, VEC, C>(raw, i);
            a = swiglu::add_x2(a, d[i]);
        }
        float m0[1] = {ANY ? both(a) + x1 : both(a)};
        group_sum<G, T, 1>(m0, part[g], g);
        // every thread of the group has read the row: its slot takes the next one
        if constexpr (G == 32) __syncwarp();
        if (t == 0 && ok && row + p.slots * step < p.rows) issue(row + p.slots * step, slot);
        if (++slot == p.slots) {
            slot = 0;
            parity ^= 1;
        }
        m0[0] *= p.inv_n;
        const uint64_t m = twice(m0[0]);
        a = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = swiglu::sub_x2(d[i], m);
        if (!whole) {  // columns past the row count as the mean
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float lo, hi;
                swiglu::x2_split(d[i], lo, hi);
                d[i] = swiglu::x2(in[2 * i / VEC] ? lo : 0.0f, in[(2 * i + 1) / VEC] ? hi : 0.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a = swiglu::add_x2(a, d[i]);
            q = swiglu::fma_x2(d[i], d[i], q);
        }
        float s[2] = {both(a), both(q)};
        if constexpr (ANY) {
            x1 = t < 32 && cols.single >= 0 ? x1 - m0[0] : 0.0f;
            s[0] += x1;
            s[1] = fmaf(x1, x1, s[1]);
        }
        group_sum<G, T, 2>(s, part[g] + W, g);
        const float dm = s[0] * p.inv_n, rstd = inverse_std(s[1] * p.inv_n, dm, p.eps);
        if (t == 0) {
            if (p.mean != nullptr) p.mean[row] = m0[0] + dm;
            if (p.rstd != nullptr) p.rstd[row] = rstd;
        }
        const uint64_t scale = twice(rstd), shift = twice(-dm * rstd);  // xhat = d rstd - dm rstd
        char *dst = p.y + row * p.y_stride;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            d[i] = swiglu::fma_x2(d[i], scale, shift);
            if constexpr (HOLD)
                d[i] = swiglu::fma_x2(d[i], pair_of<P, VEC, C>(pw, i), pair_of<P, VEC, C>(pb, i));
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!in[c]) continue;
            const int64_t col = (int64_t)(t + c * G) * VEC;
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float lo, hi;
                swiglu::x2_split(d[(c * VEC + k) / 2], lo, hi);
                v[k] = (c * VEC + k) % 2 ? hi : lo;
            }
            if constexpr (ANY) {
                if constexpr (!HOLD) {
                    uint32_t q[PN];
                    if (p.w != nullptr) {
                        load_elements<P, VEC>(p.w, cols.col(c), q);
#pragma unroll
                        for (int k = 0; k < VEC; ++k) v[k] *= P::get(q, k);
                    }
                    if (p.b != nullptr) {
                        load_elements<P, VEC>(p.b, cols.col(c), q);
#pragma unroll
                        for (int k = 0; k < VEC; ++k) v[k] += P::get(q, k);
                    }
                }
                store_once<E, VEC>(dst + (int64_t)cols.col(c) * EB, v);
            } else {
                if constexpr (!HOLD) affine<P, VEC>(p, col, v);
                store_once<E, VEC>(dst + col * EB, v);
            }
        }
        if (ANY && t < 32) {
            const float v[1] = {fmaf(fmaf(x1, rstd, -dm * rstd), w1, b1)};
            if (cols.single >= 0) store_once<E, 1>(dst + (int64_t)cols.single * EB, v);
        }
    }
    if (!ok && t == 0) tc::settle();  // a wait ran out: no copy lands in shared memory that the CTA has left
}

// Aligned fp32 rows: read straight to registers, R neighbouring rows a group (the same columns in
// each thread, so that w and b are read once for all of them), as many CTAs as there are
// rows.  An fp32 row has half the instructions a byte of a bf16 one, and CTAs that start in
// the order of their addresses keep DRAM's window small: [8192, 4096] 41 us (97 % of the
// copy rate) against 48 us through the ring.
template <typename E, typename P, int VEC, int C, int G, int T, int R>
__global__ void __launch_bounds__(T) layer_norm_fwd_rows_kernel(const __grid_constant__ FwdParams p) {
    constexpr int EB = E::kBytes, B = EB * VEC, WN = B < 4 ? 1 : B / 4, N = C * VEC / 2;  // pairs a row
    constexpr int W = G / 32;
    __shared__ __align__(16) float part[T / G][3 * R * W];  // the two sums' own places
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    const int t = threadIdx.x % G, g = threadIdx.x / G;
    const int64_t row0 = ((int64_t)blockIdx.x * (T / G) + g) * R;
    if (row0 >= p.rows) return;  // the whole group
    bool in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = (int64_t)(t + c * G) * VEC < p.n;
    uint32_t raw[R][C][WN];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int k = 0; k < WN; ++k) raw[r][c][k] = 0;
            if (in[c] && row0 + r < p.rows)
                load_once<B>(p.x + (row0 + r) * p.x_stride + (int64_t)(t + c * G) * B, raw[r][c]);
        }
    float m0[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint64_t a = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) a = swiglu::add_x2(a, pair_of<E, VEC, C>(raw[r], i));
        m0[r] = both(a);
    }
    group_sum<G, T, R>(m0, part[g], g);
    uint64_t d[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m0[r] *= p.inv_n;
        const uint64_t m = twice(m0[r]);
        uint64_t a = 0, q = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float lo, hi;
            swiglu::x2_split(swiglu::sub_x2(pair_of<E, VEC, C>(raw[r], i), m), lo, hi);
            // columns past the row count as the mean
            d[r][i] = swiglu::x2(in[2 * i / VEC] ? lo : 0.0f, in[(2 * i + 1) / VEC] ? hi : 0.0f);
            a = swiglu::add_x2(a, d[r][i]);
            q = swiglu::fma_x2(d[r][i], d[r][i], q);
        }
        s[2 * r] = both(a);
        s[2 * r + 1] = both(q);
    }
    group_sum<G, T, 2 * R>(s, part[g] + R * W, g);
    float scale[R], shift[R];  // xhat = d rstd - dm rstd
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float dm = s[2 * r] * p.inv_n;
        scale[r] = inverse_std(s[2 * r + 1] * p.inv_n, dm, p.eps);
        shift[r] = -dm * scale[r];
        if (t == 0 && row0 + r < p.rows) {
            if (p.mean != nullptr) p.mean[row0 + r] = m0[r] + dm;
            if (p.rstd != nullptr) p.rstd[row0 + r] = scale[r];
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (!in[c]) continue;
        const int64_t col = (int64_t)(t + c * G) * VEC;
        float w[VEC], b[VEC];
        if (p.w != nullptr) load_params<P, VEC>(p.w, col, w);
        if (p.b != nullptr) load_params<P, VEC>(p.b, col, b);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= p.rows) continue;
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float lo, hi;
                swiglu::x2_split(d[r][(c * VEC + k) / 2], lo, hi);
                v[k] = fmaf((c * VEC + k) % 2 ? hi : lo, scale[r], shift[r]);
                if (p.w != nullptr) v[k] *= w[k];
                if (p.b != nullptr) v[k] += b[k];
            }
            store_once<E, VEC>(p.y + (row0 + r) * p.y_stride + col * EB, v);
        }
    }
}

// Rows too long for a CTA's registers: three passes, of which the last two find the
// row in L2.
template <typename E, typename P, int VEC, int T>
__global__ void __launch_bounds__(T) layer_norm_fwd_long_kernel(FwdParams p) {
    constexpr int EB = E::kBytes, B = EB * VEC, WN = B < 4 ? 1 : B / 4;
    __shared__ __align__(16) float part[3 * (T / 32)];
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const char *src = p.x + row * p.x_stride;
        float m0[1] = {0.0f}, s[2] = {0.0f, 0.0f};
#pragma unroll 4
        for (int64_t col = (int64_t)threadIdx.x * VEC; col < p.n; col += (int64_t)T * VEC) {
            uint32_t w[WN];
            load_once<B>(src + col * EB, w);
            float a = 0.0f;
#pragma unroll
            for (int k = 0; k < VEC; ++k) a += E::get(w, k);
            m0[0] += a;
        }
        group_sum<T, T, 1>(m0, part, 0);
        m0[0] *= p.inv_n;
#pragma unroll 4
        for (int64_t col = (int64_t)threadIdx.x * VEC; col < p.n; col += (int64_t)T * VEC) {
            uint32_t w[WN];
            load_once<B>(src + col * EB, w);
            float a = 0.0f, q = 0.0f;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float d = E::get(w, k) - m0[0];
                a += d;
                q = fmaf(d, d, q);
            }
            s[0] += a;
            s[1] += q;
        }
        group_sum<T, T, 2>(s, part + T / 32, 0);
        const float dm = s[0] * p.inv_n;
        const float rstd = inverse_std(s[1] * p.inv_n, dm, p.eps);
        if (threadIdx.x == 0) {
            if (p.mean != nullptr) p.mean[row] = m0[0] + dm;
            if (p.rstd != nullptr) p.rstd[row] = rstd;
        }
        char *dst = p.y + row * p.y_stride;
#pragma unroll 2
        for (int64_t col = (int64_t)threadIdx.x * VEC; col < p.n; col += (int64_t)T * VEC) {
            uint32_t w[WN];
            load_once<B>(src + col * EB, w);
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = ((E::get(w, k) - m0[0]) - dm) * rstd;
            affine<P, VEC>(p, col, v);
            store_once<E, VEC>(dst + col * EB, v);
        }
    }
}

// ---------------------------------------------------------------- backward ---
struct BwdParams {
    Rows rows_x, rows_dy;
    int32_t slots, slot_bytes;
    const char *dy, *x, *w;  // w or NULL
    const float *mean, *rstd;
    char *dx;
    char *dw, *db;    // final sums of P, written by the kernel itself when it is one CTA
    float *partial;   // [groups][2][pitch]: sums of dy xhat, then of dy; NULL: no gradient of either
    float *sums;      // [rows][2]: mean(h), mean(h xhat); long rows only
    int64_t rows, n, pitch;
    int32_t groups;   // of partial sums (host)
    int32_t period;   // rows so far apart lie alike within 16 bytes
    int64_t dy_stride, x_stride, dx_stride;  // bytes
    float inv_n;
};

// dy, x and w as fp32 to xhat and h.
template <typename E, int VEC>
__device__ __forceinline__ void unpack(const uint32_t *xw, const uint32_t *dw, float mean, float rstd, int k, float &xhat,
                                       float &dy) {
    xhat = (E::get(xw, k) - mean) * rstd;
    dy = E::get(dw, k);
}

template <typename P>
__device__ __forceinline__ void put_one(char *out, int64_t col, float v) {
    uint32_t w[1] = {0};
    P::put(w, 0, v);
    swiglu::St<P::kBytes, swiglu::kStPlain>::run(out + col * P::kBytes, w);
}

// A group's sums of K columns from `col` on: dw (which = 0) or db (1), to the partial
// sums or, of the only group, to the results.
template <typename P, int K>
__device__ __forceinline__ void emit(const BwdParams &p, int64_t group, int which, int64_t col, const float *v) {
    if (p.partial != nullptr) {
        float *at = p.partial + (group * 2 + which) * p.pitch + col;
        if constexpr (K == 4)
            *reinterpret_cast<float4 *>(at) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *at = v[0];
    } else if (char *out = which ? p.db : p.dw) {
#pragma unroll
        for (int k = 0; k < K; ++k) put_one<P>(out, col + k, v[k]);
    }
}

// A group of G threads walks over rows with the same columns in every thread, so the
// column sums stay in registers until the end, when the CTA's groups are added up and
// leave one partial row of them.
//
// CLUSTER: the columns of a row are split over the CTAs of a cluster, COLS each.  Group g
// of every CTA sends its two sums into the shared memory of all of them (st.async, counted
// on a barrier there); two groups a CTA, so that one works while the other's sums travel.
template <typename E, typename P, int VEC, int C, int G, int T, bool CLUSTER, bool ANY>
__global__ void __launch_bounds__(T, 1) layer_norm_bwd_kernel(const __grid_constant__ BwdParams p) {
    constexpr int EB = E::kBytes, B = EB * VEC, WN = B < 4 ? 1 : B / 4, N = C * VEC / 2;
    constexpr int PB = P::kBytes * VEC, PN = PB < 4 ? 1 : PB / 4;
    constexpr int R = T / G, COLS = G * C * VEC, W = G / 32;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(16) float part[R][2 * 2 * W];
    __shared__ float2 peers[R][2][8];  // by rank, for a row and the one after it
    __shared__ __align__(8) uint64_t full[R][kMaxSlots], arrived[R][2];
    const int t = threadIdx.x % G, g = threadIdx.x / G;
    uint32_t rank = 0, ctas = 1;
    if constexpr (CLUSTER) {
        rank = tc::cluster_rank();
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    }
    if (threadIdx.x < R * kMaxSlots) tc::mbar_init(tc::smem_addr(&full[0][0] + threadIdx.x), 1);
    if (CLUSTER && threadIdx.x < R * 2) tc::mbar_init(tc::smem_addr(&arrived[0][0] + threadIdx.x), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    if constexpr (CLUSTER) tc::cluster_sync();  // every CTA of the cluster has started, its barriers exist
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    const int64_t group = blockIdx.x / ctas, step = (int64_t)(gridDim.x / ctas) * R;
    // ANY: a CTA takes rows of one kind, and the first of a cluster the columns before the
    // first pack as well
    int64_t row = ANY ? group % p.period + p.period * (group / p.period * R + g) : group * R + g;
    const int lead = ANY ? (int)((reinterpret_cast<uint64_t>(p.dx) + (uint64_t)(row * p.dx_stride)) & 15) / EB : 0;
    const int64_t head = (VEC - lead) & (VEC - 1), first_col = rank == 0 ? 0 : min(p.n, (int64_t)rank * COLS + head);
    // this CTA's columns (where a cluster has more CTAs than the row needs: none, at the row's
    // end, so that its copies stay inside the tensor)
    const int64_t n = min(p.n, (int64_t)(rank + 1) * COLS + head) - first_col, bytes = n * EB;
    const Columns<VEC, G> cols(t, rank == 0 ? lead : 0, n);
    const uint32_t slot0 = tc::smem_addr(ring) + (uint32_t)g * p.slots * p.slot_bytes, bar0 = tc::smem_addr(&full[g][0]);
    const uint32_t half = (uint32_t)p.slot_bytes / 2;
    const auto x_row = [&](int64_t r) { return p.x + r * p.x_stride + first_col * EB; };
    const auto dy_row = [&](int64_t r) { return p.dy + r * p.dy_stride + first_col * EB; };
    const auto issue = [&](int64_t r, int slot) {
        const uint32_t bar = bar0 + 8 * slot, at = slot0 + slot * p.slot_bytes;
        tc::mbar_arrive_expect_tx(bar, prepare_row<E>(p.rows_x, x_row(r), bytes, at) +
                                           prepare_row<E>(p.rows_dy, dy_row(r), bytes, at + half));
        copy_row(p.rows_x, x_row(r), bytes, at, bar);
        copy_row(p.rows_dy, dy_row(r), bytes, at + half, bar);
    };
    if (t == 0)
        for (int k = 0; k < p.slots && row + k * step < p.rows; ++k) issue(row + k * step, k);
    uint32_t ww[C][PN];
    uint64_t aw[N], ab[N];
    bool in[C];
#pragma unroll
    for (int i = 0; i < N; ++i) aw[i] = ab[i] = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        in[c] = cols.in(c);
#pragma unroll
        for (int k = 0; k < PN; ++k) ww[c][k] = P::kBytes == 4 ? 0x3f800000u : 0x3f803f80u;  // ones
        if constexpr (ANY) {
            if (p.w != nullptr && in[c]) load_elements<P, VEC>(p.w, first_col + cols.col(c), ww[c]);
        } else {
            if (p.w != nullptr && in[c]) load_words<PB>(p.w + (first_col + cols.col(c)) * P::kBytes, ww[c]);
        }
    }
    // of the single columns, out of the registers: w, the sums for dw and db, xhat, h
    __shared__ float lone[R][5][32];
    if (ANY && t < 32) lone[g][0][t] = 1.0f, lone[g][1][t] = lone[g][2][t] = 0.0f;
    if constexpr (ANY)
        if (t < 32 && p.w != nullptr && cols.single >= 0) lone[g][0][t] = load_param<P>(p.w, first_col + cols.single);
    bool ok = true;
    int slot = 0, turn = 0;
    uint32_t parity = 0, uses = 0;  // of the ring's barriers; exchanges so far
    float mean = row < p.rows ? p.mean[row] : 0.0f, rstd = row < p.rows ? p.rstd[row] : 0.0f;
    for (; row < p.rows; row += step) {
        ok = ok && row_arrived(bar0 + 8 * slot, parity);  // one that ran out is not waited for again
        const uint32_t at = slot0 + slot * p.slot_bytes;
        uint64_t xhat[N], h[N], s0 = 0, s1 = 0;
        const uint64_t scale = twice(rstd);
        uint32_t xw[C][WN], dw[C][WN];
        if constexpr (ANY) {
            const float x1 = shifted_packs<E>(x_row(row), at, cols, xw), dy1 = shifted_packs<E>(dy_row(row), at + half, cols, dw);
            if (t < 32) {
                const float xhat1 = cols.single >= 0 ? (x1 - mean) * rstd : 0.0f;
                lone[g][1][t] = fmaf(dy1, xhat1, lone[g][1][t]);
                lone[g][2][t] += dy1;
                const float h1 = dy1 * lone[g][0][t];
                lone[g][3][t] = xhat1, lone[g][4][t] = h1;
            }
        } else {
            packs<E, VEC, G>(x_row(row), at, t, in, xw);
            packs<E, VEC, G>(dy_row(row), at + half, t, in, dw);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint64_t dy = pair_of<E, VEC, C>(dw, i);
            // (columns past the row hold x = 0 and dy = 0; with a mean of 0 they add nothing,
            // where -mean rstd may be infinite)
            const uint64_t m = swiglu::x2(in[2 * i / VEC] ? mean : 0.0f, in[(2 * i + 1) / VEC] ? mean : 0.0f);
            xhat[i] = swiglu::mul_x2(swiglu::sub_x2(pair_of<E, VEC, C>(xw, i), m), scale);
            aw[i] = swiglu::fma_x2(dy, xhat[i], aw[i]);
            ab[i] = swiglu::add_x2(dy, ab[i]);
            h[i] = swiglu::mul_x2(dy, pair_of<P, VEC, C>(ww, i));
            s0 = swiglu::add_x2(s0, h[i]);
            s1 = swiglu::fma_x2(h[i], xhat[i], s1);
        }
        const int64_t next = row + step;
        const float mean_n = next < p.rows ? p.mean[next] : 0.0f, rstd_n = next < p.rows ? p.rstd[next] : 0.0f;
        float s[2] = {both(s0), both(s1)};
        if (ANY && t < 32) {
            s[0] += lone[g][4][t];
            s[1] = fmaf(lone[g][4][t], lone[g][3][t], s[1]);
        }
        group_sum<G, T, 2>(s, part[g] + turn * 2 * W, g);
        // every thread of the group has read the row: its slot takes the next one
        if constexpr (G == 32) __syncwarp();
        if (t == 0 && ok && row + p.slots * step < p.rows) issue(row + p.slots * step, slot);
        if constexpr (CLUSTER) {
            const uint32_t mine = tc::smem_addr(&peers[g][turn][rank]), bar = tc::smem_addr(&arrived[g][turn]);
            if (t == 0) tc::mbar_arrive_expect_tx(bar, 8 * ctas);
            if (t < (int)ctas)  // into the place of this rank in every CTA
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                                 tc::map_to_rank(mine, (uint32_t)t)),
                             "f"(s[0]), "f"(s[1]), "r"(tc::map_to_rank(bar, (uint32_t)t))
                             : "memory");
            ok = ok && tc::mbar_wait_or_flag<true>(bar, uses >> 1 & 1, &g_norm_timeout);
            ++uses;
            s[0] = s[1] = 0.0f;
            for (uint32_t r = 0; r < ctas; ++r) {
                float a, b;
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                             : "=f"(a), "=f"(b)
                             : "r"(tc::smem_addr(&peers[g][turn][r]))
                             : "memory");
                s[0] += a;
                s[1] += b;
            }
        }
        // dx = rstd h - rstd c1 - xhat rstd c2
        const uint64_t c1 = twice(-rstd * (s[0] * p.inv_n)), c2 = twice(-rstd * (s[1] * p.inv_n));
        char *dst = p.dx + row * p.dx_stride + first_col * EB;
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = swiglu::fma_x2(xhat[i], c2, swiglu::fma_x2(h[i], scale, c1));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!in[c]) continue;
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float lo, hi;
                swiglu::x2_split(h[(c * VEC + k) / 2], lo, hi);
                v[k] = (c * VEC + k) % 2 ? hi : lo;
            }
            store_once<E, VEC>(dst + (int64_t)cols.col(c) * EB, v);
        }
        if (ANY && t < 32) {
            float k1, k2, unused;
            swiglu::x2_split(c1, k1, unused);
            swiglu::x2_split(c2, k2, unused);
            const float v[1] = {fmaf(lone[g][3][t], k2, fmaf(lone[g][4][t], rstd, k1))};
            if (cols.single >= 0) store_once<E, 1>(dst + (int64_t)cols.single * EB, v);
        }
        mean = mean_n;
        rstd = rstd_n;
        turn ^= 1;
        if (++slot == p.slots) {
            slot = 0;
            parity ^= 1;
        }
    }
    if (!ok && t == 0) tc::settle();  // a wait ran out: no copy lands in shared memory that is used again
    if constexpr (CLUSTER) {
        __syncwarp();
        tc::cluster_sync();  // no CTA leaves while another may still send to it
    }
    if (p.partial == nullptr && p.dw == nullptr && p.db == nullptr) return;
    // the groups' sums in their order, through the ring
    float *fold = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        constexpr int M = 2 * N + (ANY ? 1 : 0);
        float v[M];
#pragma unroll
        for (int i = 0; i < N; ++i) swiglu::x2_split(which ? ab[i] : aw[i], v[2 * i], v[2 * i + 1]);
        if constexpr (ANY) v[2 * N] = t < 32 ? lone[g][1 + which][t] : 0.0f;
        if constexpr (R > 1) {
            __syncthreads();
            if (g > 0)
#pragma unroll
                for (int e = 0; e < M; ++e) fold[((g - 1) * M + e) * G + t] = v[e];
            __syncthreads();
            if (g == 0)
                for (int k = 0; k < R - 1; ++k)
#pragma unroll
                    for (int e = 0; e < M; ++e) v[e] += fold[(k * M + e) * G + t];
        }
        if constexpr (ANY) {  // in the order of the columns
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (in[c])
#pragma unroll
                        for (int k = 0; k < VEC; ++k) fold[cols.col(c) + k] = v[c * VEC + k];
                if (cols.single >= 0) fold[cols.single] = v[2 * N];
            }
            __syncthreads();
            for (int col = threadIdx.x; col < n; col += T) emit<P, 1>(p, group, which, first_col + col, fold + col);
        } else if (g == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in[c])
#pragma unroll
                    for (int k = 0; k < VEC; k += (VEC > 1 ? 4 : 1))
                        emit<P, (VEC > 1 ? 4 : 1)>(p, group, which, first_col + cols.col(c) + k, v + c * VEC + k);
        }
    }
}

// Rows too long for a cluster's registers: mean(h) and mean(h xhat) of each row, then
// dx and the column sums of a tile of columns, which reads dy and x once more.
template <typename E, typename P, int VEC, int T>
__global__ void __launch_bounds__(T) layer_norm_bwd_sums_kernel(BwdParams p) {
    constexpr int EB = E::kBytes, B = EB * VEC, WN = B < 4 ? 1 : B / 4;
    __shared__ __align__(16) float part[2][2 * (T / 32)];
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        float s[2] = {0.0f, 0.0f};
#pragma unroll 2
        for (int64_t col = (int64_t)threadIdx.x * VEC; col < p.n; col += (int64_t)T * VEC) {
            uint32_t xw[WN], dw[WN];
            load_once<B>(p.x + row * p.x_stride + col * EB, xw);
            load_once<B>(p.dy + row * p.dy_stride + col * EB, dw);
            float q[VEC], a = 0.0f, b = 0.0f;
            if (p.w != nullptr) load_params<P, VEC>(p.w, col, q);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float xhat, dy;
                unpack<E, VEC>(xw, dw, mean, rstd, k, xhat, dy);
                const float h = p.w != nullptr ? dy * q[k] : dy;
                a += h;
                b = fmaf(h, xhat, b);
            }
            s[0] += a;
            s[1] += b;
        }
        group_sum<T, T, 2>(s, part[turn], 0);
        turn ^= 1;
        if (threadIdx.x == 0) {
            p.sums[2 * row] = s[0] * p.inv_n;
            p.sums[2 * row + 1] = s[1] * p.inv_n;
        }
    }
}

// blockIdx.x: the tile of T * VEC columns, blockIdx.y: the group of rows.  Where the tiles are
// many the groups are few (one from 156 thousand columns on that are not in packs).  SEGMENTS:
// a group has more than kSegment rows, so its column sums are cut into segments of as many,
// which are added up in their order (in every launch: [500, 70001] bf16 169 instead of 151 us).
constexpr int kSegment = 256;

template <typename E, typename P, int VEC, int T, bool SEGMENTS>
__global__ void __launch_bounds__(T) layer_norm_bwd_tile_kernel(BwdParams p) {
    constexpr int EB = E::kBytes, B = EB * VEC, WN = B < 4 ? 1 : B / 4;
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    const int64_t col = ((int64_t)blockIdx.x * T + threadIdx.x) * VEC;
    if (col >= p.n) return;
    __shared__ float total[SEGMENTS ? 2 * VEC : 1][T];  // of the segments so far, out of the registers
    if constexpr (SEGMENTS)
#pragma unroll
        for (int k = 0; k < 2 * VEC; ++k) total[k][threadIdx.x] = 0.0f;
    float q[VEC], aw[VEC], ab[VEC];
    if (p.w != nullptr) load_params<P, VEC>(p.w, col, q);
#pragma unroll
    for (int k = 0; k < VEC; ++k) aw[k] = ab[k] = 0.0f;
    for (int64_t first = blockIdx.y; first < p.rows; first += (int64_t)kSegment * gridDim.y) {
        const int64_t last = SEGMENTS ? min(p.rows, first + (int64_t)kSegment * gridDim.y) : p.rows;
#pragma unroll 4
        for (int64_t row = first; row < last; row += gridDim.y) {
            uint32_t xw[WN], dw[WN];
            load_once<B>(p.x + row * p.x_stride + col * EB, xw);
            load_once<B>(p.dy + row * p.dy_stride + col * EB, dw);
            const float mean = p.mean[row], rstd = p.rstd[row], c1 = p.sums[2 * row],
                        c2 = p.sums[2 * row + 1];
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float xhat, dy;
                unpack<E, VEC>(xw, dw, mean, rstd, k, xhat, dy);
                aw[k] = fmaf(dy, xhat, aw[k]);
                ab[k] += dy;
                const float h = p.w != nullptr ? dy * q[k] : dy;
                v[k] = rstd * fmaf(-xhat, c2, h - c1);
            }
            store_once<E, VEC>(p.dx + row * p.dx_stride + col * EB, v);
        }
        if constexpr (SEGMENTS) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                total[k][threadIdx.x] += aw[k];
                total[VEC + k][threadIdx.x] += ab[k];
                aw[k] = ab[k] = 0.0f;
            }
        } else {
            break;
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        if constexpr (SEGMENTS) {
            aw[k] = total[k][threadIdx.x];
            ab[k] = total[VEC + k][threadIdx.x];
        }
        emit<P, 1>(p, blockIdx.y, 0, col + k, aw + k);
        emit<P, 1>(p, blockIdx.y, 1, col + k, ab + k);
    }
}

// The groups' column sums added up in a fixed order: a lane a column, each warp a
// segment of the groups.  blockIdx.y: 0 for dw, 1 for db.
template <typename P, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) layer_norm_reduce_kernel(const float *partial, char *dw, char *db, int64_t n,
                                                                      int64_t pitch, int groups) {
    __shared__ float part[WARPS][32];
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    char *out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr) return;
    const int each = (groups + WARPS - 1) / WARPS, first = warp * each, last = min(groups, first + each);
    float s = 0.0f;
    if (col < n) {
        const float *at = partial + (int64_t)blockIdx.y * pitch + col;
#pragma unroll 16
        for (int g = first; g < last; ++g) s += at[(int64_t)g * 2 * pitch];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < n) {
        s = part[0][lane];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) s += part[w][lane];
        put_one<P>(out, col, s);
    }
}

}  // namespace lnorm
