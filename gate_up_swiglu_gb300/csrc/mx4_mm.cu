// mx4_mm.cu -- products of tensors in microscaled 4-bit floating point, and the
// gated MLP made of them (the contract is in include/swiglu_mx4.h).
//
// tcgen05.mma kind::mxf4 multiplies blocks of 64 codes: each product of two codes
// and their two scales is exact, and the sums are kept in fp32 in tensor memory.
// Codes come to shared memory by TMA, 256 of a row (128 bytes, one swizzle row) a
// stage; scale tiles come by TMA as they lie in memory and go on to tensor memory
// (tcgen05.cp), where the instruction wants them: byte b of row i in lane i % 32,
// column i / 32, repeated in the four lane quarters.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "mx4.cuh"
#include "mx4_host.h"
#include "tc_pair.cuh"

namespace mx4 {

using namespace tc;

__device__ int g_mx4_timeout = 0;

template <bool kCluster = false>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    return mbar_wait_or_flag<kCluster>(bar, parity, &g_mx4_timeout);
}

// ------------------------------------------------------------ instructions ---

// Instruction descriptor of kind::mxf4: A and B e2m1 (bits 7-9 and 10-11 = 1), both
// K-major, scales of type e8m0 (bit 23), N / 8 in bits 17-22, M / 128 in bits 27-28;
// bits 4-5 and 29-30 pick the scale bytes of B and A in each 32-bit column (0 or 2:
// an instruction of K = 64 takes two).
__host__ __device__ constexpr uint32_t instr_desc(int M, int N, int sf) {
    return (1u << 7) | (1u << 10) | (1u << 23) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 7) << 27) |
           ((uint32_t)sf << 4) | ((uint32_t)sf << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t acc) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// Shared-memory descriptor of a scale tile: 32 rows of 16 bytes without a swizzle,
// groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// A scale tile to four columns of tensor memory, the same in each lane quarter.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// silu(g) * u, as the streaming kernels' bf16 form.
__device__ __forceinline__ float swiglu_of(float g, float u) {
    const swiglu::Act act = swiglu::activation<swiglu::BF16, false, true>(g);
    return __fmul_rn(__fmul_rn(act.silu, u), act.scale);
}

// silu(g) * u of N columns.  Without a gate below -64 (one test of the smallest) the
// branch-free form does, two lanes an instruction: the same operations and roundings,
// so the same bits, as swiglu_of.
template <int N>
__device__ __forceinline__ void activate(const uint32_t *g, const uint32_t *u, float *v) {
    float gmin = __uint_as_float(g[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) gmin = fminf(gmin, __uint_as_float(g[i]));
    if (!(gmin < -64.0f)) {
        const uint64_t neg_log2e = swiglu::x2(-swiglu::kLog2e, -swiglu::kLog2e), one = swiglu::x2(1.0f, 1.0f);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint64_t g2 = swiglu::x2(__uint_as_float(g[i]), __uint_as_float(g[i + 1]));
            const uint64_t u2 = swiglu::x2(__uint_as_float(u[i]), __uint_as_float(u[i + 1]));
            float t0, t1, d0, d1;
            swiglu::x2_split(swiglu::mul_x2(g2, neg_log2e), t0, t1);
            swiglu::x2_split(swiglu::add_x2(one, swiglu::x2(swiglu::ex2_approx(t0), swiglu::ex2_approx(t1))), d0, d1);
            const uint64_t s2 = swiglu::x2(swiglu::rcp_approx(d0), swiglu::rcp_approx(d1));
            swiglu::x2_split(swiglu::mul_x2(swiglu::mul_x2(g2, s2), u2), v[i], v[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = swiglu_of(__uint_as_float(g[i]), __uint_as_float(u[i]));
    }
}

// A stage is 256 columns: 128 bytes of codes a row, two scale tiles.
constexpr int kCodesTile = 128 * 128;
constexpr int kScalesTile = 2 * kTileBytes;

// Where the results go: y, or (of the first product) the activation in 4 bits.
struct Out {
    __nv_bfloat16 *y;
    uint8_t *q, *scales;
    int32_t cols;    // of the result
    int32_t nb, chunks;  // blocks and scale tiles of its rows
};

// ------------------------------------------------------------ split kernel ---
// Few rows: the weights are the instruction's 128 rows, NT rows of x its columns, so
// that the weights stream through once whatever the number of rows, and a cluster of
// CTAs shares a tile's contraction (its slices are added up through each other's
// shared memory in the order of the slices).  TILES = 2: a gate and an up tile.
//
// `early` (only where the grid before this one is of this library, so that it has waited
// for those before it, and does not write the weights): the first weights are loaded
// before the wait for that grid.
//
// X: void where x is in 4 bits; else the type of the rows, which the CTA rounds itself,
// block by block as it needs them (16 rows at most: a launch less, and every CTA reads the
// few rows from L2).
//
// Bound by the weights' bytes, and by its start and join where these are few: 16 rows by
// [4096, 14336] 8.6 us (4.6 us at the copy rate), 128 rows 11.1 us.
//
// Warp 0 issues the loads, warp 1 the scale copies and products, warps 2-5 round x where
// that is asked for and read the accumulator, each its own quarter of the lanes; all of
// them add up the slices.

// PER_SM: two CTAs an SM where four stages' worth of weights allow it and there are more
// CTAs than SMs: one works while the other starts or ends ([128, 4096] x [28672, 4096] 20 ->
// 16 us; one alone on its SM wants the whole ring).
template <int NT, int TILES, int PER_SM>
struct SplitShape {
    static constexpr int kCodesX = NT * 128;
    static constexpr int kStage = TILES * (kCodesTile + kScalesTile) + kCodesX + kScalesTile;
    static constexpr int kRing = PER_SM == 2 ? 113 * 1024 : 220 * 1024;
    static constexpr int kStages = (kRing - 2048) / kStage < 8 ? (kRing - 2048) / kStage : 8;
    static constexpr int kAccCols = TILES * NT;
    static constexpr int kScaleCols = (TILES + 1) * 8;  // of a stage
    static constexpr int kNeed = kAccCols + 2 * kScaleCols;
    static constexpr int kTmemCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static constexpr int kSmem = kStages * kStage + 1024 + 256;
    // (twice the warps where a CTA has many rows to finish)
    static constexpr int kThreads = NT >= 64 ? 384 : 192;
    static_assert(PER_SM * kTmemCols <= 512, "no CTA waits for tensor memory that its neighbour on the SM holds");
    static_assert(kStages >= 2 && kStages * kStage >= kAccCols * 512, "the partial sums fit the ring");
};


// Four values of row t, columns j .. j + 3 (a warp: 128 columns of a row): rounded to
// bf16, or as part of a block of 4 bits, of which 8 lanes hold one.
template <int TILES>
__device__ __forceinline__ void put4(const Out &o, int t, int j, int lane, const float (&g)[4], const float (&u)[4]) {
    if constexpr (TILES == 1) {
        __nv_bfloat16 *y = o.y + (int64_t)t * o.cols + j;
        if (j + 4 <= o.cols && reinterpret_cast<uintptr_t>(y) % 8 == 0) {
            uint32_t w[2];
            swiglu::BF16::put2(w, 0, g[0], g[1]);
            swiglu::BF16::put2(w, 2, g[2], g[3]);
            swiglu::St<8, swiglu::kStPlain>::run(y, w);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k < o.cols) y[k] = __float2bfloat16_rn(g[k]);
        }
    } else {
        float v[4];
        activate<4>(reinterpret_cast<const uint32_t *>(g), reinterpret_cast<const uint32_t *>(u), v);
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (j + k >= o.cols) v[k] = 0.0f;
            m = max(m, magnitude(v[k]));
        }
#pragma unroll
        for (int d = 1; d < 8; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const uint32_t sc = scale_byte(m);
        scale_values<4>(v, sc);
        const int b = j >> 5;
        if (b < o.nb)
            *reinterpret_cast<uint16_t *>(o.q + ((int64_t)t * o.nb + b) * 16 + (lane & 7) * 2) =
                (uint16_t)(codes2(v[0], v[1]) | codes2(v[2], v[3]) << 8);
        if ((lane & 7) == 0) o.scales[scale_offset(0, t, b, o.chunks)] = (uint8_t)sc;
    }
}

__device__ __forceinline__ float4 load_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// A CTA finishes the rows of x slice, slice + SLICES, ...: all slices' sums in their
// order.  A warp takes a row, a lane four columns; the loads of all slices, and of
// several rows where the slices are few, are in flight at a time.
template <int TILES, int NT, int THREADS, int SLICES>
__device__ __forceinline__ void join(const Out &out, uint32_t sums, int rows, int t0, int tile, uint32_t slice) {
    constexpr int kRows = SLICES * TILES >= 8 ? 1 : 8 / (SLICES * TILES), kStep = SLICES * (THREADS / 32);
    const int lane = threadIdx.x & 31, live = min(NT, rows);
    for (int t = (int)slice + SLICES * (int)(threadIdx.x >> 5); t < live; t += kRows * kStep) {
        float4 part[kRows][TILES][SLICES];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                // (a row past the last one reads the last one's place)
                const uint32_t at = sums + (uint32_t)((i * NT + min(t + k * kStep, live - 1)) * 128 + 4 * lane) * 4;
#pragma unroll
                for (uint32_t r = 0; r < SLICES; ++r)
                    part[k][i][r] = load_cluster_f32x4(SLICES == 1 ? at : map_to_rank(at, r));
            }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            float v[TILES][4];
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                float4 a = part[k][i][0];
#pragma unroll
                for (int r = 1; r < SLICES; ++r) {
                    const float4 b = part[k][i][r];
                    a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
                }
                v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
            }
            if (t + k * kStep < live)  // the whole warp
                put4<TILES>(out, t0 + t + k * kStep, tile * 128 + 4 * lane, lane, v[0], v[TILES - 1]);
        }
    }
}

// Rows of x as they are.
struct Rows16 {
    const char *x;
    int64_t stride;  // bytes
};

// Thread i (of 128) loads and rounds block i % 8 of row i / 8 of a stage of 16 rows: the
// codes go where TMA would put them (16-byte piece j of row r at j ^ (r % 8) of its 128
// bytes), the scale to its byte of the tiles.
template <typename X>
__device__ __forceinline__ void load_block(const Rows16 &x, int M, int64_t blocks, int ks, int i, uint32_t *w) {
    constexpr int B = 32 * X::kBytes;
    const int row = i >> 3;
    const int64_t b = (int64_t)ks * 8 + (i & 7);
#pragma unroll
    for (int k = 0; k < B / 4; ++k) w[k] = 0;
    if (row < M && b < blocks)
#pragma unroll
        for (int k = 0; k < B; k += 16) swiglu::load_after<16, true>(x.x + row * x.stride + b * B + k, w + k / 4);
}

template <typename X>
__device__ __forceinline__ void round_block(const uint32_t *w, int i, uint32_t codes, uint32_t scales) {
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        v[k] = X::get(w, k);
        m = max(m, magnitude(v[k]));
    }
    const uint32_t sc = scale_byte(m);
    scale_values<32>(v, sc);
    const int row = i >> 3, j = i & 7;
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(codes + row * 128 + ((j ^ (row & 7)) << 4)), "r"(codes8(v)),
                 "r"(codes8(v + 8)), "r"(codes8(v + 16)), "r"(codes8(v + 24))
                 : "memory");
    asm volatile("st.shared.b8 [%0], %1;" ::"r"(scales + (j >> 2) * kTileBytes + row * 16 + (j & 3)), "r"(sc) : "memory");
}

template <int NT, int TILES, int PER_SM, typename X>
__global__ void __launch_bounds__(SplitShape<NT, TILES, PER_SM>::kThreads)
    mx4_split_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_up,
                     const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_ws,
                     const __grid_constant__ CUtensorMap tm_xs, Rows16 rows, Out out, int M, int nb, int chunks, int tiles,
                     int early) {
    using S = SplitShape<NT, TILES, PER_SM>;
    constexpr bool kRaw = !std::is_void_v<X>;
    static_assert(!kRaw || NT == 16, "a stage's 128 blocks are one to a thread of four warps");
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_addr(smem);
    unsigned char *state = smem + S::kStages * S::kStage;
    const uint32_t full0 = smem_addr(state), empty0 = full0 + 8 * S::kStages, acc_full = empty0 + 8 * S::kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(state + 16 * S::kStages + 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    uint32_t slices;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(slices));
    const uint32_t slice = cluster_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = (int)(blockIdx.x / slices) % tiles, t0 = (int)(blockIdx.x / slices) / tiles * NT;
    const int total = (nb + 7) / 8;  // stages of the whole contraction
    const int first = (int)((int64_t)total * slice / slices), last = (int)((int64_t)total * (slice + 1) / slices);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, kRaw ? 1 + 4 : 1);  // the producer, and the warps that round x
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(S::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (elect_one()) {
            const auto load_w = [&](int ks, int s) {
                const uint32_t full = full0 + 8 * s, at = ring + s * S::kStage, scales = at + TILES * kCodesTile + S::kCodesX;
                mbar_arrive_expect_tx(full, kRaw ? TILES * (kCodesTile + kScalesTile) : S::kStage);
                tma_load_2d(at, &tm_w, full, ks * 128, tile * 128);
                if (TILES == 2) tma_load_2d(at + kCodesTile, &tm_up, full, ks * 128, tile * 128);
                tma_load_2d(scales, &tm_ws, full, 0, tile * chunks + 2 * ks);
                if (TILES == 2) tma_load_2d(scales + kScalesTile, &tm_ws, full, 0, (tiles + tile) * chunks + 2 * ks);
            };
            const auto load_x = [&](int ks, int s) {
                if (kRaw) return;
                const uint32_t full = full0 + 8 * s, at = ring + s * S::kStage + TILES * kCodesTile;
                tma_load_2d(at, &tm_x, full, ks * 128, t0);
                tma_load_2d(at + S::kCodesX + TILES * kScalesTile, &tm_xs, full, 0, (t0 / 128) * chunks + 2 * ks);
            };
            // `early`: the ring's first weights come while the grid before this one runs
            const int ahead = early ? min(S::kStages, last - first) : 0;
            for (int k = 0; k < ahead; ++k) load_w(first + k, k);
            swiglu::await_previous_grid();
            swiglu::allow_next_grid();
            for (int k = 0; k < ahead; ++k) load_x(first + k, k);
            int it = ahead;
            for (int ks = first + ahead; ks < last; ++ks, ++it) {
                const int s = it % S::kStages;
                if (!wait(empty0 + 8 * s, ((it / S::kStages) & 1) ^ 1)) {
                    *abort_flag = 1;
                    break;
                }
                load_w(ks, s);
                load_x(ks, s);
            }
            // nothing is in flight when the CTA leaves, also after a wait ran out
            for (int k = it > S::kStages ? it - S::kStages : 0; k < it; ++k)
                if (!wait(full0 + 8 * (k % S::kStages), (k / S::kStages) & 1)) settle();
        }
    } else if (warp == 1) {
        swiglu::await_previous_grid();
        if (elect_one()) {
            bool ok = true;
            int it = 0;
            for (int ks = first; ks < last; ++ks, ++it) {
                const int s = it % S::kStages;
                if (!wait(full0 + 8 * s, (it / S::kStages) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t base = ring + s * S::kStage;
                const uint32_t xcodes = base + TILES * kCodesTile, scales = xcodes + S::kCodesX;
                const uint32_t sf = tmem + S::kAccCols + (it & 1) * S::kScaleCols;
                const int steps = min(4, (nb - 8 * ks + 1) / 2);  // products of 64 columns
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (2 * c < steps)
#pragma unroll
                        for (int i = 0; i <= TILES; ++i)
                            copy_scales(sf + 8 * i + 4 * c, scale_desc(scales + i * kScalesTile + c * kTileBytes));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    if (kk < steps) {
                        const uint64_t b = smem_desc_128b(xcodes + kk * 32);
                        const uint32_t idesc = instr_desc(128, NT, (kk & 1) * 2);
#pragma unroll
                        for (int i = 0; i < TILES; ++i)
                            mma_mxf4(tmem + i * NT, smem_desc_128b(base + i * kCodesTile + kk * 32), b, idesc,
                                     sf + 8 * i + 4 * (kk >> 1), sf + 8 * TILES + 4 * (kk >> 1),
                                     (it | kk) != 0 ? 1u : 0u);
                    }
                mma_commit(empty0 + 8 * s);
            }
            mma_commit(acc_full);
            if (!ok) *abort_flag = 1;
            wait(acc_full, 0);
        }
    } else if (warp < 6) {
        swiglu::await_previous_grid();
        if constexpr (kRaw) {
            const int i = (warp - 2) * 32 + lane;
            constexpr int kWords = 8 * X::kBytes;
            uint32_t w[kWords], next[kWords];
            load_block<X>(rows, M - t0, nb, first, i, next);
            int it = 0;
            for (int ks = first; ks < last; ++ks, ++it) {
                const int s = it % S::kStages;
#pragma unroll
                for (int k = 0; k < kWords; ++k) w[k] = next[k];
                if (ks + 1 < last) load_block<X>(rows, M - t0, nb, ks + 1, i, next);
                if (!__all_sync(0xffffffffu, wait(empty0 + 8 * s, ((it / S::kStages) & 1) ^ 1))) {
                    *abort_flag = 1;
                    break;
                }
                const uint32_t codes = ring + s * S::kStage + TILES * kCodesTile;
                round_block<X>(w, i, codes, codes + S::kCodesX + TILES * kScalesTile);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(full0 + 8 * s) : "memory");
            }
        }
        const int quarter = warp & 3;
        const bool ok = __all_sync(0xffffffffu, wait(acc_full, 0));
        tc_fence_after();
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        const int row = 32 * quarter + lane, live = min(NT, M - t0);
        // every product has read its stage: the ring holds the sums now, [accumulator
        // column][128 rows]
        float *sums = reinterpret_cast<float *>(smem);
        if (ok)
#pragma unroll 1
            for (int i = 0; i < TILES; ++i)
#pragma unroll 1
                for (int c = 0; c < live; c += 16) {
                    uint32_t v[16];
                    tmem_load16(lanes + i * NT + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) sums[(i * NT + c + k) * 128 + row] = __uint_as_float(v[k]);
                }
    }
    __syncwarp();
    tc_fence_before();
    if (slices > 1)
        cluster_sync();
    else
        __syncthreads();
    swiglu::await_previous_grid();  // of every thread that writes results
    switch (slices) {
        case 1: join<TILES, NT, S::kThreads, 1>(out, ring, M - t0, t0, tile, slice); break;
        case 2: join<TILES, NT, S::kThreads, 2>(out, ring, M - t0, t0, tile, slice); break;
        case 4: join<TILES, NT, S::kThreads, 4>(out, ring, M - t0, t0, tile, slice); break;
        default: join<TILES, NT, S::kThreads, 8>(out, ring, M - t0, t0, tile, slice);
    }
    if (slices > 1) cluster_sync_read();  // no CTA leaves while another reads its sums
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmemCols) : "memory");
    }
}

// ------------------------------------------------------------- pair kernel ---
// Many rows: a cluster of two CTAs computes a tile of 256 rows of x by 256 rows of W
// (of the first product: 128 gate rows, then the 128 up rows that go with them) with
// tcgen05.mma.cta_group::2.  Each CTA loads its own 128 rows of x and one half of the
// W tile, and the scales of its own rows and of all of W's; the leader's MMA thread
// drives both SMs.  A CTA's accumulator holds its own 128 rows by 256 columns.
//
// Scales go to tensor memory by four warps of their own (each writes its quarter of
// the lanes), up to three stages ahead of the products.  Copied by the MMA thread
// (tcgen05.cp, as in the split kernel), each of a stage's six scale tiles held up the
// products by some 47 cycles: [8192, 14336] x [4096, 14336] took 199 us, with four warps
// 148 us (145 us now, 6.6 PFLOP/s; 151 us after seconds at the power limit).  A stage takes
// some 740 cycles, of which the four products are 512: the tensor pipe is active 67 % of the time,
// the port into an SM (35.8 KB a stage and CTA) 36 %.  Where the rest goes is not shown.
//
// Tensor memory has 512 columns: two accumulators of 256 leave no room for three
// stages' scales, 24 columns each.  So the two overlap by 72 columns, and the epilogue
// reads a tile to registers before it does anything else: the next tile's products
// start as soon as the columns they share have been read.
//
// 512 threads a CTA: warp 0 issues the loads (the leader's takes tiles by cluster
// launch control, too), warp 1 the products (the leader's), warps 4-11 read the
// accumulator, two to each quarter of the lanes, 128 columns each (of the first
// product: 64 gate columns and the 64 up columns that go with them), warps 12-15 write
// the scales.  The epilogue's two warpgroups take 192 registers a thread, the others 64:
// together the 4 x 128 that the CTA starts with.  Roles, tile ring and waits are those
// of the linear_fc1 kernel.

constexpr int kPairThreads = 512;
constexpr int kEpilogueRegs = 192, kOtherRegs = 64;
static_assert(2 * kEpilogueRegs + 2 * kOtherRegs <= 4 * (65536 / kPairThreads), "the registers of the launch");
constexpr int kPairStage = 2 * kCodesTile + 3 * kScalesTile;  // of a CTA
constexpr int kPairState = 320;                // bytes of barriers and state
constexpr int kStagingPitch = 144;             // of a row of 64 bf16 columns, 16 bytes between rows: no bank conflicts
// What a tile's results become: the activation in 4 bits (of the first product); y of rows
// that are whole 32-byte packs, which go out from registers; y of any rows, which pass
// through shared memory on their way, 32 rows of a warp at a time, at the price of a stage.
// ([8192, 2000] x [n, 2000] with n = 5504, 5496, 5503: 59, 78, 94 us from registers; 62, 64,
// 81 us through shared memory.)
enum Results { kGatedBlocks, kWholePacks, kAnyRows };

template <Results kTo>
struct PairShape {
    static constexpr int kStages = kTo == kAnyRows ? 5 : 6;  // of the ring
    static constexpr int kStaging = kTo == kAnyRows ? 8 * 32 * kStagingPitch : 0;
    static constexpr int kSmem = kStages * kPairStage + kStaging + 1024 + kPairState;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};
constexpr int kPairBars = 6;                   // barriers of a kind, of the longer ring
constexpr int kScaleSlots = 3;                 // stages whose scales are in tensor memory
constexpr int kScaleCols = 24;                 // of a stage: 8 of x, 16 of W
constexpr int kScaleCol = 512 - kScaleSlots * kScaleCols;
constexpr int kAccShift = kScaleCol - 256;     // the second accumulator's first column
constexpr int kTileSlots = 4;
constexpr int kTileReaders = 1 + 1 + 2 * 12;   // peer producer, MMA thread, epilogue and scale warps
constexpr int kAskAhead = 6;                   // the next tile is asked for this many stages before the last load
constexpr int kGroupM = 16;                    // row tiles that share W tiles in L2 at a time

constexpr int OFF_FULL = 0, OFF_EMPTY = OFF_FULL + 8 * kPairBars, OFF_ACC_FULL = OFF_EMPTY + 8 * kPairBars,
              OFF_ACC_EMPTY = OFF_ACC_FULL + 16, OFF_MMA_DONE = OFF_ACC_EMPTY + 8, OFF_TILE_FULL = OFF_MMA_DONE + 8,
              OFF_TILE_EMPTY = OFF_TILE_FULL + 8 * kTileSlots, OFF_CLC_BAR = OFF_TILE_EMPTY + 8 * kTileSlots,
              OFF_CLC_RESP = (OFF_CLC_BAR + 8 + 15) / 16 * 16, OFF_TILE_ID = OFF_CLC_RESP + 16,
              OFF_TMEM = OFF_TILE_ID + 4 * kTileSlots, OFF_ABORT = OFF_TMEM + 4,
              OFF_SFULL = (OFF_ABORT + 4 + 7) / 8 * 8, OFF_SCALES = OFF_SFULL + 8 * kPairBars;
static_assert(OFF_SCALES + 8 * kScaleSlots <= kPairState, "barriers and state fit their region");

__device__ __forceinline__ void mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// Eight columns of this warp's lanes.
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint4 &a, const uint4 &b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

__device__ __forceinline__ uint4 load_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void store_shared16(uint32_t addr, const uint32_t *w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

__device__ __forceinline__ void pair_tile(int t, int tiles_m, int tiles_n, int &m0, int &tn) {
    const int per_group = kGroupM * tiles_n, g = t / per_group, first = g * kGroupM;
    const int gm = min(kGroupM, tiles_m - first), local = t - g * per_group;
    m0 = (first + local % gm) * 256;
    tn = local / gm;
}

// 64 fp32 values as bf16 to row p (columns col .. col + 63 of a row of n, n % 16 == 0).
// Stores that leave L1 alone: [8192, 4096] x [28672, 4096] 349 us, evict-first 365 us.
__device__ __forceinline__ void store64(__nv_bfloat16 *p, const uint32_t (&v)[64], int col, int n) {
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2)
            swiglu::BF16::put2(w, i, __uint_as_float(v[c + i]), __uint_as_float(v[c + i + 1]));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (col + c + 16 * k < n) swiglu::St<32, swiglu::kStNoAlloc>::run(p + c + 16 * k, w + 8 * k);
    }
}

// 64 columns of a warp's 32 rows (a lane has a row: v) as bf16 to y (the first of the rows,
// columns `left` and on are not there; rows `cols` apart; `live` of them exist), by way of
// the warp's part of shared memory: eight lanes write 128 bytes of a row at a time.
// `pieces`: every row starts at 16 bytes and has whole 16 bytes.  Else a row is shifted by
// its distance from the 16 bytes before it, and its lane stores what is less than 16 bytes
// at both ends; columns of a row that ends inside the 64 go one by one.
__device__ __forceinline__ void store64_any(__nv_bfloat16 *y, int cols, const uint32_t (&v)[64], int left, int live,
                                            bool pieces, uint32_t staging) {
    using swiglu::St;
    constexpr auto kind = swiglu::kStPlain;
    if (left <= 0) return;
    const int lane = threadIdx.x & 31;
    __nv_bfloat16 *p = y + (int64_t)lane * cols;
    if (!pieces && left < 64) {
        if (lane < live)
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i < left) p[i] = __float2bfloat16_rn(__uint_as_float(v[i]));
        return;
    }
    uint32_t w[36];
#pragma unroll
    for (int i = 0; i < 64; i += 2) swiglu::BF16::put2(w, i, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    if (!pieces) {
        const uint32_t off = (uint32_t)(reinterpret_cast<uint64_t>(p) & 15) >> 1;  // columns
#pragma unroll
        for (int k = 32; k < 36; ++k) w[k] = 0;
        // from the last word on, so that a step's sources are those of the step before
#pragma unroll
        for (int k = 35; k >= 0; --k) w[k] = off & 1 ? __funnelshift_l(k > 0 ? w[k - 1] : 0, w[k], 16) : w[k];
#pragma unroll
        for (int k = 35; k >= 0; --k) w[k] = off & 2 ? (k > 0 ? w[k - 1] : 0) : w[k];
#pragma unroll
        for (int k = 35; k >= 0; --k) w[k] = off & 4 ? (k > 1 ? w[k - 2] : 0) : w[k];
        __nv_bfloat16 *at = p - off;  // column c of the shifted row: half c % 2 of word c / 2
        if (lane < live) {
            if (off == 0) {
                St<16, kind>::run(at, w);
            } else {
                if (off & 1) {
                    const uint32_t h[1] = {(off & 4 ? (off & 2 ? w[3] : w[2]) : (off & 2 ? w[1] : w[0])) >> 16};
                    St<2, kind>::run(at + off, h);
                }
                const uint32_t c = off + (off & 1);
                const uint32_t two[1] = {c & 4 ? w[3] : w[1]};
                if (c & 2) St<4, kind>::run(at + c, two);
                if (c <= 4) St<8, kind>::run(at + 4, w + 2);
            }
            at += 64;
            if (off & 4) St<8, kind>::run(at, w + 32);
            const uint32_t two[1] = {off & 4 ? w[34] : w[32]};
            if (off & 2) St<4, kind>::run(at + (off & 4), two);
            if (off & 1) {
                const uint32_t h[1] = {(off & 4 ? (off & 2 ? w[35] : w[34]) : (off & 2 ? w[33] : w[32])) & 0xffffu};
                St<2, kind>::run(at + (off & 6), h);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) store_shared16(staging + lane * kStagingPitch + 16 * k, w + 4 * k);
    __syncwarp();
    const int piece = lane & 7;
    const bool mine = pieces ? 8 * piece < left : piece > 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = (lane >> 3) + 4 * j;
        const uint4 q = load_shared16(staging + r * kStagingPitch + 16 * piece);
        const uint32_t o[4] = {q.x, q.y, q.z, q.w};
        const uint64_t at = reinterpret_cast<uint64_t>(y + (int64_t)r * cols) & ~(uint64_t)15;
        if (mine && r < live) St<16, kind>::run(reinterpret_cast<char *>(at) + 16 * piece, o);
    }
    __syncwarp();
}

// 64 columns of the activation as two blocks: 32 bytes of codes, two scale bytes.
__device__ __forceinline__ void store_blocks(const Out &o, int row, int col, const uint32_t (&g)[64], const uint32_t (&u)[64],
                                             bool wide) {
    uint32_t codes[8], sc[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float v[32];
        activate<32>(g + 32 * c, u + 32 * c, v);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max(m, magnitude(v[i]));
        sc[c] = scale_byte(m);
        scale_values<32>(v, sc[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) codes[4 * c + i] = codes8(v + 8 * i);
    }
    const int b = col >> 5;
    uint8_t *q = o.q + ((int64_t)row * o.nb + b) * 16;
    if (wide && b + 2 <= o.nb) {
        swiglu::St<32, swiglu::kStPlain>::run(q, codes);
    } else {
        if (b < o.nb) swiglu::St<16, swiglu::kStPlain>::run(q, codes);
        if (b + 1 < o.nb) swiglu::St<16, swiglu::kStPlain>::run(q + 16, codes + 4);
    }
    *reinterpret_cast<uint16_t *>(o.scales + scale_offset(0, row, b, o.chunks)) = (uint16_t)(sc[0] | sc[1] << 8);
}

// tm_w: the W rows of the leader's half of a tile; tm_w2: those of the peer's.  Of the
// first product: gate rows and up rows, each n rows long, so that a last tile reads
// zeros past them; else both all of W.
template <Results kTo>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx4_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_w2, const __grid_constant__ CUtensorMap tm_xs,
                    const __grid_constant__ CUtensorMap tm_ws, Out out, int M, int nb, int chunks, int up_tile) {
    constexpr bool kGated = kTo == kGatedBlocks;
    constexpr int kStages = PairShape<kTo>::kStages;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_addr(smem);
    unsigned char *state = smem + kStages * kPairStage + PairShape<kTo>::kStaging;
    const uint32_t st0 = smem_addr(state);
    const uint32_t full0 = st0 + OFF_FULL, empty0 = st0 + OFF_EMPTY, acc_full0 = st0 + OFF_ACC_FULL,
                   acc_empty = st0 + OFF_ACC_EMPTY, mma_done = st0 + OFF_MMA_DONE, tile_full0 = st0 + OFF_TILE_FULL,
                   tile_empty0 = st0 + OFF_TILE_EMPTY, clc_bar = st0 + OFF_CLC_BAR, clc_resp = st0 + OFF_CLC_RESP,
                   tile_ids_addr = st0 + OFF_TILE_ID, sfull0 = st0 + OFF_SFULL, scales0 = st0 + OFF_SCALES;
    volatile int *tile_ids = reinterpret_cast<volatile int *>(state + OFF_TILE_ID);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(state + OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(state + OFF_ABORT);

    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = (nb + 7) / 8;
    const int tiles_m = (M + 255) / 256;
    const int cols = kGated ? 128 : 256;  // result columns a tile
    const int tiles_n = (out.cols + cols - 1) / cols;
    const int tiles = tiles_m * tiles_n;
    const uint32_t tile_empty_leader0 = map_to_rank(tile_empty0, 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);   // the leader's producer (plus both CTAs' bytes)
            mbar_init(empty0 + 8 * s, 1);  // the leader's commit, multicast to both CTAs
            mbar_init(sfull0 + 8 * s, 1);  // this CTA's producer and its scales' bytes
        }
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(scales0 + 8 * i, 8);  // the scale warps of both CTAs (leader's copy)
        for (int a = 0; a < 2; ++a) mbar_init(acc_full0 + 8 * a, 1);  // the leader's commit, multicast
        mbar_init(acc_empty, 16);  // the epilogue warps of both CTAs (leader's copy)
        mbar_init(mma_done, 1);
        for (int i = 0; i < kTileSlots; ++i) {
            mbar_init(tile_full0 + 8 * i, 1);              // the leader's producer
            mbar_init(tile_empty0 + 8 * i, kTileReaders);  // leader's copy only
        }
        mbar_init(clc_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    swiglu::await_previous_grid();
    swiglu::allow_next_grid();

    // a wait of this thread ran out: both CTAs stop (see settle)
    const auto give_up = [&]() {
        *abort_flag = 1;
        store_cluster(map_to_rank(st0 + OFF_ABORT, rank ^ 1u), 1);
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 0 && lane == 0) {
            // ---- producer (both CTAs); the leader's also schedules
            const CUtensorMap *wmap = leader ? &tm_w : &tm_w2;
            int it = 0, asks = 0;
            int tile = (int)(blockIdx.x >> 1);
            for (int k = 0;; ++k) {
                const int slot = k % kTileSlots;
                if (leader) {
                    if (!wait<true>(tile_empty0 + 8 * slot, ((k / kTileSlots) & 1) ^ 1)) {
                        give_up();
                        tile = -1;
                    }
                    publish_tile(tile_ids_addr, tile_full0, slot, tile);
                } else {
                    tile = -1;
                    if (wait<true>(tile_full0 + 8 * slot, (k / kTileSlots) & 1))
                        tile = tile_ids[slot];
                    else
                        give_up();
                    mbar_arrive_cluster(tile_empty_leader0 + 8 * slot);
                }
                if (tile < 0) break;
                int m0, tn;
                pair_tile(tile, tiles_m, tiles_n, m0, tn);
                const int my_m0 = m0 + 128 * (int)rank;
                // rows of W: 128 of each half (gated), or of the tile's own half
                const int w_row = kGated ? tn * 128 : tn * 256 + 128 * (int)rank;
                const int scale0 = kGated ? tn : 2 * tn, scale1 = kGated ? up_tile + tn : 2 * tn + 1;
                const int ask_at = stages > kAskAhead ? stages - kAskAhead : 0;
                bool asked = false;
                for (int ks = 0; ks < stages && !*abort_flag; ++ks, ++it) {
                    if (leader && ks == ask_at) {
                        mbar_arrive_expect_tx(clc_bar, 16);
                        clc_try_cancel(clc_resp, clc_bar);
                        asked = true;
                    }
                    const int s = it % kStages;
                    if (!wait(empty0 + 8 * s, ((it / kStages) & 1) ^ 1)) {
                        give_up();
                        break;
                    }
                    const uint32_t full = map_to_rank(full0 + 8 * s, 0), at = ring + s * kPairStage;
                    const uint32_t sc = at + 2 * kCodesTile, sfull = sfull0 + 8 * s;
                    mbar_arrive_expect_tx(sfull, 3 * kScalesTile);
                    tma_load_2d(sc, &tm_xs, sfull, 0, (my_m0 >> 7) * chunks + 2 * ks);
                    tma_load_2d(sc + kScalesTile, &tm_ws, sfull, 0, scale0 * chunks + 2 * ks);
                    tma_load_2d(sc + 2 * kScalesTile, &tm_ws, sfull, 0, scale1 * chunks + 2 * ks);
                    if (leader) mbar_arrive_expect_tx(full0 + 8 * s, 4 * kCodesTile);
                    tma_load_2d_pair(at, &tm_x, full, ks * 128, my_m0);
                    tma_load_2d_pair(at + kCodesTile, wmap, full, ks * 128, w_row);
                }
                if (leader) {
                    // the answer is waited for even after an abort, so it never lands in
                    // shared memory the CTA has left
                    int next = -1;
                    if (asked && !wait<true>(clc_bar, asks++ & 1)) {
                        give_up();
                    } else if (asked) {
                        const int x = clc_cancelled_cta(clc_resp);
                        if (x >= 0) {
                            next = x >> 1;
                            if ((x & 1) != 0 || next >= tiles) {  // not a cluster's first CTA of this grid
                                give_up();
                                atomicExch(&g_mx4_timeout, 1);
                                next = -1;
                            }
                        }
                    }
                    tile = *abort_flag ? -1 : next;
                }
            }
            // the leader's full barriers count both CTAs' codes, each CTA's own its scales:
            // once their last phases complete, every load of the pair has landed
            for (int k = it > kStages ? it - kStages : 0; k < it; ++k) {
                if (!wait(sfull0 + 8 * (k % kStages), (k / kStages) & 1)) give_up();
                if (leader && !wait(full0 + 8 * (k % kStages), (k / kStages) & 1)) give_up();
            }
        } else if (warp == 1 && lane == 0 && leader) {
            // ---- products (leader only)
            int it = 0;
            for (int k = 0;; ++k) {
                const int slot = k % kTileSlots;
                int tile = -1;
                if (wait<true>(tile_full0 + 8 * slot, (k / kTileSlots) & 1))
                    tile = tile_ids[slot];
                else
                    give_up();
                mbar_arrive_cluster(tile_empty_leader0 + 8 * slot);
                if (tile < 0 || *abort_flag) break;
                // tile k - 1's shared columns are in registers, and all of tile k - 2
                if (k > 0 && !wait<true>(acc_empty, (k - 1) & 1)) {
                    give_up();
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (k & 1) * kAccShift;
                bool ok = true;
                for (int ks = 0; ks < stages; ++ks, ++it) {
                    const int s = it % kStages;
                    if (!wait(full0 + 8 * s, (it / kStages) & 1) ||
                        !wait<true>(scales0 + 8 * (it % kScaleSlots), (it / kScaleSlots) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = ring + s * kPairStage, b = a + kCodesTile;
                    const uint32_t sfa = tmem + kScaleCol + (it % kScaleSlots) * kScaleCols, sfb = sfa + 8;
                    const int steps = min(4, (nb - 8 * ks + 1) / 2);  // products of 64 columns
    #pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < steps)
                            mma_mxf4_pair(d, smem_desc_128b(a + kk * 32), smem_desc_128b(b + kk * 32),
                                          instr_desc(256, 256, (kk & 1) * 2), sfa + 4 * (kk >> 1), sfb + 8 * (kk >> 1),
                                          (ks | kk) != 0 ? 1u : 0u);
                    mma_commit_both(empty0 + 8 * s);
                }
                if (!ok) {
                    give_up();
                    break;
                }
                mma_commit_both(acc_full0 + 8 * (k & 1));
            }
            mma_commit_local_pair(mma_done);
            if (!wait(mma_done, 0)) give_up();
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ---- scales (both CTAs): a stage's six tiles to this quarter of the lanes
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kScaleCol;
        const uint32_t scales_leader0 = map_to_rank(scales0, 0);
        int it = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k % kTileSlots;
            int tile = -1;
            if (lane == 0) {
                if (wait<true>(tile_full0 + 8 * slot, (k / kTileSlots) & 1)) tile = tile_ids[slot];
                mbar_arrive_cluster(tile_empty_leader0 + 8 * slot);
            }
            tile = __shfl_sync(0xffffffffu, tile, 0);
            if (tile < 0 || __shfl_sync(0xffffffffu, *abort_flag, 0)) break;
            for (int ks = 0; ks < stages && ok; ++ks, ++it) {
                const int s = it % kStages, done = it - kScaleSlots;
                ok = wait(sfull0 + 8 * s, (it / kStages) & 1);
                const uint32_t at = ring + s * kPairStage + 2 * kCodesTile + lane * 16;
                uint4 v[6];  // x, W's two halves: first tile, second tile
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    v[c] = load_shared16(at + c * kTileBytes);
                    v[2 + 2 * c] = load_shared16(at + kScalesTile + c * kTileBytes);
                    v[3 + 2 * c] = load_shared16(at + 2 * kScalesTile + c * kTileBytes);
                }
                // the products that used this slot before are done
                if (ok && done >= 0) ok = wait(empty0 + 8 * (done % kStages), (done / kStages) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    if (lane == 0) *abort_flag = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t to = lanes + (it % kScaleSlots) * kScaleCols;
                tmem_store8(to, v[0], v[1]);
                tmem_store8(to + 8, v[2], v[3]);
                tmem_store8(to + 16, v[4], v[5]);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                // (the stores to tensor memory are complete; see mbar_arrive_cluster_read)
                if (lane == 0) mbar_arrive_cluster_read(scales_leader0 + 8 * (it % kScaleSlots));
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        // ---- epilogue (both CTAs): this CTA's 128 rows of the accumulator
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t acc_empty_leader = map_to_rank(acc_empty, 0);
        const bool wide = out.nb % 2 == 0 && reinterpret_cast<uintptr_t>(out.q) % 32 == 0;
        const bool pieces = out.cols % 8 == 0 && reinterpret_cast<uintptr_t>(out.y) % 16 == 0;
        const uint32_t staging = ring + kStages * kPairStage + (warp - 4) * 32 * kStagingPitch;
        // the warp leaves the loop as one: tile id, abort flag and waits are warp-uniform
        for (int k = 0;; ++k) {
            const int slot = k % kTileSlots, acc = k & 1;
            int tile = -1;
            if (lane == 0) {
                if (wait<true>(tile_full0 + 8 * slot, (k / kTileSlots) & 1)) tile = tile_ids[slot];
                mbar_arrive_cluster(tile_empty_leader0 + 8 * slot);
            }
            tile = __shfl_sync(0xffffffffu, tile, 0);
            if (tile < 0 || __shfl_sync(0xffffffffu, *abort_flag, 0)) break;
            int m0, tn;
            pair_tile(tile, tiles_m, tiles_n, m0, tn);
            const int row = m0 + 128 * (int)rank + 32 * quarter + lane;
            // the shared columns: the last 72 of the first accumulator, the first 72 of the
            // second.  A warp that has some of them (a gated one does: its gate and up
            // columns lie 128 apart) arrives when it has read them, the others once this
            // tile's products are done, since they have read the tile before.  No warp
            // arrives for a tile before that: its products start when every warp has arrived
            // for the tile before, so no warp counts twice among the 16 of a tile (one that
            // arrived without waiting would take the place of a warp that has still to read)
            const bool sharing = kGated || half != acc;
            if (!__all_sync(0xffffffffu, wait(acc_full0 + 8 * acc, (k >> 1) & 1))) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const auto read = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_read(acc_empty_leader);
            };
            if (!sharing) read();
            const uint32_t base = tmem + ((uint32_t)(32 * quarter) << 16) + acc * kAccShift;
            uint32_t v[64], u[64];
            const auto load64 = [&](int col, uint32_t(&to)[64]) {
                tmem_load32(base + col, reinterpret_cast<uint32_t(&)[32]>(to[0]));
                tmem_load32(base + col + 32, reinterpret_cast<uint32_t(&)[32]>(to[32]));
            };
            const int first = kGated ? 64 * half : 128 * half, second = kGated ? 128 + 64 * half : first + 64;
            load64(first, v);
            load64(second, u);
            tmem_wait_ld();
            if (sharing) read();
            if constexpr (kGated) {
                if (row < M) store_blocks(out, row, tn * 128 + first, v, u, wide);
            } else if constexpr (kTo == kWholePacks) {
                if (row < M) {
                    __nv_bfloat16 *y = out.y + (int64_t)row * out.cols + tn * 256;
                    store64(y + first, v, tn * 256 + first, out.cols);
                    store64(y + second, u, tn * 256 + second, out.cols);
                }
            } else {
                const int col = tn * 256 + first, live = M - (row - lane);
                __nv_bfloat16 *y = out.y + (int64_t)(row - lane) * out.cols + col;
                store64_any(y, out.cols, v, out.cols - col, live, pieces, staging);
                store64_any(y + 64, out.cols, u, out.cols - col - 64, live, pieces, staging);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal it
    if (threadIdx.x == 0 && *abort_flag) settle();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- host side ---

namespace {

using moe::Span;

// A tensor in 4 bits, of one part or of the part that starts at `row`.
struct Operand {
    const uint8_t *q;
    const uint8_t *scales;
    int64_t rows, cols, parts;
};

// Codes [rows, 16 nb] bytes: boxes of 128 bytes by `box` rows, zeros outside.
bool codes_map(EncodeTiled enc, CUtensorMap *map, const uint8_t *q, int64_t rows, int64_t cols, int box) {
    const cuuint64_t pitch = (cuuint64_t)blocks_of(cols) * 16;
    const cuuint64_t dims[2] = {pitch, (cuuint64_t)rows}, strides[1] = {pitch};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(q), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles, [tiles * chunks][512] bytes: boxes of two.
bool scales_map(EncodeTiled enc, CUtensorMap *map, const Operand &t) {
    const cuuint64_t dims[2] = {128, (cuuint64_t)(scale_bytes(t.rows, t.cols, t.parts) / kTileBytes)}, strides[1] = {kTileBytes};
    const cuuint32_t boxes[2] = {128, 2}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(t.scales), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// The kernel's shared memory, allowed once per device.
template <auto kernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && done[dev].load()) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true);
    return e;
}

// X: see the kernel; x.q and x.scales are not read where it is not void.
template <int NT, int TILES, int PER_SM, typename X = void>
swiglu_status_t run_split(const Operand &x, const Operand &w, const Out &out, int slices, bool early, swiglu_stream_t stream,
                          Rows16 rows = {}) {
    using S = SplitShape<NT, TILES, PER_SM>;
    EncodeTiled enc;
    cudaError_t e = encoder(enc);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    const int64_t wrows = w.rows / TILES, nb = blocks_of(x.cols);
    CUtensorMap tm_w, tm_up, tm_x, tm_ws, tm_xs;
    if (!codes_map(enc, &tm_w, w.q, wrows, w.cols, 128) ||
        !codes_map(enc, &tm_up, w.q + (TILES - 1) * wrows * nb * 16, wrows, w.cols, 128) ||
        !scales_map(enc, &tm_ws, w))
        return moe::cuda_fail(cudaErrorInvalidValue);
    if constexpr (std::is_void_v<X>) {
        if (!codes_map(enc, &tm_x, x.q, x.rows, x.cols, NT) || !scales_map(enc, &tm_xs, x))
            return moe::cuda_fail(cudaErrorInvalidValue);
    } else {
        tm_x = tm_w;  // not used
        tm_xs = tm_ws;
    }
    if ((e = allow_smem<mx4_split_kernel<NT, TILES, PER_SM, X>>(S::kSmem)) != cudaSuccess) return moe::cuda_fail(e);
    const int64_t tiles = tiles_of(wrows), ytiles = (x.rows + NT - 1) / NT;
    e = moe::launch(mx4_split_kernel<NT, TILES, PER_SM, X>, dim3((unsigned)(tiles * ytiles * slices)), S::kThreads, S::kSmem, stream,
                    slices, tm_w, tm_up, tm_x, tm_ws, tm_xs, rows, out, (int)x.rows, (int)nb, (int)chunks_of(x.cols), (int)tiles, early ? 1 : 0);
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

template <Results kTo>
swiglu_status_t run_pair(const Operand &x, const Operand &w, const Out &out, swiglu_stream_t stream) {
    constexpr bool kGated = kTo == kGatedBlocks;
    EncodeTiled enc;
    cudaError_t e = encoder(enc);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    const int64_t wrows = kGated ? w.rows / 2 : w.rows, nb = blocks_of(x.cols);
    CUtensorMap tm_x, tm_w, tm_w2, tm_xs, tm_ws;
    if (!codes_map(enc, &tm_x, x.q, x.rows, x.cols, 128) || !codes_map(enc, &tm_w, w.q, wrows, w.cols, 128) ||
        !codes_map(enc, &tm_w2, w.q + (kGated ? wrows * nb * 16 : 0), wrows, w.cols, 128) || !scales_map(enc, &tm_xs, x) ||
        !scales_map(enc, &tm_ws, w))
        return moe::cuda_fail(cudaErrorInvalidValue);
    if ((e = allow_smem<mx4_pair_kernel<kTo>>(PairShape<kTo>::kSmem)) != cudaSuccess) return moe::cuda_fail(e);
    const int64_t tiles = (x.rows + 255) / 256 * ((out.cols + (kGated ? 127 : 255)) / (kGated ? 128 : 256));
    if (tiles > INT32_MAX / 2) return SWIGLU_ERR_SHAPE;
    // one cluster per tile; the pairs that start take the others' tiles
    e = moe::launch(mx4_pair_kernel<kTo>, dim3((unsigned)(2 * tiles)), kPairThreads, PairShape<kTo>::kSmem, stream, 0, tm_x, tm_w,
                    tm_w2, tm_xs, tm_ws, out, (int)x.rows, (int)nb, (int)chunks_of(x.cols), (int)tiles_of(wrows));
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

constexpr int64_t kSms = 152;

// What the two kernels take, in ns, fitted to times of [129 .. 2048] rows by [1000 ..
// 28672] by [512 .. 14336]: a CTA of the split kernel takes one tile, its start and end
// in full; a pair takes the next tile while it finishes one.  ([256, 14336] x [4096,
// 14336] 13.4 and 24.0 us, [1024, 14336] x [4096, 14336] 27.4 and 24.4 us.)  Beyond that range
// it decides well for many rows by many columns (8192 x 1000 x 512 11.0 and 10.3 us, 4096 x
// 4096 x 14336 101 and 83 us), and takes pairs too early below 129 rows (100 x 20000 x 256
// 4.5 and 6.9 us) and for up to 256 columns (30000 x 100 x 300 7.3 and 18.7 us).
int64_t split_cost(int64_t ctas, int tiles, int64_t stages) {
    if (tiles == 1 && ctas > kSms) return (ctas + 2 * kSms - 1) / (2 * kSms) * (300 * stages + 11000);  // two an SM
    return (ctas + kSms - 1) / kSms * (tiles == 1 ? 214 * stages + 5600 : 380 * stages + 6500);
}
int64_t pair_cost(int64_t rows, int64_t cols, int tiles, int64_t stages) {
    const int64_t width = tiles == 1 ? 256 : 128;
    const int64_t n = (rows + 255) / 256 * ((cols + width - 1) / width);
    return 6500 + (n + kSms / 2 - 1) / (kSms / 2) * (340 * stages + 1000);
}

// As many slices as one wave of CTAs holds (two an SM for few rows, see SplitShape), each of
// two stages at least.
int slices_of(int64_t tiles, int nt, int64_t stages) {
    const int64_t wave = nt <= 32 ? 2 * kSms : kSms;
    int slices = 1;
    while (slices < 8 && tiles * slices * 2 <= wave && stages >= 4 * slices) slices *= 2;
    return slices;
}

template <int TILES>
swiglu_status_t product(const Operand &x, const Operand &w, const Out &out, bool early, swiglu_stream_t stream) {
    const int64_t M = x.rows;
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const int64_t tiles = tiles_of(w.rows / TILES), ytiles = (M + nt - 1) / nt;
    if (tiles * ytiles * 8 > INT32_MAX || tiles_of(M) * chunks_of(x.cols) > INT32_MAX - 2 ||
        tiles * TILES * chunks_of(x.cols) > INT32_MAX - 2)
        return SWIGLU_ERR_SHAPE;
    const int64_t stages = (blocks_of(x.cols) + 7) / 8;
    const int slices = slices_of(tiles * ytiles, nt, stages);
    if (M > 64 && pair_cost(M, out.cols, TILES, stages) <
                      split_cost(tiles * ytiles * slices, TILES, (stages + slices - 1) / slices)) {
        if constexpr (TILES == 2) return run_pair<kGatedBlocks>(x, w, out, stream);
        const bool packs = out.cols % 16 == 0 && (uintptr_t)out.y % 32 == 0;
        return packs ? run_pair<kWholePacks>(x, w, out, stream) : run_pair<kAnyRows>(x, w, out, stream);
    }
    const bool two = TILES == 1 && tiles * ytiles * slices > kSms;
    switch (nt) {
        case 16: return run_split<16, TILES, 2>(x, w, out, slices, early, stream);
        case 32: return run_split<32, TILES, 2>(x, w, out, slices, early, stream);
        case 64:
            if constexpr (TILES == 1)
                if (two) return run_split<64, TILES, 2>(x, w, out, slices, early, stream);
            return run_split<64, TILES, 1>(x, w, out, slices, early, stream);
        default:
            if constexpr (TILES == 1)
                if (two) return run_split<128, TILES, 2>(x, w, out, slices, early, stream);
            return run_split<128, TILES, 1>(x, w, out, slices, early, stream);
    }
}

// Scratch of the MLP: x and the activation in 4 bits, each part 256-byte aligned.
struct Scratch {
    int64_t xq, xs, yq, ys, bytes;
};

Scratch scratch_of(int64_t M, int64_t H, int64_t n) {
    const auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    Scratch s;
    s.xq = 0;
    s.xs = s.xq + up(q_bytes(M, H));
    s.yq = s.xs + up(scale_bytes(M, H, 1));
    s.ys = s.yq + up(q_bytes(M, n));
    s.bytes = s.ys + up(scale_bytes(M, n, 1));
    return s;
}

bool aligned16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if ((uintptr_t)p % 16 != 0) return false;
    return true;
}

swiglu_status_t zero(void *y, int64_t bytes, swiglu_stream_t stream) {
    const cudaError_t e = cudaMemsetAsync(y, 0, (size_t)bytes, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

}  // namespace
}  // namespace mx4

extern "C" {

swiglu_status_t swiglu_mx4_mm_fwd(const void *x_q, const void *x_scales, const void *w_q, const void *w_scales, void *y,
                                  int64_t M, int64_t N, int64_t K, swiglu_dtype_t dtype, swiglu_stream_t stream) {
    using namespace mx4;
    if (dtype != SWIGLU_BF16) return SWIGLU_ERR_DTYPE;
    if (!sizes_ok(M, K) || !sizes_ok(N, K)) return SWIGLU_ERR_SHAPE;
    if (M == 0 || N == 0) return SWIGLU_OK;
    if (y == nullptr || (K > 0 && (x_q == nullptr || x_scales == nullptr || w_q == nullptr || w_scales == nullptr)))
        return SWIGLU_ERR_NULL;
    Span sy, sxq, sxs, swq, sws;
    if (!moe::span_of(y, M, N, N, 2, sy)) return SWIGLU_ERR_SHAPE;
    if ((uintptr_t)y % 2 != 0) return SWIGLU_ERR_STRIDE;
    if (K == 0) return zero(y, M * N * 2, stream);
    if (!span_bytes(x_q, q_bytes(M, K), sxq) || !span_bytes(x_scales, scale_bytes(M, K, 1), sxs) ||
        !span_bytes(w_q, q_bytes(N, K), swq) || !span_bytes(w_scales, scale_bytes(N, K, 1), sws))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sy}, {sxq, sxs, swq, sws})) return SWIGLU_ERR_ALIAS;
    if (!aligned16({x_q, x_scales, w_q, w_scales})) return SWIGLU_ERR_STRIDE;
    const Operand x{static_cast<const uint8_t *>(x_q), static_cast<const uint8_t *>(x_scales), M, K, 1};
    const Operand w{static_cast<const uint8_t *>(w_q), static_cast<const uint8_t *>(w_scales), N, K, 1};
    return product<1>(x, w, Out{static_cast<__nv_bfloat16 *>(y), nullptr, nullptr, (int32_t)N, 0, 0}, false, stream);
}

swiglu_status_t swiglu_mx4_mlp_workspace_size(int64_t M, int64_t H, int64_t n, size_t *bytes) {
    using namespace mx4;
    if (bytes == nullptr) return SWIGLU_ERR_NULL;
    if (!sizes_ok(M, H) || !sizes_ok(M, n)) return SWIGLU_ERR_SHAPE;
    *bytes = (size_t)scratch_of(M, H, n).bytes;
    return SWIGLU_OK;
}

swiglu_status_t swiglu_mx4_mlp_fwd(const void *x, const void *w1_q, const void *w1_scales, const void *w2_q,
                                   const void *w2_scales, void *out, void *workspace, size_t workspace_bytes, int64_t M,
                                   int64_t H, int64_t n, int64_t N, int64_t x_row_stride, swiglu_dtype_t dtype,
                                   swiglu_stream_t stream) {
    using namespace mx4;
    const int eb = dtype == SWIGLU_BF16 ? 2 : dtype == SWIGLU_F32 ? 4 : 0;
    if (eb == 0) return SWIGLU_ERR_DTYPE;
    if (!sizes_ok(M, H) || !sizes_ok(M, n) || !sizes_ok(N, n) || n > SWIGLU_MX4_MAX_ROWS / 2) return SWIGLU_ERR_SHAPE;
    if (M == 0 || N == 0) return SWIGLU_OK;
    if (out == nullptr) return SWIGLU_ERR_NULL;
    Span so;
    if (!moe::span_of(out, M, N, N, 2, so)) return SWIGLU_ERR_SHAPE;
    if ((uintptr_t)out % 2 != 0) return SWIGLU_ERR_STRIDE;
    if (H == 0 || n == 0) return zero(out, M * N * 2, stream);  // the activation is zero, or there is none
    if (x == nullptr || w1_q == nullptr || w1_scales == nullptr || w2_q == nullptr || w2_scales == nullptr)
        return SWIGLU_ERR_NULL;
    if (x_row_stride < H) return SWIGLU_ERR_STRIDE;
    const Scratch s = scratch_of(M, H, n);
    Span sx, s1q, s1s, s2q, s2s, sw;
    if (!moe::span_of(x, M, H, x_row_stride, eb, sx) || !span_bytes(w1_q, q_bytes(2 * n, H), s1q) ||
        !span_bytes(w1_scales, scale_bytes(2 * n, H, 2), s1s) || !span_bytes(w2_q, q_bytes(N, n), s2q) ||
        !span_bytes(w2_scales, scale_bytes(N, n, 1), s2s))
        return SWIGLU_ERR_SHAPE;
    if (workspace == nullptr || workspace_bytes < (size_t)s.bytes || !aligned16({workspace})) return SWIGLU_ERR_WORKSPACE;
    if (!span_bytes(workspace, s.bytes, sw)) return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({so, sw}, {sx, s1q, s1s, s2q, s2s})) return SWIGLU_ERR_ALIAS;
    if ((uintptr_t)x % eb != 0 || !aligned16({w1_q, w1_scales, w2_q, w2_scales})) return SWIGLU_ERR_STRIDE;
    uint8_t *at = static_cast<uint8_t *>(workspace);
    const Operand xo{at + s.xq, at + s.xs, M, H, 1}, yo{at + s.yq, at + s.ys, M, n, 1};
    const Operand w1{static_cast<const uint8_t *>(w1_q), static_cast<const uint8_t *>(w1_scales), 2 * n, H, 2};
    const Operand w2{static_cast<const uint8_t *>(w2_q), static_cast<const uint8_t *>(w2_scales), N, n, 1};
    const Out act{nullptr, at + s.yq, at + s.ys, (int32_t)n, (int32_t)blocks_of(n), (int32_t)chunks_of(n)};
    swiglu_status_t st;
    if (M <= 16 && H % 32 == 0 && x_row_stride * eb % 16 == 0 && aligned16({x})) {
        // the first product's CTAs round the few rows themselves
        const int64_t tiles = tiles_of(n), stages = (blocks_of(H) + 7) / 8;
        if (tiles * 8 > INT32_MAX || 2 * tiles * chunks_of(H) > INT32_MAX - 2) return SWIGLU_ERR_SHAPE;
        const int slices = slices_of(tiles, 16, stages);
        const Rows16 rows{static_cast<const char *>(x), x_row_stride * eb};
        st = dtype == SWIGLU_BF16 ? run_split<16, 2, 2, swiglu::BF16>(xo, w1, act, slices, false, stream, rows)
                                  : run_split<16, 2, 2, swiglu::F32>(xo, w1, act, slices, false, stream, rows);
    } else {
        st = launch_quantize(x, at + s.xq, at + s.xs, M, H, 1, x_row_stride, dtype, stream);
        if (st == SWIGLU_OK) st = product<2>(xo, w1, act, true, stream);
    }
    if (st != SWIGLU_OK) return st;
    return product<1>(yo, w2, Out{static_cast<__nv_bfloat16 *>(out), nullptr, nullptr, (int32_t)N, 0, 0}, true, stream);
}

swiglu_status_t swiglu_mx4_timeout_flag(int *flag) {
    if (flag == nullptr) return SWIGLU_ERR_NULL;
    const cudaError_t e = cudaMemcpyFromSymbol(flag, mx4::g_mx4_timeout, sizeof(int));
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

}  // extern "C"
