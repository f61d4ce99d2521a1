// grouped_mm.cu -- the routed experts' matrix products on the tensor cores
// (tcgen05, TMEM, TMA, CTA pairs): one weight matrix per expert, rows sorted by
// expert, ragged groups.
//
//   forward      y[t]  = W[e] x[t]                 (kMm)
//   first layer  y[t]  = probs[t] silu(Wg[e] x[t]) * (Wu[e] x[t])   (kFc1)
//   data grad    dx[t] = W[e]^T dy[t]              (kDgrad)
//   weight grad  dW[e] = sum_t dy[t]^T x[t]        (kWgrad)
//
// A cluster of two CTAs computes a tile with tcgen05.mma.cta_group::2 (M = 256:
// 128 accumulator lanes in each CTA's tensor memory; N a multiple of 32 up to
// 256; bf16 in, fp32 accumulate).  In the three products over rows the FEATURES
// (rows of W, or its columns for the data gradient) are the M side and the rows
// t are the N side: N is a field of the instruction, so the last tile of a
// group is as wide as its rows need, to 32, where rows on the M side would pad
// every group to 256 (with 64 groups of 128 rows on average, half the work).
// The weight gradient has W's rows as M and its columns as N.  A block of 64 of the
// contraction takes a pair 516 cycles at 256 rows, where the tensor cores need 512;
// a tile of w rows fewer is bound by the SM's 64 bytes a cycle from L2, 256 + w
// cycles.  16384 rows over 8 groups of [14336, 4096], at the GPU's power limit: 1735
// TFLOP/s forward, 1672 fc1 with its checkpoint, 1655 and 1705 the gradients.
//
// Operand tiles are 64 elements of the contraction deep, 128-byte swizzle.
// Where the contraction runs along memory rows the tile is K-major; the data
// gradient's W and both operands of the weight gradient have it across memory
// rows and are loaded as they lie (MN-major descriptors): nothing is
// transposed in memory.
//
// The ring of six 32 KiB stages, the two accumulators and the scheduling by
// cluster launch control follow fc1_swiglu.cu; a warp of its own takes the tiles
// and finds their groups.  The number of tiles depends on
// the groups, which only the device knows: the grid holds as many clusters as
// the sizes allow at most, and a pair that finds its tile beyond the last one
// drops it.
//
// The weight gradient's contraction runs over a group's rows, so its last block
// of 64 would take in rows of the next group (and a product with 0 would not do
// for them: a neighbour's row may hold NaN).  The pair kernel puts that block
// together from boxes of 1, 2, 4, ... 32 rows, and up to the next multiple of 16,
// an instruction's depth, from boxes beyond the tensor's end, which are filled with
// zeros: the tensor cores see nothing but what TMA wrote.  (Zeroing the rows from a
// warp instead, handed on with a release to the other CTA, took 2000 cycles per
// tile that the ring did not cover.)
#include <climits>

#include "ckpt8.cuh"
#include "moe_host.h"
#include "swiglu_kernels.cuh"
#include "tc_pair.cuh"

namespace gmm {

using namespace tc;

enum : int { kFc1 = 0, kMm = 1, kDgrad = 2, kWgrad = 3 };

constexpr int BK = 64;               // contraction elements per stage
constexpr int UMMA_K = 16;           // per tcgen05.mma of kind::f16
constexpr int TILE_N = 256;          // accumulator columns per tile at most
constexpr int A_BYTES = 128 * BK * 2;            // a CTA's half of the M side
constexpr int STAGE_BYTES = 2 * A_BYTES;         // and at most as much of the N side
constexpr int STAGES = 6;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int TMEM_COLS = 2 * TILE_N;            // two accumulators
constexpr int kMaxGroups = SWIGLU_MAX_GROUPS;
constexpr int kGroupN = 16;          // N tiles per block of the tile order
// The tensor cores truncate the running fp32 sum at every step of 16 terms, by less
// than 2^-23 of it: for a weight gradient over rows of one sign 1.4e-5 of the sum was
// measured for 4096 rows, 3.9e-4 for 65,536 and 6.8e-3 for 1,048,576 (of random signs
// 4.4e-6, 7.6e-5 and 1.2e-3).  Where more than kSegmentRows (fp32 result) or kLongRows
// (bf16: a quarter of its rounding) could meet in one sum, the kernels with SUMS add
// up segments of kSegmentRows with rounded additions, in the epilogue's registers: the
// two accumulators take turns, and while one is read the other is summed in.  What is
// left in fp32: 9e-7 of one sign, 5e-7 of random signs, over any number of rows.  Eight
// groups of 2048 rows, [4096, 7168]: 634 us, 618 in one sum each; 6932 rows, [5224, 10240],
// 509 us, 548 with segments of 4096 rows that were added in dW.
constexpr int kSegmentRows = 512;
constexpr int kLongRows = 131072;

constexpr int kTileSlots = 2;
// byte offsets in the region after the ring
constexpr int OFF_FULL = 0;
constexpr int OFF_EMPTY = OFF_FULL + 8 * STAGES;
constexpr int OFF_ACC_FULL = OFF_EMPTY + 8 * STAGES;
constexpr int OFF_ACC_EMPTY = OFF_ACC_FULL + 16;
constexpr int OFF_MMA_DONE = OFF_ACC_EMPTY + 16;
constexpr int OFF_TILE_FULL = OFF_MMA_DONE + 8;
constexpr int OFF_TILE_EMPTY = OFF_TILE_FULL + 8 * kTileSlots;
constexpr int OFF_CLC_BAR = OFF_TILE_EMPTY + 8 * kTileSlots;
constexpr int OFF_CLC_RESP = (OFF_CLC_BAR + 8 + 15) / 16 * 16;
constexpr int OFF_TILE = (OFF_CLC_RESP + 16 + 31) / 32 * 32;  // tile[kTileSlots], 32 bytes each
constexpr int OFF_TMEM = OFF_TILE + 32 * kTileSlots;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int STATE_BYTES = 512;
static_assert(OFF_ABORT + 4 <= STATE_BYTES, "barriers and state fit their region");
// the epilogue's staging, per warp: 32 rows of 64 bytes for bulk stores (64-byte
// swizzle); kFc1: 16 rows of 32 gates and 32 ups per pair of warps, fp32, rows
// padded by 4 words
constexpr int STG_WARP_BYTES = 32 * 64;
constexpr int STG_ROW_FC1 = 68;
constexpr int STG_PAIR_FC1 = 16 * STG_ROW_FC1 * 4;
constexpr int STG_BYTES = 18 * 1024;
constexpr int TABLE_BYTES = 2 * (kMaxGroups + 2) * 4;
constexpr int SMEM_BYTES = RING_BYTES + STG_BYTES + STATE_BYTES + (TABLE_BYTES + 15) / 16 * 16 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "fits one SM");

__device__ int g_timeout = 0;

template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    return mbar_wait_or_flag<kCluster>(bar, parity, &g_timeout);
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

struct Params {
    CUtensorMap a;     // the M side
    CUtensorMap b[8];  // the N side, boxes of 16, 32, 48, ... 128 rows (kWgrad: b[0] alone, 64 rows)
    CUtensorMap part_a[6], part_b[6];  // kWgrad, a group's last rows: boxes of 1, 2, ... 32 rows
    CUtensorMap c;     // the result (not kFc1), boxes of 64 bytes by 32 rows
    const int32_t *ends;
    const float *probs;      // kFc1
    void *out;               // y, dx or dW
    __nv_bfloat16 *fc1;      // kFc1: what the backward keeps
    uint8_t *q;
    uint8_t *scales;
    int rows, groups;
    int features;    // kFc1: n; kMm: N; kDgrad: K; kWgrad: N
    int cols;        // kWgrad: K (split kernel: features K and cols N)
    int depth;       // contraction length (kWgrad: unused)
    int f32_out, accumulate;  // kWgrad
};

// Features of a tile: kFc1 has a gate and an up row for each.
template <int MODE>
constexpr int kTileF = MODE == kFc1 ? 128 : 256;

// Where the tiles of a call lie.  starts[e] is group e's first row (e < groups;
// starts[groups] the first row of no group, starts[groups + 1] = rows) and
// base[e] its first tile.
struct Groups {
    const int *starts;
    const int *base;
};

struct Tile {
    int group, m0, n0, cnt;  // first feature, first row (kWgrad: column), rows (kWgrad: columns)
    int r0, rows;            // the group's rows
};

// Write a tile (group -1: none left) into the slot at `slot` of both CTAs, counted
// as bytes on each CTA's barrier `bar`; read one.
constexpr uint32_t kTileBytes = 24;

__device__ __forceinline__ void publish(uint32_t slot, uint32_t bar, const Tile &t) {
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r) {
        const uint32_t to = map_to_rank(slot, r), on = map_to_rank(bar, r);
        asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(on),
                     "r"(kTileBytes)
                     : "memory");
        asm volatile(
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(to),
            "r"(on), "r"(t.group), "r"(t.m0), "r"(t.n0), "r"(t.cnt)
            : "memory");
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%2, %3}, [%1];" ::"r"(to + 16),
                     "r"(on), "r"(t.r0), "r"(t.rows)
                     : "memory");
    }
}

__device__ __forceinline__ Tile read_tile(uint32_t slot) {
    Tile t;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(t.group), "=r"(t.m0), "=r"(t.n0), "=r"(t.cnt)
                 : "r"(slot)
                 : "memory");
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(t.r0), "=r"(t.rows) : "r"(slot + 16) : "memory");
    return t;
}

// Fill starts and base (one warp) for tiles of TF features by at most TN rows
// (kWgrad: columns).  The last "group" is that of the rows that belong to none.
// A lane takes Q neighbouring groups, so that many are read and scanned at a time.
template <int MODE, int TF, int TN, int Q>
__device__ void build_groups_by(const Params &p, int *starts, int *base) {
    const int lane = threadIdx.x & 31;
    const int tf = (p.features + TF - 1) / TF;
    const int per_group = MODE == kWgrad ? tf * ((p.cols + TN - 1) / TN) : 0;
    int end_before = 0, tiles_before = 0;
    for (int e0 = 0; e0 <= p.groups; e0 += 32 * Q) {
        const int e = e0 + lane * Q;
        int end[Q];
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            end[j] = e + j == p.groups ? p.rows : 0;
            if (e + j < p.groups) asm volatile("ld.global.b32 %0, [%1];" : "=r"(end[j]) : "l"(p.ends + e + j) : "memory");
        }
        int most = end_before;  // of the groups up to this lane's last
#pragma unroll
        for (int j = 0; j < Q; ++j) most = max(most, min(end[j], p.rows));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, most, o);
            if (lane >= o) most = max(most, v);
        }
        int start = __shfl_up_sync(0xffffffffu, most, 1);
        if (lane == 0) start = end_before;
        int first[Q], tiles[Q], mine = 0;
#pragma unroll
        for (int j = 0, at = start; j < Q; ++j) {
            first[j] = at;
            at = end[j] = max(at, min(end[j], p.rows));
            if (MODE == kWgrad)
                tiles[j] = e + j < p.groups ? per_group : 0;
            else
                tiles[j] = e + j <= p.groups ? (at - first[j] + TN - 1) / TN * tf : 0;
            mine += tiles[j];
        }
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        int at = tiles_before + sum - mine;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            if (e + j <= p.groups) {
                starts[e + j] = first[j];
                base[e + j] = at;
                if (e + j == p.groups) {
                    starts[e + j + 1] = end[j];
                    base[e + j + 1] = at + tiles[j];
                }
            }
            at += tiles[j];
        }
        end_before = __shfl_sync(0xffffffffu, most, 31);
        tiles_before += __shfl_sync(0xffffffffu, sum, 31);
    }
    __syncwarp();
}

// With one group per lane 64 rows over 256 experts [512, 1024] took 11.7 us instead of
// 9.5; with four, calls of few groups take 0.1 - 0.2 us longer.
template <int MODE, int TF, int TN>
__device__ __forceinline__ void build_groups(const Params &p, int *starts, int *base) {
    if (p.groups < 32)
        build_groups_by<MODE, TF, TN, 1>(p, starts, base);
    else
        build_groups_by<MODE, TF, TN, 4>(p, starts, base);
}

// Tile order: within a group, blocks of up to kGroupN N tiles; within a block
// the N tile varies fastest, so a slab of W is read from HBM once per block and
// the block's rows stay in L2.
// N tiles of a group are equal, to STEP rows (the last one may be shorter).
template <int MODE, int TF, int TN, int STEP>
__device__ __forceinline__ Tile tile_at(const Params &p, const Groups &g, int t) {
    int lo = 0, hi = p.groups;  // the last e with base[e] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.base[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    Tile o;
    o.group = lo;
    o.r0 = g.starts[lo];
    o.rows = g.starts[lo + 1] - o.r0;
    const int extent = MODE == kWgrad ? p.cols : o.rows;
    const int nt = (extent + TN - 1) / TN;
    const int tf = (p.features + TF - 1) / TF;
    const int local = t - g.base[lo];
    if (MODE != kWgrad && nt <= 1) {  // (saves four divisions, 300 cycles of a short call)
        o.m0 = local * TF;
        o.n0 = 0;
        o.cnt = extent;
        return o;
    }
    const int block = local / (kGroupN * tf);
    const int first = block * kGroupN;
    const int width = min(kGroupN, nt - first);
    const int in = local - block * (kGroupN * tf);
    o.m0 = in / width * TF;
    const int j = first + in % width;
    const int step = MODE == kWgrad ? TN : ((extent + nt - 1) / nt + STEP - 1) / STEP * STEP;
    o.n0 = j * step;
    o.cnt = min(step, extent - o.n0);
    return o;
}

__device__ __forceinline__ float4 lds128(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// y for N gates and ups of one row, from fp32, rounded once: the operations of
// the streaming kernels (swiglu::activation), with the row weight last.  Without a
// gate below -64 two elements go through each multiplication and addition (each
// lane rounded as the scalar operation rounds).
template <int N>
__device__ __forceinline__ void activate(const float (&g)[N], const float (&u)[N], float w, uint32_t (&out)[N / 2]) {
    float gmin = g[0];
#pragma unroll
    for (int i = 1; i < N; ++i) gmin = fminf(gmin, g[i]);
    if (gmin < -64.0f) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float r[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const swiglu::Act act = swiglu::activation<swiglu::BF16, false, true>(g[i + h]);
                r[h] = __fmul_rn(__fmul_rn(__fmul_rn(act.silu, u[i + h]), w), act.scale);
            }
            swiglu::BF16::put2(out, i, r[0], r[1]);
        }
    } else {
        using namespace swiglu;
        const uint64_t neg_log2e = x2(-kLog2e, -kLog2e), one = x2(1.0f, 1.0f), w2 = x2(w, w);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint64_t g2 = x2(g[i], g[i + 1]), u2 = x2(u[i], u[i + 1]);
            float t0, t1, d0, d1, r0, r1;
            x2_split(mul_x2(g2, neg_log2e), t0, t1);
            x2_split(add_x2(one, x2(ex2_approx(t0), ex2_approx(t1))), d0, d1);
            const uint64_t s2 = x2(rcp_approx(d0), rcp_approx(d1));
            x2_split(mul_x2(mul_x2(mul_x2(g2, s2), u2), w2), r0, r1);
            BF16::put2(out, i, r0, r1);
        }
    }
}

// True in both warps of a pair (barrier `id`) when `v` holds in either.
__device__ __forceinline__ bool any_of_pair(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.ne.u32 p, %2, 0;\n"
        "bar.red.or.pred q, %1, 64, p;\n"
        "selp.u32 %0, 1, 0, q;\n"
        "}\n"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Instruction descriptor of tcgen05.mma kind::f16: fp32 accumulator (bits 4-5 =
// 1), A and B bf16 (bits 7-9 and 10-12 = 1), A / B MN-major (bits 15, 16), N / 8
// in bits 17-22, M / 16 in bits 24-28 (M = 256 across a pair).
__device__ __forceinline__ uint32_t instr_desc(bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Warps: 0 loads, 1 MMA, 2 .. epilogue, then the scheduler.  The epilogue has two warps per quarter of the accumulator's
// lanes, which take every other chunk of columns each (with one the tile of a
// short contraction took 3.1 instead of 2.2 us, kFc1 5.4 instead of 3.5).
constexpr int kEpi = 8;
constexpr int kScheduler = 2 + kEpi;
constexpr int kPairThreads = 32 * (3 + kEpi);
static_assert(kEpi * STG_WARP_BYTES <= STG_BYTES && kEpi / 2 * STG_PAIR_FC1 <= STG_BYTES, "the epilogue's staging");

template <int MODE, bool SUMS = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    grouped_mm_kernel(const __grid_constant__ Params p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_addr(smem);
    unsigned char *staging = smem + RING_BYTES;
    unsigned char *state = staging + STG_BYTES;
    const uint32_t st0 = smem_addr(state);
    const uint32_t full0 = st0 + OFF_FULL, empty0 = st0 + OFF_EMPTY;
    const uint32_t acc_full0 = st0 + OFF_ACC_FULL, acc_empty0 = st0 + OFF_ACC_EMPTY;
    const uint32_t mma_done = st0 + OFF_MMA_DONE;
    const uint32_t tile_full0 = st0 + OFF_TILE_FULL, tile_empty0 = st0 + OFF_TILE_EMPTY;
    const uint32_t clc_bar = st0 + OFF_CLC_BAR, clc_resp = st0 + OFF_CLC_RESP;
    const uint32_t tile0 = st0 + OFF_TILE;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(state + OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(state + OFF_ABORT);
    int *starts = reinterpret_cast<int *>(state + STATE_BYTES);
    int *base = starts + kMaxGroups + 2;

    constexpr bool kAMn = MODE == kDgrad || MODE == kWgrad;
    constexpr bool kBMn = MODE == kWgrad;
    // readers of a tile: the MMA thread and, of both CTAs, the producer and the
    // epilogue warps
    constexpr int kReaders = 1 + 2 * (1 + kEpi);

    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tile_empty_leader0 = map_to_rank(tile_empty0, 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full0 + 8 * a, 1);
            mbar_init(acc_empty0 + 8 * a, 2 * kEpi);
        }
        mbar_init(mma_done, 1);
        for (int i = 0; i < kTileSlots; ++i) {
            mbar_init(tile_full0 + 8 * i, 1);
            mbar_init(tile_empty0 + 8 * i, kReaders);
        }
        mbar_init(clc_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.a)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    // from here on global memory is read: the previous grid must have completed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 2) build_groups<MODE, kTileF<MODE>, TILE_N>(p, starts, base);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Groups groups = {starts, base};
    const int tiles = base[p.groups + 1];

    // A wait of this thread ran out: both CTAs stop.  (The epilogue's warps set their own
    // CTA's flag alone: its producer stops then, and the leader's MMA thread, left without
    // operands, tells both.  Two instructions more in their loop cost 1 - 2 % of a call
    // that writes mostly zeros.)
    const auto give_up = [&]() {
        *abort_flag = 1;
        store_cluster(map_to_rank(st0 + OFF_ABORT, rank ^ 1u), 1);
    };

    // contraction blocks of a tile
    const auto blocks_of = [&](const Tile &t) {
        if (MODE == kWgrad) return (t.rows + BK - 1) / BK;
        return t.group == p.groups ? 0 : (p.depth + BK - 1) / BK;
    };
    // columns of the instruction
    const auto width_of = [&](const Tile &t) { return MODE == kWgrad ? TILE_N : (t.cnt + 31) / 32 * 32; };
    // contraction blocks per accumulation
    constexpr int kSegBlocks = SUMS ? kSegmentRows / BK : INT_MAX;

    // tile k of this pair, for a single thread; group -1 when none is left
    const auto next_tile = [&](int k) {
        const int slot = k % kTileSlots;
        Tile t;
        t.group = -1;
        if (mbar_wait<true>(tile_full0 + 8 * slot, (k / kTileSlots) & 1))
            t = read_tile(tile0 + 32 * slot);
        else
            give_up();
        mbar_arrive_cluster_read(tile_empty_leader0 + 8 * slot);
        return t;
    };
    // the same for a whole warp
    const auto next_tile_warp = [&](int k) {
        const int slot = k % kTileSlots;
        const bool ok =
            __all_sync(0xffffffffu, mbar_wait<true>(tile_full0 + 8 * slot, (k / kTileSlots) & 1));
        Tile t = read_tile(tile0 + 32 * slot);
        if (!ok) t.group = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_read(tile_empty_leader0 + 8 * slot);
        return t;
    };

    if (warp == kScheduler) {
        // ---- scheduler (the leader's): finds each tile's group and publishes it to
        // both CTAs while the one before is worked on.  The next tile is that of a
        // cluster whose launch it cancels, asked for once there is room for it: pairs
        // that ran ahead of their loads would take the last tiles from the others.
        if (leader && elect_one()) {
            int tile = (int)(blockIdx.x >> 1), asks = 0;
            const auto next = [&]() {
                do {
                    mbar_arrive_expect_tx(clc_bar, 16);
                    clc_try_cancel(clc_resp, clc_bar);
                    if (!mbar_wait<true>(clc_bar, asks++ & 1)) {
                        give_up();
                        return -1;
                    }
                    const int x = clc_cancelled_cta(clc_resp);
                    if (x < 0) return -1;  // no pending cluster was left
                    if ((x & 1) != 0 || x >= (int)gridDim.x) {  // not a cluster's first CTA of this grid
                        give_up();
                        atomicExch(&g_timeout, 1);
                        return -1;
                    }
                    tile = x >> 1;
                } while (tile >= tiles);  // beyond the last tile
                return tile;
            };
            for (int k = 0;; ++k) {
                const int slot = k % kTileSlots;
                if (!mbar_wait<true>(tile_empty0 + 8 * slot, ((k / kTileSlots) & 1) ^ 1)) give_up();
                Tile t;
                t.group = -1;
                if (k > 0 || tile >= tiles) tile = *abort_flag ? -1 : next();
                while (tile >= 0 && !*abort_flag) {
                    t = tile_at<MODE, kTileF<MODE>, TILE_N, 32>(p, groups, tile);
                    // a group without rows whose dW is added to: dW stays as it is (adding
                    // zeros would turn -0 into 0 and rewrite NaNs)
                    if (!(MODE == kWgrad && p.accumulate && t.rows == 0)) break;
                    t.group = -1;
                    tile = next();
                }
                publish(tile0 + 32 * slot, tile_full0 + 8 * slot, t);
                if (t.group < 0) break;
            }
        }
    } else if (warp == 0 && elect_one()) {
        // ---- producer (both CTAs).  (With the thread picked by `lane == 0` each load
        // cost ~400 cycles to issue: 8192 x 4096 x 8192 ran at 1390 TFLOP/s with
        // three loads a stage and 740 with four, against 1875 and 814.)
        int it = 0;
        for (int k = 0;; ++k) {
            const Tile t = next_tile(k);
            if (t.group < 0) break;
            const int kblocks = blocks_of(t);
            const int half = width_of(t) / 2;  // this CTA's rows of the N side
            const uint32_t bytes = (uint32_t)(A_BYTES + half * BK * 2);
            for (int kb = 0; kb < kblocks && !*abort_flag; ++kb, ++it) {
                const int s = it % STAGES;
                if (!mbar_wait(empty0 + 8 * s, ((it / STAGES) & 1) ^ 1)) {
                    give_up();
                    break;
                }
                const uint32_t sa = ring + s * STAGE_BYTES, sb = sa + A_BYTES;
                const uint32_t bar = map_to_rank(full0 + 8 * s, 0);
                if constexpr (MODE == kWgrad) {
                    const int live = t.rows - kb * BK;
                    if (live < BK) {  // the group's last rows
                        const int padded = (live + UMMA_K - 1) / UMMA_K * UMMA_K;
                        if (leader) mbar_arrive_expect_tx(full0 + 8 * s, 2 * 4 * 128 * padded);
                        int at = 0;
                        const auto rows = [&](int h, int row) {  // 1 << h rows
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t to = sa + i * (A_BYTES / 2) + 128 * at;
                                tma_load_2d_pair(to, &p.part_a[h], bar, t.m0 + 128 * (int)rank + 64 * i, row);
                                tma_load_2d_pair(to + A_BYTES, &p.part_b[h], bar, t.n0 + 128 * (int)rank + 64 * i,
                                                 row);
                            }
                            at += 1 << h;
                        };
#pragma unroll 1
                        for (int h = 5; h >= 0; --h)
                            if (live & (1 << h)) rows(h, t.r0 + kb * BK + at);
#pragma unroll 1
                        for (int h = 0; at < padded; ++h)  // beyond the tensor: zeros
                            if (at & (1 << h)) rows(h, p.rows);
                        continue;
                    }
                }
                if (leader) mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
                if (MODE == kFc1) {
                    // 32 gate rows and the 32 up rows of the same features, twice
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tma_load_3d_pair(sa + i * (A_BYTES / 2), &p.a, bar, kb * BK,
                                         t.m0 + 64 * (int)rank + 32 * i, 2 * t.group);
                } else if (MODE == kMm) {
                    tma_load_3d_pair(sa, &p.a, bar, kb * BK, t.m0 + 128 * (int)rank, t.group);
                } else if (MODE == kDgrad) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tma_load_3d_pair(sa + i * (A_BYTES / 2), &p.a, bar, t.m0 + 128 * (int)rank + 64 * i, kb * BK,
                                         t.group);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tma_load_2d_pair(sa + i * (A_BYTES / 2), &p.a, bar, t.m0 + 128 * (int)rank + 64 * i,
                                         t.r0 + kb * BK);
                }
                if (MODE == kWgrad) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tma_load_2d_pair(sb + i * (A_BYTES / 2), &p.b[0], bar, t.n0 + 128 * (int)rank + 64 * i,
                                         t.r0 + kb * BK);
                } else {
                    tma_load_2d_pair(sb, &p.b[half / 16 - 1], bar, kb * BK, t.r0 + t.n0 + half * (int)rank);
                }
            }
        }
        // the leader's full barriers count both CTAs' bytes: once their last
        // phases complete, every load of the pair has landed
        if (leader)
            for (int k = it > STAGES ? it - STAGES : 0; k < it; ++k)
                if (!mbar_wait(full0 + 8 * (k % STAGES), (k / STAGES) & 1)) give_up();
    } else if (warp == 1 && leader && elect_one()) {
        // ---- MMA issuer (leader only)
        int it = 0, lt = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Tile t = next_tile(k);
            if (t.group < 0 || *abort_flag) break;
            const int kblocks = blocks_of(t);
            const uint32_t idesc = instr_desc(kAMn, kBMn, 256, width_of(t));
            const int deep = MODE == kWgrad ? t.rows : p.depth;
            int kb = 0;
            do {  // one accumulation
                const int acc = lt & 1;
                if (!mbar_wait(acc_empty0 + 8 * acc, ((lt >> 1) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * TILE_N);
                const int first = kb, last = kblocks - kb > kSegBlocks ? kb + kSegBlocks : kblocks;
                for (; kb < last; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(full0 + 8 * s, (it / STAGES) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = ring + s * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk) {
                        if (kb * BK + kk * UMMA_K >= deep) break;
                        // K-major: 16 elements along the swizzled row; MN-major: 16
                        // rows of 128 bytes, 64-element groups A_BYTES / 2 apart
                        const uint64_t a = kAMn ? smem_desc_128b(sa + kk * UMMA_K * 128, A_BYTES / 2)
                                                : smem_desc_128b(sa + kk * UMMA_K * 2);
                        const uint64_t b = kBMn ? smem_desc_128b(sb + kk * UMMA_K * 128, A_BYTES / 2)
                                                : smem_desc_128b(sb + kk * UMMA_K * 2);
                        mma_bf16_pair(d, a, b, idesc, (kb != first || kk != 0) ? 1u : 0u);
                    }
                    mma_commit_both(empty0 + 8 * s);
                }
                if (!ok) break;
                mma_commit_both(acc_full0 + 8 * acc);
                ++lt;
            } while (kb < kblocks);
            if (!ok) give_up();
        }
        mma_commit_local_pair(mma_done);
        if (!mbar_wait(mma_done, 0)) give_up();
    } else if (warp >= 2 && warp < 2 + kEpi) {
        // ---- epilogue (both CTAs): this CTA's 128 lanes of the accumulator,
        // a quarter per warp
        const int quarter = warp & 3, set = (warp - 2) >> 2;
        constexpr int kChunk = MODE == kFc1 ? 16 : 32;  // columns of a warp at a time, and
        constexpr int kStep = kChunk * kEpi / 4;        // from one chunk to its next
        const uint32_t acc_empty_leader0 = map_to_rank(acc_empty0, 0);
        float *stg_pair = reinterpret_cast<float *>(staging + (2 * set + (quarter >> 1)) * STG_PAIR_FC1);
        unsigned char *to = staging + (4 * set + quarter) * STG_WARP_BYTES;
        // the buffer, once the bulk store that read it last is done with it
        const auto free_buffer = [&]() {
            if (elect_one()) bulk_wait_read<0>();
            __syncwarp();
        };
        // kWgrad: 32 columns of a tile, from column c on.  A lane is a row of dW; stores
        // beyond its rows and columns are cut off by the tensor map.
        const auto put_weights = [&](const Tile &t, const uint32_t (&v)[kChunk], int c) {
            if constexpr (MODE == kWgrad) {
                const int row0 = t.m0 + 128 * (int)rank + 32 * quarter;
                const int swz = (lane >> 1) & 3;
                if (p.f32_out) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        free_buffer();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4 *>(to + lane * 64 + ((i ^ swz) << 4)) =
                                make_uint4(v[16 * h + 4 * i], v[16 * h + 4 * i + 1], v[16 * h + 4 * i + 2],
                                           v[16 * h + 4 * i + 3]);
                        fence_async_shared();
                        __syncwarp();
                        const bool in = row0 < p.features && t.n0 + c + 16 * h < p.cols;
                        if (elect_one()) {
                            if (in && p.accumulate)
                                tma_add_3d(&p.c, smem_addr(to), t.n0 + c + 16 * h, row0, t.group);
                            else if (in)
                                tma_store_3d(&p.c, smem_addr(to), t.n0 + c + 16 * h, row0, t.group);
                            bulk_commit();
                        }
                    }
                } else {
                    free_buffer();
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        swiglu::BF16::put2(w, i, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4 *>(to + lane * 64 + ((i ^ swz) << 4)) =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    fence_async_shared();
                    __syncwarp();
                    if (elect_one()) {
                        if (row0 < p.features && t.n0 + c < p.cols)
                            tma_store_3d(&p.c, smem_addr(to), t.n0 + c, row0, t.group);
                        bulk_commit();
                    }
                }
            }
        };
        const int bar_id = 1 + 2 * set + (quarter >> 1);
        int lt = 0;
        bool ok = true;
        // the warp leaves the loop as one: the tile id, the abort flag and the
        // waits' outcome are warp-uniform
        for (int k = 0; ok; ++k) {
            const Tile t = next_tile_warp(k);
            // the barriers below need both warps of a pair, so the two leave
            // together, whichever of them gave up on its wait
            if (MODE == kFc1 ? any_of_pair(bar_id, t.group < 0) : t.group < 0) break;
            const int kblocks = blocks_of(t);
            const int width = width_of(t);
            // after a wait that ran out the values are undefined, but the warps stay in
            // step and the accumulator is handed back
            const auto wait_full = [&]() {
                if (!__all_sync(0xffffffffu, mbar_wait(acc_full0 + 8 * (lt & 1), (lt >> 1) & 1))) {
                    if (lane == 0) *abort_flag = 1;
                    ok = MODE == kFc1;  // (a pair leaves at the next tile id)
                }
                tc_fence_after();
            };
            const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
            wait_full();
            if constexpr (SUMS) {
                if (kblocks > kSegBlocks) {  // this warp's columns of the segments, added up
                    constexpr int kChunks = TILE_N / kStep;
                    uint32_t total[kChunks][kChunk];
                    uint32_t from = lanes + (uint32_t)((lt & 1) * TILE_N + kChunk * set);
#pragma unroll
                    for (int j = 0; j < kChunks; ++j) tmem_load32(from + kStep * j, total[j]);
                    tmem_wait_ld();
#pragma unroll 1
                    for (int left = kblocks - kSegBlocks; left > 0 && ok; left -= kSegBlocks) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_read(acc_empty_leader0 + 8 * (lt & 1));
                        ++lt;
                        wait_full();
                        from = lanes + (uint32_t)((lt & 1) * TILE_N + kChunk * set);
#pragma unroll
                        for (int j = 0; j < 2 * kChunks; ++j) {  // (16 columns: 32 at a time spill)
                            uint32_t v[16];
                            tmem_load16(from + kStep * (j / 2) + 16 * (j % 2), v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                uint32_t &sum = total[j / 2][16 * (j % 2) + i];
                                sum = __float_as_uint(__fadd_rn(__uint_as_float(sum), __uint_as_float(v[i])));
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_read(acc_empty_leader0 + 8 * (lt & 1));
                    ++lt;
                    // (with the accumulator kept until it is written: 6 % slower over 2048 rows)
#pragma unroll
                    for (int j = 0; j < kChunks; ++j) put_weights(t, total[j], kChunk * set + kStep * j);
                    continue;
                }
            }
            const int acc = lt & 1;
            ++lt;
            const uint32_t tbase = lanes + (uint32_t)(acc * TILE_N);
            if (kChunk * set >= width) {  // no columns for this warp
                if (lane == 0) mbar_arrive_cluster_read(acc_empty_leader0 + 8 * acc);
                continue;
            }
#pragma unroll 1
            for (int c = kChunk * set; c < width; c += kStep) {
                uint32_t v[kChunk];
                if constexpr (MODE == kMm || MODE == kDgrad) {
                    tmem_load_16x32(tbase + c, v);  // lanes 0 - 15 and 16 - 31 of the quarter
                    tmem_load_16x32(tbase + (16u << 16) + c, v + 16);
                } else if constexpr (MODE == kFc1) {
                    tmem_load16(tbase + c, v);
                } else {
                    tmem_load32(tbase + c, v);
                }
                tmem_wait_ld();
                if (c + kStep >= width) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_read(acc_empty_leader0 + 8 * acc);
                }
                if (kblocks == 0) {  // nothing was accumulated
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[i] = 0u;
                }
                if constexpr (MODE == kFc1) {
                    const auto pair_sync = [&]() {
                        asm volatile("bar.sync %0, 64;" ::"r"(bar_id) : "memory");
                    };
                    pair_sync();  // the previous chunk has been read
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        stg_pair[i * STG_ROW_FC1 + 32 * (quarter & 1) + lane] = __uint_as_float(v[i]);
                    pair_sync();
                    // four lanes per row, 8 features each
                    const int tk = 8 * (quarter & 1) + (lane >> 2), part = lane & 3;
                    const float *src = stg_pair + tk * STG_ROW_FC1 + 8 * part;
                    float g[8], u[8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 a = lds128(src + 4 * i), b = lds128(src + 32 + 4 * i);
                        g[4 * i] = a.x, g[4 * i + 1] = a.y, g[4 * i + 2] = a.z, g[4 * i + 3] = a.w;
                        u[4 * i] = b.x, u[4 * i + 1] = b.y, u[4 * i + 2] = b.z, u[4 * i + 3] = b.w;
                    }
                    const int n = p.features;
                    const int col = t.m0 + 64 * (int)rank + 32 * (quarter >> 1) + 8 * part;
                    const bool in = c + tk < t.cnt && col < n;  // (n is a multiple of 8)
                    const int64_t row = (int64_t)t.r0 + t.n0 + c + tk;
                    if (p.q != nullptr) {
                        // the row's four lanes hold its 32-column block
                        float mg = ckpt8::finite_amax<8>(g), mu = ckpt8::finite_amax<8>(u);
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) {
                            mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
                            mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
                        }
                        const uint32_t cg = ckpt8::scale_code(mg), cu = ckpt8::scale_code(mu);
                        if (in) {
                            using St8 = swiglu::St<8, swiglu::kStStream>;
                            uint32_t q[2];
                            uint8_t *qr = p.q + row * 2 * n + col;
                            ckpt8::encode<8>(g, ckpt8::encode_factor(cg), q);
                            St8::run(qr, q);
                            ckpt8::encode<8>(u, ckpt8::encode_factor(cu), q);
                            St8::run(qr + n, q);
                            if (part == 0) {
                                const int nb = (n + ckpt8::kBlock - 1) / ckpt8::kBlock;
                                uint8_t *sr = p.scales + row * 2 * nb + col / ckpt8::kBlock;
                                sr[0] = (uint8_t)cg;
                                sr[nb] = (uint8_t)cu;
                            }
                        }
                    }
                    if (in) {
                        uint32_t o[4];
                        if (p.fc1 != nullptr) {
                            __nv_bfloat16 *fr = p.fc1 + row * 2 * n + col;
                            swiglu::store_pack<swiglu::BF16, 8>(o, g);
                            store16(fr, o[0], o[1], o[2], o[3]);
                            swiglu::store_pack<swiglu::BF16, 8>(o, u);
                            store16(fr + n, o[0], o[1], o[2], o[3]);
                        }
                        const float w = p.probs != nullptr && t.group != p.groups ? p.probs[row] : 1.0f;
                        activate(g, u, w, o);
                        store16(static_cast<__nv_bfloat16 *>(p.out) + row * n + col, o[0], o[1], o[2], o[3]);
                    }
                } else if constexpr (MODE == kWgrad) {
                    put_weights(t, v, c);
                } else {
                    // transposed on the way to shared memory: row r of the buffer
                    // is row c + r of the tile, its 16-byte pieces 8 features each
                    free_buffer();
                    const uint32_t at = smem_addr(to) + (lane & 7) * 64 +
                                        (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // 8 rows each
                        uint32_t w[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {  // features 8 m ..
                            const int r = 16 * (m >> 1) + 4 * j + 2 * (m & 1);
                            uint32_t two[1];
                            swiglu::BF16::put2(two, 0, __uint_as_float(v[r]), __uint_as_float(v[r + 1]));
                            w[m] = two[0];
                        }
                        stmatrix_x4_trans(at + j * 8 * 64, w[0], w[1], w[2], w[3]);
                    }
                    const int col = t.m0 + 128 * (int)rank + 32 * quarter;
                    const int row = t.r0 + t.n0 + c;
                    const int live = t.cnt - c;
                    if (live >= 32) {
                        fence_async_shared();
                        __syncwarp();
                        if (elect_one()) {
                            if (col < p.features) tma_store_2d(&p.c, smem_addr(to), col, row);
                            bulk_commit();
                        }
                    } else {  // the rows after these are another group's
                        __syncwarp();
                        const int f = col + 8 * (lane & 3);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + (lane >> 2);
                            const uint4 w = *reinterpret_cast<const uint4 *>(
                                to + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
                            if (r < live && f < p.features)
                                store16(static_cast<__nv_bfloat16 *>(p.out) + (int64_t)(row + r) * p.features + f,
                                        w.x, w.y, w.z, w.w);
                        }
                    }
                }
            }
        }
        if (elect_one()) bulk_wait<0>();  // the stores, before their shared memory goes
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal it
    if (threadIdx.x == 0 && *abort_flag) settle();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// ------------------------------------------------- few tiles: split the depth ---
// When a call has fewer tiles than the GPU has pairs of SMs (a few rows, or a
// narrow product over many), its time is that of one tile's loads.  Then a
// cluster of S CTAs (1, 2, 4 or 8), each on its own (cta_group::1), takes a tile
// of 128 accumulator lanes by at most NT rows and each CTA a slice of the
// contraction.  The partial sums meet in shared memory: every CTA leaves its own
// as [row][lane] fp32 over its (by then idle) ring, and CTA r adds up all S of
// every S-th row, in rank order, and stores them.  The order is fixed, and
// nothing passes through global memory.  One tile per cluster, no tile
// scheduling; shared memory is held to half an SM, so that the next launch's
// CTAs can set up beside this one's last.
constexpr int kSplitThreads = 192;
template <int NT>
constexpr int kSplitStageBytes = A_BYTES + NT * BK * 2;
template <int NT>
constexpr int kSplitStages = NT == 32 ? 5 : 3;
constexpr int kPartialRow = 132;  // fp32 lanes of a row of partial sums, padded
template <int NT>
constexpr int kSplitRing = kSplitStages<NT> * kSplitStageBytes<NT>;
static_assert(kSplitRing<32> >= 32 * kPartialRow * 4 && kSplitRing<128> >= 128 * kPartialRow * 4,
              "the partial sums fit the ring");
template <int NT>
constexpr int kSplitSmem = kSplitRing<NT> + STATE_BYTES + (TABLE_BYTES + 15) / 16 * 16 + 1024;
static_assert(kSplitSmem<32> <= 113 * 1024 && kSplitSmem<128> <= 113 * 1024, "two CTAs per SM");

// Features of a tile (kFc1: a gate and an up lane for each).
template <int MODE>
constexpr int kSplitF = MODE == kFc1 ? 64 : 128;

// Partial sums, which other threads and CTAs have written: neither load may be moved
// over the barrier before it.
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_own(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// First block of slice s of `blocks` blocks cut into `size` (a power of two) slices.
__device__ __forceinline__ int slice_begin(int blocks, uint32_t s, uint32_t size) {
    return (int)(((uint64_t)(uint32_t)blocks * s) >> (31 - __clz((int)size)));
}

// Rows rank, rank + S, ... of a tile: their slices' sums added up in rank order and
// stored.  A thread takes four features of every kPass-th of these rows, R rows at a
// time, everything they need loaded before the first is used (a load from another
// SM, a row's weight or dW's old value takes long, and a CTA has six warps).  `ring`:
// this CTA's partial sums; bit s of `have`: slice s has a part.
template <int MODE, int R, int SL>
__device__ __forceinline__ void join_rows(const Params &p, const Tile &t, uint32_t ring, int rank, int size,
                                          uint32_t have) {
    using St8 = swiglu::St<8, swiglu::kStStream>;
    constexpr int kRowThreads = kSplitF<MODE> / 4;
    constexpr int kPass = kSplitThreads / kRowThreads;  // rows of the CTA per pass
    static_assert(kSplitThreads % kRowThreads == 0, "whole rows of threads");
    const int f = (int)threadIdx.x % kRowThreads, col = t.m0 + 4 * f, n = p.features;
    const int step = kPass * size, first = rank + (int)threadIdx.x / kRowThreads * size;
    // this thread's rows, and the turns of all (the same for a whole warp: the block
    // maximum is shuffled)
    int left = col < n && first < t.cnt ? (t.cnt - first + step - 1) / step : 0;
    const int turns = rank < t.cnt ? (t.cnt - rank + step * R - 1) / (step * R) : 0;
    // kFc1: 32 gates, 32 ups, 32 gates, 32 ups
    uint32_t from = ring + (uint32_t)(first * kPartialRow + (MODE == kFc1 ? f / 8 * 64 + f % 8 * 4 : f * 4)) * 4;
    int64_t row = (int64_t)t.r0 + t.n0 + first;
    // the M side of kWgrad are dW's columns, the N side its rows
    const int eb = MODE == kWgrad && p.f32_out ? 4 : 2;
    char *out = static_cast<char *>(p.out) +
                ((MODE == kWgrad ? (int64_t)t.group * p.cols + t.n0 + first : row) * n + col) * eb;
    const int64_t out_step = (int64_t)step * n * eb;
    const auto pack = [](const float (&v)[4], uint32_t (&w)[2]) {
        swiglu::BF16::put2(w, 0, v[0], v[1]);
        swiglu::BF16::put2(w, 2, v[2], v[3]);
    };
#pragma unroll 1
    for (int turn = 0; turn < turns; ++turn) {
        float4 a[R][SL], b[R][SL], old[R];
        float wr[R];
#pragma unroll
        for (int s = 0; s < SL; ++s) {
            if (!(have >> s & 1)) continue;
            const uint32_t at = SL == 1 ? from : map_to_rank(from, (uint32_t)s);
            const auto load = [&](uint32_t offset) { return SL == 1 ? ld_own(at + offset) : ld_cluster(at + offset); };
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i < left) {
                    a[i][s] = load((uint32_t)(i * step * kPartialRow) * 4);
                    if (MODE == kFc1) b[i][s] = load((uint32_t)(i * step * kPartialRow + 32) * 4);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            wr[i] = 1.0f;
            if (MODE == kFc1 && i < left && p.probs != nullptr && t.group != p.groups) wr[i] = p.probs[row + i * step];
            if (MODE == kWgrad && i < left && p.accumulate)
                old[i] = *reinterpret_cast<const float4 *>(out + i * out_step);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool in = i < left;
            float g[4] = {}, u[4] = {};
#pragma unroll
            for (int s = 0; s < SL; ++s) {
                if (in && (have >> s & 1)) {
                    g[0] = __fadd_rn(g[0], a[i][s].x), g[1] = __fadd_rn(g[1], a[i][s].y);
                    g[2] = __fadd_rn(g[2], a[i][s].z), g[3] = __fadd_rn(g[3], a[i][s].w);
                    if (MODE == kFc1) {
                        u[0] = __fadd_rn(u[0], b[i][s].x), u[1] = __fadd_rn(u[1], b[i][s].y);
                        u[2] = __fadd_rn(u[2], b[i][s].z), u[3] = __fadd_rn(u[3], b[i][s].w);
                    }
                }
            }
            uint32_t w[2];
            if constexpr (MODE == kFc1) {
                if (p.q != nullptr) {
                    float mg = ckpt8::finite_amax<4>(g), mu = ckpt8::finite_amax<4>(u);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) {  // eight threads hold a block
                        mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
                        mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
                    }
                    if (in) {
                        const uint32_t cg = ckpt8::scale_code(mg), cu = ckpt8::scale_code(mu);
                        uint32_t qg, qu;
                        ckpt8::encode<4>(g, ckpt8::encode_factor(cg), &qg);
                        ckpt8::encode<4>(u, ckpt8::encode_factor(cu), &qu);
                        uint8_t *qr = p.q + row * 2 * n + col;
                        swiglu::St<4, swiglu::kStStream>::run(qr, &qg);
                        swiglu::St<4, swiglu::kStStream>::run(qr + n, &qu);
                        if (f % 8 == 0) {
                            const int nb = (n + ckpt8::kBlock - 1) / ckpt8::kBlock;
                            uint8_t *sr = p.scales + row * 2 * nb + col / ckpt8::kBlock;
                            sr[0] = (uint8_t)cg;
                            sr[nb] = (uint8_t)cu;
                        }
                    }
                }
                if (in) {
                    if (p.fc1 != nullptr) {
                        __nv_bfloat16 *fr = p.fc1 + row * 2 * n + col;
                        pack(g, w);
                        St8::run(fr, w);
                        pack(u, w);
                        St8::run(fr + n, w);
                    }
                    activate(g, u, wr[i], w);
                    St8::run(out, w);
                }
            } else if (in) {
                if (MODE == kWgrad && p.f32_out) {
                    if (p.accumulate) {
                        g[0] = __fadd_rn(old[i].x, g[0]), g[1] = __fadd_rn(old[i].y, g[1]);
                        g[2] = __fadd_rn(old[i].z, g[2]), g[3] = __fadd_rn(old[i].w, g[3]);
                    }
                    store16(out, __float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]),
                            __float_as_uint(g[3]));
                } else {
                    pack(g, w);
                    St8::run(out, w);
                }
            }
            row += step;
            out += out_step;
        }
        left -= R;
        from += (uint32_t)(R * step * kPartialRow) * 4;
    }
}

template <int MODE, int NT, bool SUMS = false>
__global__ void __launch_bounds__(kSplitThreads, 2) grouped_mm_split_kernel(const __grid_constant__ Params p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_addr(smem);
    unsigned char *state = smem + kSplitRing<NT>;
    const uint32_t st0 = smem_addr(state);
    constexpr int kStages = kSplitStages<NT>;
    constexpr int kStage = kSplitStageBytes<NT>;
    const uint32_t full0 = st0, empty0 = st0 + 8 * kStages, acc_full = st0 + 16 * kStages;
    const uint32_t landed = acc_full + 8, zeroed = acc_full + 16;  // of a group's last block (kWgrad)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(state + 16 * kStages + 24);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(state + 16 * kStages + 28);
    // SUMS: two accumulators in turn
    constexpr int kSegBlocks = SUMS ? kSegmentRows / BK : INT_MAX;
    constexpr int kTmem = SUMS ? 2 * NT : NT;
    const auto full_of = [&](int a) { return SUMS && a != 0 ? acc_full + 32 : acc_full; };
    const auto empty_of = [&](int a) { return acc_full + 40 + 8 * a; };
    static_assert(16 * kStages + 56 <= STATE_BYTES, "barriers and state fit their region");
    int *starts = reinterpret_cast<int *>(state + STATE_BYTES);
    int *base = starts + kMaxGroups + 2;
    constexpr bool kAMn = MODE == kDgrad || MODE == kWgrad, kBMn = MODE == kWgrad;
    static_assert(MODE != kWgrad || NT == 128, "the weight gradient's N side comes in boxes of 64 columns");

    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(landed, 1);
        mbar_init(zeroed, 1);
        if (SUMS) {
            mbar_init(full_of(1), 1);
            mbar_init(empty_of(0), 4);
            mbar_init(empty_of(1), 4);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.b[0])) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 2) build_groups<MODE, kSplitF<MODE>, NT>(p, starts, base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Groups groups = {starts, base};
    const int tile = (int)(blockIdx.x >> (31 - __clz((int)size)));
    const bool live = tile < base[p.groups + 1];  // the same in the whole cluster
    Tile t = {};
    int kb0 = 0, kb1 = 0;
    if (live) {
        t = tile_at<MODE, kSplitF<MODE>, NT, 16>(p, groups, tile);
        if (t.group != p.groups) {
            const int kblocks = ((MODE == kWgrad ? t.rows : p.depth) + BK - 1) / BK;
            kb0 = slice_begin(kblocks, rank, size);
            kb1 = slice_begin(kblocks, rank + 1, size);
        }
    }
    const int width = (t.cnt + 15) / 16 * 16;
    // kWgrad: the rows of the group's last block, where it is this CTA's and not full
    const int last_rows = MODE == kWgrad && kb1 > kb0 && kb1 * BK > t.rows ? t.rows % BK : 0;
    if (warp == 0 && elect_one()) {
        const int box_cols = (width + 63) / 64;  // kWgrad
        const uint32_t bytes =
            (uint32_t)(A_BYTES + (MODE == kWgrad ? box_cols * (A_BYTES / 2) : width * BK * 2));
        int it = 0;
        for (int kb = kb0; kb < kb1 && !*abort_flag; ++kb, ++it) {
            const int s = it % kStages;
            if (!mbar_wait(empty0 + 8 * s, ((it / kStages) & 1) ^ 1)) {
                *abort_flag = 1;
                break;
            }
            const uint32_t sa = ring + s * kStage;
            const uint32_t bar = last_rows != 0 && kb == kb1 - 1 ? landed : full0 + 8 * s;
            mbar_arrive_expect_tx(bar, bytes);
            if (MODE == kFc1) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tma_load_3d(sa + i * (A_BYTES / 2), &p.a, bar, kb * BK, t.m0 + 32 * i, 2 * t.group);
            } else if (MODE == kMm) {
                tma_load_3d(sa, &p.a, bar, kb * BK, t.m0, t.group);
            } else if (MODE == kDgrad) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tma_load_3d(sa + i * (A_BYTES / 2), &p.a, bar, t.m0 + 64 * i, kb * BK, t.group);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tma_load_2d(sa + i * (A_BYTES / 2), &p.a, bar, t.m0 + 64 * i, t.r0 + kb * BK);
                for (int i = 0; i < box_cols; ++i)
                    tma_load_2d(sa + A_BYTES + i * (A_BYTES / 2), &p.b[0], bar, t.n0 + 64 * i, t.r0 + kb * BK);
                continue;
            }
            tma_load_2d(sa + A_BYTES, &p.b[width / 16 - 1], bar, kb * BK, t.r0 + t.n0);
        }
        // every load has landed before this CTA can leave, also when a wait ran out
        for (int k = it > kStages ? it - kStages : 0; k < it; ++k) {
            if (last_rows != 0 && k == kb1 - 1 - kb0)
                mbar_wait(landed, 0);
            else
                mbar_wait(full0 + 8 * (k % kStages), (k / kStages) & 1);
        }
    } else if (warp == 1 && kb1 > kb0 && elect_one()) {
        const uint32_t idesc = instr_desc(kAMn, kBMn, 128, width);
        int seg = 0;
        for (int kb = kb0, it = 0; kb < kb1; ++kb, ++it) {
            const int s = it % kStages;
            if (SUMS && it != 0 && it % kSegBlocks == 0) {
                mma_commit(full_of(seg & 1));
                ++seg;
                if (!mbar_wait(empty_of(seg & 1), ((seg >> 1) & 1) ^ 1)) {
                    *abort_flag = 1;
                    break;
                }
            }
            if (!(last_rows != 0 && kb == kb1 - 1 ? mbar_wait(zeroed, 0)
                                                  : mbar_wait(full0 + 8 * s, (it / kStages) & 1))) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const uint32_t sa = ring + s * kStage, sb = sa + A_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / UMMA_K; ++kk) {
                const uint64_t a = kAMn ? smem_desc_128b(sa + kk * UMMA_K * 128, A_BYTES / 2)
                                        : smem_desc_128b(sa + kk * UMMA_K * 2);
                const uint64_t b = kBMn ? smem_desc_128b(sb + kk * UMMA_K * 128, A_BYTES / 2)
                                        : smem_desc_128b(sb + kk * UMMA_K * 2);
                const bool first = (SUMS ? it % kSegBlocks == 0 : kb == kb0) && kk == 0;
                mma_bf16(SUMS ? tmem + (uint32_t)((seg & 1) * NT) : tmem, a, b, idesc, first ? 0u : 1u);
            }
            mma_commit(empty0 + 8 * s);
        }
        mma_commit(full_of(seg & 1));
    } else if (warp >= 2 && kb1 > kb0) {
        // this CTA's partial sums, from tensor memory to [row][lane]; every load
        // of the ring has been consumed by then
        const int quarter = warp & 3;
        float *part = reinterpret_cast<float *>(smem);
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        const auto zero_next = [&]() {  // the next group's rows in the last block
            if (MODE == kWgrad && last_rows != 0 && warp == 2) {
                if (!__all_sync(0xffffffffu, mbar_wait(landed, 0)) && lane == 0) *abort_flag = 1;
                unsigned char *stage = smem + (kb1 - 1 - kb0) % kStages * kStage;
                for (int i = lane; i < (BK - last_rows) * 8; i += 32) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        *reinterpret_cast<uint4 *>(stage + b * (A_BYTES / 2) + last_rows * 128 + i * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(zeroed);
            }
        };
        if constexpr (SUMS) {
            constexpr int kChunk = 16;
            float total[NT / kChunk][kChunk] = {};
            const int segs = (kb1 - kb0 + kSegBlocks - 1) / kSegBlocks;
#pragma unroll 1
            for (int seg = 0; seg < segs; ++seg) {
                // (not sooner: the last block's loads wait for the segments before)
                if (seg + 1 == segs) zero_next();
                if (!__all_sync(0xffffffffu, mbar_wait(full_of(seg & 1), (seg >> 1) & 1))) {
                    if (lane == 0) *abort_flag = 1;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < NT / kChunk; ++j) {
                    if (kChunk * j < width) {
                        uint32_t v[kChunk];
                        tmem_load16(lanes + (uint32_t)((seg & 1) * NT + kChunk * j), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < kChunk; ++i)
                            total[j][i] = __fadd_rn(total[j][i], __uint_as_float(v[i]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_of(seg & 1));
            }
#pragma unroll
            for (int j = 0; j < NT / kChunk; ++j) {
                if (kChunk * j < width) {  // (width is a multiple of 16)
#pragma unroll
                    for (int i = 0; i < kChunk; ++i)
                        part[(kChunk * j + i) * kPartialRow + 32 * quarter + lane] = total[j][i];
                }
            }
        } else {
            zero_next();
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full, 0)) && lane == 0) *abort_flag = 1;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < width; c += 32) {
                uint32_t v[32];
                tmem_load32(lanes + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c + i < width) part[(c + i) * kPartialRow + 32 * quarter + lane] = __uint_as_float(v[i]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (size > 1) cluster_sync();
    if (live) {
        uint32_t have = 0;  // slices with a block (a short group of kWgrad leaves some without)
        if (t.group != p.groups) {
            const int blocks = ((MODE == kWgrad ? t.rows : p.depth) + BK - 1) / BK;
            for (uint32_t s = 0; s < size; ++s)
                if (slice_begin(blocks, s, size) < slice_begin(blocks, s + 1, size)) have |= 1u << s;
        }
        // (more rows at once are slower: the code that is fetched for them costs more
        // than the latency that they hide, 6.7 against 6.3 us for 128 rows in 2 slices)
        if (MODE == kWgrad && p.accumulate && have == 0) {
            // nothing to add: dW stays as it is
        } else if (size == 1)
            join_rows<MODE, 4, 1>(p, t, ring, (int)rank, (int)size, have);
        else if (size == 2)
            join_rows<MODE, MODE == kFc1 ? 2 : 4, 2>(p, t, ring, (int)rank, (int)size, have);
        else if (size == 4)
            join_rows<MODE, MODE == kFc1 ? 1 : 2, 4>(p, t, ring, (int)rank, (int)size, have);
        else
            join_rows<MODE, 1, 8>(p, t, ring, (int)rank, (int)size, have);
    }
    __syncwarp();
    if (size > 1) cluster_sync_read();  // no CTA leaves while another may still read its sums
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

// ---------------------------------------------------------------- host side

namespace {

// A bf16 tensor of `rank` dimensions, innermost first, dense in every row, as
// boxes of 64 elements of the innermost dimension (128 bytes) with the matching
// swizzle; zero fill outside.  W is fetched into L2 256 bytes at a time, which a
// call of few rows, a stream over W, needs (32 rows, 8 experts [4096, 14336]:
// 141 us, 151 without); rows are not: where they are no multiple of 32 bytes it
// costs (16500 rows, 64 experts [2056, 1304]: 118 us, 112 without).
bool make_map(EncodeTiled enc, CUtensorMap *map, const void *p, int rank, const int64_t *dims, const int64_t *strides,
              const int *box, CUtensorMapL2promotion promotion) {
    cuuint64_t d[3], st[2];
    cuuint32_t bx[3], es[3];
    for (int i = 0; i < rank; ++i) {
        d[i] = (cuuint64_t)dims[i];
        bx[i] = (cuuint32_t)box[i];
        es[i] = 1;
    }
    for (int i = 0; i + 1 < rank; ++i) st[i] = (cuuint64_t)strides[i];
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(p), d, st, bx, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map2(EncodeTiled enc, CUtensorMap *map, const void *p, int64_t inner, int64_t rows, int box_rows) {
    const int64_t dims[2] = {inner, rows}, strides[1] = {inner * 2};
    const int box[2] = {BK, box_rows};
    return make_map(enc, map, p, 2, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// W as [outer][rows][inner] with boxes of box_rows x box_outer rows.
bool map3(EncodeTiled enc, CUtensorMap *map, const void *p, int64_t inner, int64_t rows, int64_t outer, int box_rows,
          int box_outer) {
    const int64_t dims[3] = {inner, rows, outer}, strides[2] = {inner * 2, inner * rows * 2};
    const int box[3] = {BK, box_rows, box_outer};
    return make_map(enc, map, p, 3, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// The result: boxes of 64 bytes by 32 rows with the 64-byte swizzle, one warp's
// part: 2.2 us per 256 x 256 tile of one contraction block, 4.5 TB/s.  (Rows of 128
// bytes, put together by two warps, cost more in the warps' meeting than the wider
// rows save, 4.0 - 4.3 against 3.7 us at the time; plain 32-byte stores from the
// accumulator's lanes took 5.4.  A second buffer per warp, and the two halves of a
// row's 128 bytes stored by one warp in turn, were no faster.)
bool out_map(EncodeTiled enc, CUtensorMap *map, void *p, int eb, int64_t inner, int64_t rows, int64_t outer) {
    const cuuint64_t d[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t st[2] = {(cuuint64_t)(inner * eb), (cuuint64_t)(inner * rows * eb)};
    const cuuint32_t box[3] = {(cuuint32_t)(64 / eb), 32, 1}, es[3] = {1, 1, 1};
    return enc(map, eb == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               outer > 0 ? 3 : 2, p, d, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The N side of the products over rows: boxes of 16, 32, 48, ... 128 rows, as far
// as a tile of `rows` rows (to 16) can need them; a CTA of a pair loads half of
// its tile (to 32), which is no more.  One box whatever the width: with boxes of
// powers of two, up to three loads, 10739 rows by [4096, 2048] took 1 % longer.
bool row_maps(EncodeTiled enc, CUtensorMap *maps, const void *p, int64_t inner, int64_t rows) {
    for (int i = 0; i < 8 && 16 * i < rows; ++i)
        if (!map2(enc, maps + i, p, inner, rows, 16 * (i + 1))) return false;
    return true;
}

constexpr int kSms = 152;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One cluster per tile, of which there are `clusters` at most.
template <int MODE, bool SUMS = false>
swiglu_status_t launch_pairs(const Params &p, int64_t clusters, swiglu_stream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    // the shared-memory opt-in is a per-device function attribute
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (!(dev >= 0 && dev < kMaxDevices && attr_set[dev].load())) {
        e = cudaFuncSetAttribute(grouped_mm_kernel<MODE, SUMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e != cudaSuccess) return moe::cuda_fail(e);
        if (dev >= 0 && dev < kMaxDevices) attr_set[dev].store(true);
    }
    e = moe::launch(grouped_mm_kernel<MODE, SUMS>, dim3((unsigned)(2 * clusters)), kPairThreads, SMEM_BYTES,
                    stream, 0, p);
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

// Tiles of a product over rows, at most.  g groups (those that can have a row,
// the rows of no group counted as one) of c_i rows have
// sum ceil(c_i / tn) <= (rows + (tn - 1) g) / tn row tiles.
int64_t most_tiles(int64_t rows, int64_t groups, int64_t features, int tile_f, int tn) {
    const int64_t g = rows < groups + 1 ? rows : groups + 1;
    return (rows + (tn - 1) * g) / tn * ((features + tile_f - 1) / tile_f);
}

template <int MODE, int NT, bool SUMS = false>
swiglu_status_t launch_split(const Params &p, int64_t tiles, int size, swiglu_stream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (!(dev >= 0 && dev < kMaxDevices && attr_set[dev].load())) {
        e = cudaFuncSetAttribute(grouped_mm_split_kernel<MODE, NT, SUMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSplitSmem<NT>);
        if (e != cudaSuccess) return moe::cuda_fail(e);
        if (dev >= 0 && dev < kMaxDevices) attr_set[dev].store(true);
    }
    e = moe::launch(grouped_mm_split_kernel<MODE, NT, SUMS>, dim3((unsigned)(tiles * size)), kSplitThreads,
                    kSplitSmem<NT>, stream, size, p);
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

// Pairs or split?  The rule estimates both times in nanoseconds from the tiles of
// groups of equal size, which is all the host knows: operand bytes per SM at the
// rates the two kernels reach, times the rounds of the grid, plus what a launch,
// a tile, the joining of the sums and the CTAs beyond the last tile take.  The
// constants are a fit to the times of all five choices on 14,500 shapes (forward,
// fc1 and both gradients; 1 to 32768 rows, 1 to 64 equal groups, widths 64 to 14336);
// with them the choice is on average 2.4 % slower than the best one, where always pairs
// are 22 % and always one CTA per tile 36 % slower.  (A weight gradient's pairs multiply
// 256 columns whatever N is; with that in place of N's own width the choice was no
// better, 2.5 % off the best against 2.3 % on 384 shapes with N below 256.)
struct Plan {
    int size;  // CTAs per tile of the split kernel; 0: pairs
};

// `same` groups of `rows_per` rows (kWgrad: dW's rows, N) by `features`; pair_f
// and split_f: features of a tile, nt: rows of a tile of the split kernel, most: its
// tiles at most.
Plan plan(int64_t same, int64_t rows_per, int64_t features, int pair_f, int split_f, int nt, int64_t most,
          int64_t kblocks) {
    const int64_t pair_n = rows_per < TILE_N ? ceil_div(rows_per, 32) * 32 : TILE_N;
    const int64_t pair_tiles = same * ceil_div(rows_per, TILE_N) * ceil_div(features, pair_f);
    const int64_t pair_depth = kblocks * (A_BYTES + pair_n * BK) * 100 / 8955;
    Plan best = {0};
    int64_t least = ceil_div(pair_tiles, kSms / 2) * (pair_depth > 1530 ? pair_depth : 1530) + 8270;
    const int64_t split_n = rows_per < nt ? ceil_div(rows_per, 16) * 16 : nt;
    const int64_t split_tiles = same * ceil_div(rows_per, nt) * ceil_div(features, split_f);
    const int64_t beyond = most > split_tiles ? most - split_tiles : 0;
    for (int size = 1; size <= 8 && (size == 1 || 2 * size <= kblocks); size *= 2) {
        const int64_t ctas = split_tiles * size;
        const int64_t bytes = ceil_div(kblocks, size) * (A_BYTES + split_n * BK * 2);
        const int64_t time = (ctas <= kSms ? bytes * 10 / 896 : ceil_div(ctas, kSms) * bytes * 10 / 1066) +
                             ceil_div(ctas, 2 * kSms) * 6810 + (size > 1 ? 870 : 0) + beyond * size * 17;
        if (time < least) {
            least = time;
            best.size = size;
        }
    }
    return best;
}

// Rows of a tile of the split kernel, and its tiles at most, for a product over rows.
int split_rows(int64_t rows) { return rows <= 32 ? 32 : 128; }

template <int MODE>
int64_t split_tiles(int64_t rows, int64_t groups, int64_t features) {
    return most_tiles(rows, groups, features, kSplitF<MODE>, split_rows(rows));
}

template <int MODE>
Plan plan_rows(int64_t rows, int64_t groups, int64_t features, int64_t depth) {
    const int64_t same = rows < groups ? rows : groups, tiles = split_tiles<MODE>(rows, groups, features);
    if (tiles > INT32_MAX / 16) return {0};
    return plan(same, ceil_div(rows, same), features, kTileF<MODE>, kSplitF<MODE>, split_rows(rows), tiles,
                ceil_div(depth, BK));
}

int64_t wgrad_split_tiles(int64_t groups, int64_t N, int64_t K) {
    return groups * ceil_div(N, 128) * ceil_div(K, kSplitF<kWgrad>);
}

Plan plan_wgrad(int64_t rows, int64_t groups, int64_t N, int64_t K) {
    return plan(groups, N, K, 256, kSplitF<kWgrad>, 128, wgrad_split_tiles(groups, N, K),
                ceil_div(ceil_div(rows, groups), BK));
}

// Launch a product over rows.
template <int MODE>
swiglu_status_t launch_rows(const Params &p, swiglu_stream_t stream) {
    const int64_t pairs = most_tiles(p.rows, p.groups, p.features, kTileF<MODE>, TILE_N);
    if (pairs > INT32_MAX / 4) return SWIGLU_ERR_SHAPE;
    const int size = plan_rows<MODE>(p.rows, p.groups, p.features, p.depth).size;
    if (size == 0) return launch_pairs<MODE>(p, pairs, stream);
    const int64_t tiles = split_tiles<MODE>(p.rows, p.groups, p.features);
    return split_rows(p.rows) == 32 ? launch_split<MODE, 32>(p, tiles, size, stream)
                                    : launch_split<MODE, 128>(p, tiles, size, stream);
}

// The checks that the products share.  A pair works off 64 rows of a weight gradient in
// 0.27 us, one segment after the other, while its tile's readers wait for the next tile:
// 1.1 s for SWIGLU_GROUPED_MAX_ROWS_WGRAD rows of one group.
static_assert(SWIGLU_GROUPED_MAX_ROWS == INT32_MAX - TILE_N && SWIGLU_GROUPED_MAX_FEATURES == INT32_MAX / 2,
              "rows rounded up to a tile, and twice the features, fit an int");
swiglu_status_t check(int64_t rows, int64_t groups, int64_t features, int64_t K, swiglu_dtype_t dtype) {
    if (dtype != SWIGLU_BF16) return SWIGLU_ERR_DTYPE;
    if (rows < 0 || rows > SWIGLU_GROUPED_MAX_ROWS || groups < 1 || groups > kMaxGroups) return SWIGLU_ERR_SHAPE;
    if (features < 8 || K < 8 || features % 8 != 0 || K % 8 != 0 || K > SWIGLU_GROUPED_MAX_FEATURES ||
        features > SWIGLU_GROUPED_MAX_FEATURES / groups)
        return SWIGLU_ERR_SHAPE;
    return SWIGLU_OK;
}

bool aligned(std::initializer_list<const void *> ps, uintptr_t by) {
    for (const void *p : ps)
        if ((uintptr_t)p % by != 0) return false;
    return true;
}

}  // namespace

}  // namespace gmm

using moe::Span;
using moe::span_of;

extern "C" {

swiglu_status_t swiglu_grouped_fc1_fwd(const void *x, const void *w, const int32_t *ends, const float *probs, void *y,
                                       void *fc1, void *q, void *scales, int64_t rows, int64_t groups, int64_t n,
                                       int64_t K, swiglu_dtype_t dtype, swiglu_stream_t stream) {
    using namespace gmm;
    swiglu_status_t st = check(rows, groups, n, K, dtype);
    if (st == SWIGLU_OK && 2 * n > SWIGLU_GROUPED_MAX_FEATURES / groups) st = SWIGLU_ERR_SHAPE;
    if (st != SWIGLU_OK || rows == 0) return st;
    if (x == nullptr || w == nullptr || ends == nullptr || y == nullptr || (q == nullptr) != (scales == nullptr))
        return SWIGLU_ERR_NULL;
    if (fc1 != nullptr && q != nullptr) return SWIGLU_ERR_ALIAS;  // one of the two is kept
    if (!aligned({x, w, y, fc1, q}, 16) || !aligned({ends, probs}, 4)) return SWIGLU_ERR_STRIDE;
    const int64_t nb = (n + SWIGLU_CKPT8_BLOCK - 1) / SWIGLU_CKPT8_BLOCK;
    Span sx, sw, se, sp, sy, sf, sq, ss;
    if (!span_of(x, rows, K, K, 2, sx) || !span_of(w, groups * 2 * n, K, K, 2, sw) ||
        !span_of(ends, groups, 1, 1, 4, se) || !span_of(probs, rows, 1, 1, 4, sp) || !span_of(y, rows, n, n, 2, sy) ||
        !span_of(fc1, rows, 2 * n, 2 * n, 2, sf) || !span_of(q, rows, 2 * n, 2 * n, 1, sq) ||
        !span_of(scales, rows, 2 * nb, 2 * nb, 1, ss))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sy, sf, sq, ss}, {sx, sw, se, sp})) return SWIGLU_ERR_ALIAS;

    EncodeTiled enc;
    const cudaError_t e = encoder(enc);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    Params p{};
    // [gate | up] halves of every expert: 32 rows of each per box
    if (!map3(enc, &p.a, w, K, n, 2 * groups, 32, 2) || !row_maps(enc, p.b, x, K, rows))
        return moe::cuda_fail(cudaErrorInvalidValue);
    p.ends = ends;
    p.probs = probs;
    p.out = y;
    p.fc1 = static_cast<__nv_bfloat16 *>(fc1);
    p.q = static_cast<uint8_t *>(q);
    p.scales = static_cast<uint8_t *>(scales);
    p.rows = (int)rows;
    p.groups = (int)groups;
    p.features = (int)n;
    p.depth = (int)K;
    return launch_rows<kFc1>(p, stream);
}

swiglu_status_t swiglu_grouped_mm_fwd(const void *x, const void *w, const int32_t *ends, void *y, int64_t rows,
                                      int64_t groups, int64_t N, int64_t K, swiglu_dtype_t dtype,
                                      swiglu_stream_t stream) {
    using namespace gmm;
    const swiglu_status_t st = check(rows, groups, N, K, dtype);
    if (st != SWIGLU_OK || rows == 0) return st;
    if (x == nullptr || w == nullptr || ends == nullptr || y == nullptr) return SWIGLU_ERR_NULL;
    if (!aligned({x, w, y}, 16) || !aligned({ends}, 4)) return SWIGLU_ERR_STRIDE;
    Span sx, sw, se, sy;
    if (!span_of(x, rows, K, K, 2, sx) || !span_of(w, groups * N, K, K, 2, sw) || !span_of(ends, groups, 1, 1, 4, se) ||
        !span_of(y, rows, N, N, 2, sy))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sy}, {sx, sw, se})) return SWIGLU_ERR_ALIAS;

    EncodeTiled enc;
    const cudaError_t e = encoder(enc);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    Params p{};
    if (!map3(enc, &p.a, w, K, N, groups, 128, 1) || !row_maps(enc, p.b, x, K, rows) ||
        !out_map(enc, &p.c, y, 2, N, rows, 0))
        return moe::cuda_fail(cudaErrorInvalidValue);
    p.ends = ends;
    p.out = y;
    p.rows = (int)rows;
    p.groups = (int)groups;
    p.features = (int)N;
    p.depth = (int)K;
    return launch_rows<kMm>(p, stream);
}

swiglu_status_t swiglu_grouped_mm_dgrad(const void *dy, const void *w, const int32_t *ends, void *dx, int64_t rows,
                                        int64_t groups, int64_t N, int64_t K, swiglu_dtype_t dtype,
                                        swiglu_stream_t stream) {
    using namespace gmm;
    const swiglu_status_t st = check(rows, groups, N, K, dtype);
    if (st != SWIGLU_OK || rows == 0) return st;
    if (dy == nullptr || w == nullptr || ends == nullptr || dx == nullptr) return SWIGLU_ERR_NULL;
    if (!aligned({dy, w, dx}, 16) || !aligned({ends}, 4)) return SWIGLU_ERR_STRIDE;
    Span sdy, sw, se, sdx;
    if (!span_of(dy, rows, N, N, 2, sdy) || !span_of(w, groups * N, K, K, 2, sw) ||
        !span_of(ends, groups, 1, 1, 4, se) || !span_of(dx, rows, K, K, 2, sdx))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sdx}, {sdy, sw, se})) return SWIGLU_ERR_ALIAS;

    EncodeTiled enc;
    const cudaError_t e = encoder(enc);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    Params p{};
    // the contraction runs over W's rows: boxes of 64 columns by 64 of them
    if (!map3(enc, &p.a, w, K, N, groups, BK, 1) || !row_maps(enc, p.b, dy, N, rows) ||
        !out_map(enc, &p.c, dx, 2, K, rows, 0))
        return moe::cuda_fail(cudaErrorInvalidValue);
    p.ends = ends;
    p.out = dx;
    p.rows = (int)rows;
    p.groups = (int)groups;
    p.features = (int)K;
    p.depth = (int)N;
    return launch_rows<kDgrad>(p, stream);
}

swiglu_status_t swiglu_grouped_mm_wgrad(const void *dy, const void *x, const int32_t *ends, void *dw, int64_t rows,
                                        int64_t groups, int64_t N, int64_t K, swiglu_dtype_t dtype,
                                        swiglu_dtype_t dw_dtype, int accumulate, swiglu_stream_t stream) {
    using namespace gmm;
    const swiglu_status_t st = check(rows, groups, N, K, dtype);
    if (st != SWIGLU_OK) return st;
    if (dw_dtype != SWIGLU_BF16 && dw_dtype != SWIGLU_F32) return SWIGLU_ERR_DTYPE;
    if (accumulate != 0 && dw_dtype != SWIGLU_F32) return SWIGLU_ERR_DTYPE;
    if (rows > SWIGLU_GROUPED_MAX_ROWS_WGRAD) return SWIGLU_ERR_SHAPE;
    const int eb = dw_dtype == SWIGLU_F32 ? 4 : 2;
    Span sdw;
    if (!span_of(dw, groups * N, K, K, eb, sdw)) return SWIGLU_ERR_SHAPE;
    if (rows == 0) {  // every group is empty
        if (accumulate != 0) return SWIGLU_OK;
        if (dw == nullptr) return SWIGLU_ERR_NULL;
        if (!aligned({dw}, 16)) return SWIGLU_ERR_STRIDE;
        const cudaError_t e = cudaMemsetAsync(dw, 0, sdw.hi - sdw.lo, reinterpret_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
    }
    if (dy == nullptr || x == nullptr || ends == nullptr || dw == nullptr) return SWIGLU_ERR_NULL;
    if (!aligned({dy, x, dw}, 16) || !aligned({ends}, 4)) return SWIGLU_ERR_STRIDE;
    Span sdy, sx, se;
    if (!span_of(dy, rows, N, N, 2, sdy) || !span_of(x, rows, K, K, 2, sx) || !span_of(ends, groups, 1, 1, 4, se))
        return SWIGLU_ERR_SHAPE;
    if (moe::any_alias({sdw}, {sdy, sx, se})) return SWIGLU_ERR_ALIAS;
    const int64_t pairs = groups * ceil_div(N, 256) * ceil_div(K, TILE_N);
    if (pairs > INT32_MAX / 4) return SWIGLU_ERR_SHAPE;

    EncodeTiled enc;
    const cudaError_t e = encoder(enc);
    if (e != cudaSuccess) return moe::cuda_fail(e);
    Params p{};
    p.ends = ends;
    p.out = dw;
    p.rows = (int)rows;
    p.groups = (int)groups;
    p.f32_out = dw_dtype == SWIGLU_F32;
    p.accumulate = accumulate != 0;
    // Pairs: M is dW's rows, N its columns.  Split: the other way round, so that the
    // lanes run along dW's rows.
    const int size = plan_wgrad(rows, groups, N, K).size;
    // where one group had all rows: does a sum have several segments?
    const bool sums = rows > (int64_t)(p.f32_out ? kSegmentRows : kLongRows) * (size > 0 ? size : 1);
    if (size > 0) {
        if (!map2(enc, &p.a, x, K, rows, BK) || !map2(enc, &p.b[0], dy, N, rows, BK))
            return moe::cuda_fail(cudaErrorInvalidValue);
        p.features = (int)K;
        p.cols = (int)N;
        const int64_t tiles = wgrad_split_tiles(groups, N, K);
        return sums ? launch_split<kWgrad, 128, true>(p, tiles, size, stream)
                    : launch_split<kWgrad, 128>(p, tiles, size, stream);
    }
    if (!map2(enc, &p.a, dy, N, rows, BK) || !map2(enc, &p.b[0], x, K, rows, BK) ||
        !out_map(enc, &p.c, dw, eb, K, N, groups))
        return moe::cuda_fail(cudaErrorInvalidValue);
    for (int h = 0; h < 6; ++h)
        if (!map2(enc, &p.part_a[h], dy, N, rows, 1 << h) || !map2(enc, &p.part_b[h], x, K, rows, 1 << h))
            return moe::cuda_fail(cudaErrorInvalidValue);
    p.features = (int)N;
    p.cols = (int)K;
    return sums ? launch_pairs<kWgrad, true>(p, pairs, stream) : launch_pairs<kWgrad>(p, pairs, stream);
}

swiglu_status_t swiglu_grouped_slices(swiglu_grouped_product_t product, int64_t rows, int64_t groups, int64_t N,
                                      int64_t K, swiglu_dtype_t dw_dtype, int *slices) {
    using namespace gmm;
    if (slices == nullptr) return SWIGLU_ERR_NULL;
    const swiglu_status_t st = check(rows, groups, N, K, SWIGLU_BF16);
    if (st != SWIGLU_OK) return st;
    if (product == SWIGLU_GROUPED_FC1 && 2 * N > SWIGLU_GROUPED_MAX_FEATURES / groups) return SWIGLU_ERR_SHAPE;
    if (rows == 0) {
        *slices = 0;
        return SWIGLU_OK;
    }
    switch (product) {
        case SWIGLU_GROUPED_FC1: *slices = plan_rows<kFc1>(rows, groups, N, K).size; return SWIGLU_OK;
        case SWIGLU_GROUPED_MM: *slices = plan_rows<kMm>(rows, groups, N, K).size; return SWIGLU_OK;
        case SWIGLU_GROUPED_DGRAD: *slices = plan_rows<kDgrad>(rows, groups, K, N).size; return SWIGLU_OK;
        case SWIGLU_GROUPED_WGRAD:
            if (dw_dtype != SWIGLU_BF16 && dw_dtype != SWIGLU_F32) return SWIGLU_ERR_DTYPE;
            if (rows > SWIGLU_GROUPED_MAX_ROWS_WGRAD) return SWIGLU_ERR_SHAPE;
            *slices = plan_wgrad(rows, groups, N, K).size;
            return SWIGLU_OK;
    }
    return SWIGLU_ERR_SHAPE;
}

swiglu_status_t swiglu_grouped_timeout_flag(int *flag) {
    if (flag == nullptr) return SWIGLU_ERR_NULL;
    const cudaError_t e = cudaMemcpyFromSymbol(flag, gmm::g_timeout, sizeof(int));
    return e == cudaSuccess ? SWIGLU_OK : moe::cuda_fail(e);
}

}  // extern "C"
