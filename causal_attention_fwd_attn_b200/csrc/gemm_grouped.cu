// gemm_grouped.cu -- the three products of a linear layer, grouped by expert, on tcgen05
// tensor cores: the rows [o_e, o_{e+1}) of the token matrices belong to expert e, and the
// offsets are read on the device, so that a router's counts never visit the host.
//   forward   y  = x w_e^T       backward  dx = dy w_e,   dw_e (+)= dy_e^T x_e
//
// Both kernels run on pairs of SMs (clusters of two blocks, cta_group::2): a product of
// 256 x N x 16 in which each block holds half of A's rows and half of B's, so that an
// operand byte in shared memory feeds twice the work that it does on one SM.  Shared-memory
// traffic is what paces the one-SM kernels (gemm.cu).
//
// Forward and dX are one kernel (grouped_rows_kernel).  It computes the transposed product:
// the weights' features are the 256 rows of a tile and the expert's tokens its columns, so
// that the ragged dimension is the one whose width a tcgen05 product can vary (any
// multiple of 32): an expert's rows are cut into equal tiles of at most BN tokens and
// each product is as wide as its tile.  Rows of a neighbouring expert that the last copy of
// a tile brings along only feed columns that are never stored.
// dW (grouped_dw_kernel) reduces over an expert's tokens, 64 to a step.  In the last step
// the rows after the expert's end are cleared in shared memory, in both operands (a
// neighbour's row may hold infinities, which a zero in one operand would not remove).
//
// Sums: a tensor core cuts the bits off that its accumulator has no room for, an error that
// points towards zero and grows with the number of additions (2.8e-6 relative after 2048 terms of
// both signs, 2e-5 after 16384; fp16 terms of one sign 2.8e-6 after 512, 6.9e-3 after 2^20).
// Reductions therefore leave tensor memory in chunks and go on in fp32 registers, rounded to
// nearest: every 512 terms for fp32 outputs (0.5e-6 for terms of both signs), every 4096 for 16-bit
// ones, where what a chunk loses (256 additions, 2^-23 each at most: 3.1e-5 of its terms'
// magnitudes) is small beside fp16's half step of 2^-11 and bf16's of 2^-8.
//
// What bounds them: the products and the copies that feed them where an expert has many rows (a
// k-block of a 256 x 256 tile brings 32 KB into each SM, 512 clocks at the 64 bytes a clock that L2
// gives it, as many as its products take; the forward takes 575 to 595 for it), the weights' HBM
// traffic where few.  16384 rows of eight equal experts, 2048 -> 4096, in short bursts: forward
// 184 us, 1490 TFLOP/s, dX 185; forward with fp32 outputs 210 (a chunk handed over every 512
// terms, and twice the bytes stored); dW, which has the same chunks and outputs, 215.  Experts
// whose rows are no multiple of 64 add 12 to dW (each unit's last copies wait for the rest to be
// cleared), uneven ones as much again: units have their expert's length and are dealt in order, 480
// k-blocks to the busiest pair against 450 on average: 236; accumulated 254.  Once the power limit
// has lowered the clock the forward of 16 experts takes 242 (1137 TFLOP/s), dW 278.  32 rows, 20 of 32
// experts: 58 us, 5.8 TB/s, 0.88 of the copy rate.
//
// Both are persistent, one block per SM.  Every block reads the offsets into shared
// memory (each clamped to the rows there are, so that no offsets can lead outside the
// tensors) and all pairs walk the (expert, tile) units in one common order.
#include <cmath>

#include "forge_attn.h"
#include "forge_internal.h"
#include "forge_linear.h"
#include "sm100_grouped_ptx.cuh"
#include "sm100_ptx.cuh"

namespace forge {
namespace {

constexpr int kMaxExperts = FORGE_LINEAR_MAX_EXPERTS;
constexpr int kMaxFeatures = FORGE_LINEAR_GROUPED_MAX_FEATURES;
// Warps: 0 copies, 1 issues the products (in the pair's first block), 2 clears tails (dW), from
// 4 on the epilogue, in groups of four (warp w reads tensor memory lanes 32 (w % 4)..).
constexpr int kGroups = 2;
constexpr int kThreads = 128 * (1 + kGroups);
constexpr int kBK = 64;
constexpr int kHalfM = 128;        // a block's rows of a pair's 256
constexpr int kAccCols = 256;      // tensor memory columns of one of the two accumulators
// k-blocks of a reduction's chunk, after which its sums leave tensor memory: for fp32 outputs, and
// for 16-bit ones (the forward of 16384 rows took 249 us with 8, 242 with 16, 240 with 64).  16-bit
// outputs of a single chunk are rounded as they leave (LONG = false): by way of the registers of
// sums 6712 rows of eight experts, 640 -> 992, took 16.0 us instead of 15.3.
constexpr int kChunk32 = 8, kChunk16 = 64;
constexpr int kMaxStages = 10;
constexpr int kMaxSmem = 232448;   // shared memory of a block

enum : uint32_t { kSiteFull = 1, kSiteEmpty, kSiteAccFull, kSiteAccEmpty, kSiteLanded };

struct Barriers {
    uint64_t full[kMaxStages], empty[kMaxStages], landed[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_final;
    uint32_t tmem_base;
    int abort;
    union {
        int cost[8];  // of the choices of choose_width (rows kernel)
        int begun;    // k-blocks whose copies this block's producer has begun (dW)
    };
};
static_assert(sizeof(Barriers) <= 320, "barrier block");
constexpr int kBarBytes = 320;

// The experts' rows and units: first[e] the first row, unit0[e] the first unit.  In shared
// memory, after everything else, and no larger than the experts need.
struct Tables {
    int *first, *count, *unit0;  // [experts + 1] each
    __device__ Tables(uint8_t* at, int experts)
        : first(reinterpret_cast<int*>(at)), count(first + experts + 1), unit0(count + experts + 1) {}
};
__host__ __device__ constexpr int tables_bytes(int experts) { return 3 * (experts + 1) * 4; }

// A place in the ring of stages.
struct Ring {
    int st = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++st == stages) {
            st = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t site,
                                          volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, site, abort));
}

// Fills the tables: `units_of(rows)` units to an expert, asked after `counted()`, which the
// whole block calls once the rows are known.  Ends with a barrier.
template <typename G, typename F>
__device__ __forceinline__ void fill_tables(const Tables& t, const int* offsets, int experts, int rows,
                                            G counted, F units_of) {
    for (int e = threadIdx.x; e <= experts; e += blockDim.x)
        t.first[e] = min(max(offsets[e], 0), rows);
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += blockDim.x)
        t.count[e] = max(t.first[e + 1] - t.first[e], 0);
    __syncthreads();
    counted();
    if (warp_id() == 0) {
        int base = 0;
        for (int e0 = 0; e0 < experts; e0 += 32) {
            const int e = e0 + (int)lane_id();
            int u = e < experts ? units_of(t.count[e]) : 0;
            int sum = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int below = __shfl_up_sync(0xffffffffu, sum, o);
                if ((int)lane_id() >= o) sum += below;
            }
            if (e < experts) t.unit0[e] = base + sum - u;
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane_id() == 0) t.unit0[experts] = base;
    }
    __syncthreads();
}

// Start of both kernels: barriers, tensor memory, tables; the pair begins together.
// `full_count`: arrivals that a stage's products wait for.
template <typename G, typename F>
__device__ __forceinline__ void start(Barriers* bars, const Tables& tab, int stages, int full_count,
                                      const int* offsets, int experts, int rows, G counted, F units_of) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&bars->full[i], full_count);
            mbar_init(&bars->empty[i], 1);
            mbar_init(&bars->landed[i], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 2 * 4 * kGroups);
        }
        mbar_init(&bars->mma_final, 1);
        bars->abort = 0;
        bars->begun = 0;
        fence_mbar_init();
    }
    if (warp_id() == 1) {
        tmem_alloc_pair(&bars->tmem_base, 2 * kAccCols);
        tmem_relinquish_pair();
    }
    allow_dependents_launch();
    grid_dependency_wait();  // nothing above read or wrote global memory
    fill_tables(tab, offsets, experts, rows, counted, units_of);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
}

// End of both kernels: neither block leaves (or gives up tensor memory) while the other may
// still read or signal it.  The wait for the last signal begins when the block's own work has
// ended (the second block's warp 1 has none, and a launch may take longer than a wait's limit).
__device__ __forceinline__ void finish(Barriers* bars) {
    __syncthreads();
    if (warp_id() == 1) mbar_wait_drain(&bars->mma_final, 0);  // all products and signals
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp_id() == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(bars->tmem_base, 2 * kAccCols);
    }
}

// ------------------------------------------------------------------ forward and dX ----
constexpr int kStageRows = 32;  // token rows of one staging buffer of the epilogue

// BN: tokens of a pair's tile at most.  LONG: 16-bit outputs whose reduction takes several chunks.
template <int BN, bool OUT32, bool LONG>
struct RowsCfg {
    static constexpr bool kSums = OUT32 || LONG;  // added up in registers
    static constexpr int kABytes = kHalfM * kBK * 2;
    static constexpr int kStageBytes = kABytes + BN / 2 * kBK * 2;
    static constexpr int kRowBytes = kHalfM * (OUT32 ? 4 : 2);
    static constexpr int kChunk = OUT32 ? kChunk32 : kChunk16;
    // 32-token steps of an accumulator that a group of epilogue warps takes
    static constexpr int kSteps = BN / kStageRows / kGroups;
    static constexpr int kStagingBytes = kGroups * kStageRows * kRowBytes;
    static constexpr int kRest = kStagingBytes + kBarBytes + 1024;
    // stages that fit beside the tables of that many experts
    static constexpr int stages(int experts) {
        const int fit = (kMaxSmem - kRest - tables_bytes(experts)) / kStageBytes;
        return fit < kMaxStages ? fit : kMaxStages;
    }
    static_assert(!(OUT32 && LONG) && stages(kMaxExperts) >= 4 && kSteps >= 1, "shared memory budget");
};

struct RowsShape {
    int rows, experts, features, k_blocks, feature_tiles, stages;
};

// A token matrix in boxes of 64 x 16 (n + 1): what a block copies of a product 32 (n + 1) wide,
// no more.
struct TokenMaps {
    CUtensorMap box[8];
};

__device__ __forceinline__ int round32(int n) { return (n + 31) / 32 * 32; }

// An expert's tokens are cut into equal tiles of at most `most`.
__device__ __forceinline__ int tiles_of(int count, int most) { return (count + most - 1) / most; }
__device__ __forceinline__ int width_of(int count, int tiles) {
    return round32((count + tiles - 1) / tiles);
}

// One unit: features [fm, fm + 256) of expert e for the token rows [r0, r0 + n), products of
// `width` columns.
struct RowsUnit {
    int e, fm, r0, n, width;
};
__device__ __forceinline__ RowsUnit rows_unit(const Tables& t, int most, int u, int& e) {
    while (u >= t.unit0[e + 1]) ++e;
    const int local = u - t.unit0[e], cnt = t.count[e];
    const int tiles = tiles_of(cnt, most);
    const int f = local / tiles, tn = local - f * tiles;
    const int width = width_of(cnt, tiles);
    const int n = min(width, cnt - tn * width);
    return RowsUnit{e, f * 2 * kHalfM, t.first[e] + tn * width, n, round32(n)};
}

// The widest tile (BN, or down to BN / 2 in steps of 32) with the least work for the busiest pair:
// the waves of units times what one costs.  Copies pace the kernel: a row of a k-block takes
// 256 bytes of weights and one byte for each column, 64 bytes a clock and SM, where the
// products take two clocks a column.  (Tiles of 512 columns, both accumulators to one tile,
// copy a third less but cannot overlap their epilogue: forward of 16384 rows, 16 experts,
// 2048 -> 4096 213 us against 201, not kept.)  A warp weighs each choice; called by the block.
template <int BN>
__device__ __forceinline__ int choose_width(const Tables& t, int experts, int feature_tiles,
                                            int pairs, int* cost) {
    constexpr int kChoices = BN <= 64 ? 1 : (BN / 64 < 8 ? BN / 64 : 8);
    if (kChoices == 1) return BN;
    if ((int)warp_id() < kChoices) {
        const int most = BN - 32 * (int)warp_id();
        int units = 0, columns = 0;
        for (int e = lane_id(); e < experts; e += 32) {
            const int cnt = t.count[e];
            if (cnt == 0) continue;
            const int tiles = tiles_of(cnt, most);
            units += tiles;
            columns += tiles * width_of(cnt, tiles);
        }
        units = __reduce_add_sync(0xffffffffu, units);
        columns = __reduce_add_sync(0xffffffffu, columns);
        const int waves = (int)(((long long)units * feature_tiles + pairs - 1) / pairs);
        if (lane_id() == 0)
            cost[warp_id()] = waves * (256 + (units ? columns / units : 0));
    }
    __syncthreads();
    int best = 0;
    for (int k = 1; k < kChoices; ++k)
        if (cost[k] < cost[best]) best = k;
    return BN - 32 * best;
}

template <int BN, bool W_MN, bool OUT32, bool F16, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_rows_kernel(const __grid_constant__ CUtensorMap tmap_w,
                        const __grid_constant__ TokenMaps tmap_x,
                        const int* offsets, void* out, const RowsShape s) {
    using C = RowsCfg<BN, OUT32, LONG>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = s.stages;
    uint8_t* const staging0 = smem + stages * C::kStageBytes;
    Barriers* bars = reinterpret_cast<Barriers*>(staging0 + C::kStagingBytes);
    const Tables tab(reinterpret_cast<uint8_t*>(bars) + kBarBytes, s.experts);
    volatile int* abort = &bars->abort;
    const uint32_t warp = warp_id(), lane = lane_id(), rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int ft = s.feature_tiles;
    int most = BN;
    start(bars, tab, stages, 1, offsets, s.experts, s.rows,
          [&] { most = choose_width<BN>(tab, s.experts, ft, pairs, bars->cost); },
          [&](int n) { return tiles_of(n, most) * ft; });
    const uint32_t tmem = bars->tmem_base;
    const int units = tab.unit0[s.experts];

    if (warp == 0) {
        // Producer.  Both blocks' copies are counted on the first block's barrier.
        if (lane == 0) {
            tma_prefetch_desc(&tmap_w);
            int it = 0, e = 0;
            Ring at;
            bool run = true;
            for (int u = pair; run && u < units; u += pairs) {
                const RowsUnit w = rows_unit(tab, most, u, e);
                const int fm = w.fm + (int)rank * kHalfM;
                const int r0 = w.r0 + (int)rank * (w.width / 2);
                const int bytes = C::kABytes + w.width / 2 * (kBK * 2);
                const CUtensorMap* box = &tmap_x.box[w.width / 32 - 1];
                for (int kb = 0; kb < s.k_blocks; ++kb, ++it, at.next(stages)) {
                    const int st = at.st;
                    if (it >= stages &&
                        !mbar_wait(&bars->empty[st], at.phase ^ 1, kSiteEmpty, abort)) {
                        run = false;
                        break;
                    }
                    uint8_t* sa = smem + st * C::kStageBytes;
                    const uint32_t bar = cluster_addr(&bars->full[st], 0);
                    if (rank == 0) mbar_arrive_expect_tx(&bars->full[st], 2 * bytes);
                    if constexpr (W_MN) {
                        for (int c = 0; c < kHalfM / 64; ++c)
                            tma_load_3d_pair(sa + c * (kBK * 128), &tmap_w, bar, fm + 64 * c,
                                             kb * kBK, w.e);
                    } else {
                        tma_load_3d_pair(sa, &tmap_w, bar, kb * kBK, fm, w.e);
                    }
                    tma_load_2d_pair(sa + C::kABytes, box, bar, kb * kBK, r0);
                }
            }
            if (*abort && rank == 0)  // let copies already issued land before the pair ends
                for (int k = max(0, it - stages); k < it; ++k)
                    mbar_wait_drain(&bars->full[k % stages], (k / stages) & 1);
        }
    } else if (warp == 1 && rank == 0) {
        // MMA issuer.
        constexpr uint32_t kIdesc0 = idesc_f16kind_f32(2 * kHalfM, 0, W_MN, false, F16);
        Ring at;
        int n_acc = 0, e = 0;
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs) {
            const RowsUnit w = rows_unit(tab, most, u, e);
            const uint32_t idesc = kIdesc0 | ((uint32_t)(w.width >> 3) << 17);
            for (int kb0 = 0; ok && kb0 < s.k_blocks; ++n_acc) {
                const int kb1 = C::kSums ? min(kb0 + C::kChunk, s.k_blocks) : s.k_blocks;
                const int buf = n_acc & 1, use = n_acc >> 1;
                if (use > 0 &&
                    !warp_wait(&bars->acc_empty[buf], (use - 1) & 1, kSiteAccEmpty, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tacc = tmem + buf * kAccCols;
                for (int kb = kb0; kb < kb1; ++kb, at.next(stages)) {
                    const int st = at.st;
                    if (!warp_wait(&bars->full[st], at.phase, kSiteFull, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + st * C::kStageBytes), b = a + C::kABytes;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        const uint64_t ad = W_MN ? sdesc_sw128(a + kk * 2048, kBK * 128, 1024)
                                                 : sdesc_sw128(a + kk * 32, 16, 1024);
                        mma_ss_pair_warp(tacc, ad, sdesc_sw128(b + kk * 32, 16, 1024), idesc,
                                         (kb > kb0 || kk > 0) ? 1u : 0u);
                    }
                    mma_commit_pair_warp(&bars->empty[st]);
                }
                if (ok) mma_commit_pair_warp(&bars->acc_full[buf]);
                kb0 = kb1;
            }
        }
        mma_commit_pair_warp(&bars->mma_final);
    } else if (warp >= 4) {
        // Epilogue.  A thread reads its feature's accumulators 32 tokens at a time (a group of
        // four warps every second 32), hands them back, and turns them into rows of 128
        // features in shared memory, which the group stores whole.
        const uint32_t quarter = warp & 3, group = (warp >> 2) - 1;
        const uint32_t lane_off = (quarter * 32u) << 16;
        const int tid = (int)threadIdx.x - 128 * (1 + (int)group);
        constexpr int kEl = OUT32 ? 4 : 2, kRowBytes = C::kRowBytes, kChunks = kRowBytes / 16;
        uint8_t* staging = staging0 + group * (kStageRows * kRowBytes);
        const uint32_t empty_bar[2] = {cluster_addr(&bars->acc_empty[0], 0),
                                       cluster_addr(&bars->acc_empty[1], 0)};
        int n_acc = 0, e = 0;
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs) {
            const RowsUnit w = rows_unit(tab, most, u, e);
            const int fm = w.fm + (int)rank * kHalfM;
            uint32_t kept[C::kSteps][C::kSums ? 32 : 16];  // sums in fp32, or 16-bit pairs
            if constexpr (C::kSums) {
#pragma unroll
                for (int q = 0; q < C::kSteps; ++q)
#pragma unroll
                    for (int j = 0; j < 32; ++j) kept[q][j] = 0u;
            }
            const int chunks = C::kSums ? (s.k_blocks + C::kChunk - 1) / C::kChunk : 1;
            for (int c = 0; c < chunks; ++c, ++n_acc) {
                const int buf = n_acc & 1;
                // the group goes on, or gives up, together: it meets at barriers below
                ok = named_barrier_all(
                    1 + group, 128,
                    warp_wait(&bars->acc_full[buf], (n_acc >> 1) & 1, kSiteAccFull, abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < C::kSteps; ++q) {
                    const int c0 = (kGroups * q + (int)group) * kStageRows;
                    if (c0 >= w.width) break;
                    const uint32_t from = tmem + lane_off + buf * kAccCols + c0;
                    if constexpr (C::kSums) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r[16];
                            tmem_ld16(from + 16 * h, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                kept[q][16 * h + j] =
                                    __float_as_uint(__uint_as_float(kept[q][16 * h + j]) +
                                                    __uint_as_float(r[j]));
                        }
                    } else {
                        uint32_t r[32];
                        tmem_ld32(from, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            kept[q][j] = pack16x2<F16>(__uint_as_float(r[2 * j]),
                                                       __uint_as_float(r[2 * j + 1]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(empty_bar[buf]);
            }
            if (!ok) break;
#pragma unroll
            for (int q = 0; q < C::kSteps; ++q) {
                const int c0 = (kGroups * q + (int)group) * kStageRows;
                if (c0 >= w.width) break;
                named_barrier_sync(1 + group, 128);  // the staging rows have been read
#pragma unroll
                for (int j = 0; j < kStageRows; j += 2) {
                    uint8_t* dst = staging + j * kRowBytes + (quarter * 32 + lane) * kEl;
                    if constexpr (OUT32) {
                        *reinterpret_cast<uint32_t*>(dst) = kept[q][j];
                        *reinterpret_cast<uint32_t*>(dst + kRowBytes) = kept[q][j + 1];
                    } else {
                        const uint32_t two = LONG ? pack16x2<F16>(__uint_as_float(kept[q][j]),
                                                                  __uint_as_float(kept[q][j + 1]))
                                                  : kept[q][j / 2];
                        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)two;
                        *reinterpret_cast<uint16_t*>(dst + kRowBytes) = (uint16_t)(two >> 16);
                    }
                }
                named_barrier_sync(1 + group, 128);
                const int live = min(kStageRows, w.n - c0);
                for (int k = tid; k < live * kChunks; k += 128) {
                    const int row = k / kChunks, col = (k - row * kChunks) * (16 / kEl);
                    if (fm + col >= s.features) continue;
                    const uint4 v = *reinterpret_cast<const uint4*>(staging + k * 16);
                    const long long off = (long long)(w.r0 + c0 + row) * s.features + fm + col;
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + off * kEl) = v;
                }
            }
        }
    }
    finish(bars);
}

// ---------------------------------------------------------------------------- dW ----
constexpr int kDwHalfBytes = kHalfM * kBK * 2;  // a block's half of either operand
constexpr int kDwStageBytes = 2 * kDwHalfBytes;
constexpr int kDwBoxBytes = 32 * 128;  // one 32 x 32 fp32 box; two to a warp
constexpr int kDwStagingBytes = kGroups * 4 * 2 * kDwBoxBytes;
// Five stages beside the tables of up to 143 experts, four beside larger ones (dW of 16384
// rows, 8 experts, 2048 -> 4096: 235 us with five, 240 with four, 262 with three).
constexpr int dw_stages(int experts) {
    return (kMaxSmem - kDwStagingBytes - kBarBytes - 1024 - tables_bytes(experts)) / kDwStageBytes;
}
static_assert(dw_stages(kMaxExperts) >= 4 && dw_stages(1) <= kMaxStages, "shared memory budget");

struct DwShape {
    int rows, experts, m, n, tiles_m, tiles_n, stages;
};

struct DwUnit {
    int e, m0, n0, r0, count;
};
__device__ __forceinline__ DwUnit dw_unit(const Tables& t, const DwShape& s, int u, int& e) {
    while (u >= t.unit0[e + 1]) ++e;
    const int local = u - t.unit0[e];
    const int tn = local / s.tiles_m, tm = local - tn * s.tiles_m;
    return DwUnit{e, tm * 2 * kHalfM, tn * 2 * kHalfM, t.first[e], t.count[e]};
}

// Clears rows [valid, 64) of the 64-row chunks of a stage (each row is 128 bytes, whatever
// the swizzle does inside it).
__device__ __forceinline__ void clear_rows(uint8_t* stage, int valid, uint32_t lane) {
    const int per = (kBK - valid) * 8;
    for (int c = 0; c < kDwStageBytes / (kBK * 128); ++c)
        for (int r = lane; r < per; r += 32)
            *reinterpret_cast<uint4*>(stage + c * (kBK * 128) + valid * 128 + r * 16) =
                make_uint4(0, 0, 0, 0);
}

// Waits for a tail's copies.  They come after all others of the expert's reduction, and of units
// without a tail before it: 4 million k-blocks and more, longer than one wait may take.
// The limit therefore counts from the last k-block that the producer began.
__device__ __forceinline__ bool wait_landed(uint64_t* bar, uint32_t parity, const volatile int* begun,
                                            volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    int seen = *begun;
    uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) != 0) continue;
        if (*abort) return false;
        const int now = *begun;
        if (now != seen) {
            seen = now;
            t0 = globaltimer_ns();
        } else if (globaltimer_ns() - t0 > FORGE_WAIT_LIMIT_NS) {
            record_timeout(kSiteLanded);
            *abort = 1;
            return false;
        }
    }
}

template <bool ADD, bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_dw_kernel(const __grid_constant__ CUtensorMap tmap_dy,
                      const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ CUtensorMap tmap_dw,
                      const int* offsets, const DwShape s) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = s.stages;
    uint8_t* const staging0 = smem + stages * kDwStageBytes;
    Barriers* bars = reinterpret_cast<Barriers*>(staging0 + kDwStagingBytes);
    const Tables tab(reinterpret_cast<uint8_t*>(bars) + kBarBytes, s.experts);
    volatile int *abort = &bars->abort, *begun = &bars->begun;
    const uint32_t warp = warp_id(), lane = lane_id(), rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    // an expert without rows has a zero gradient: written, or nothing to add
    const int per = s.tiles_m * s.tiles_n;
    start(bars, tab, stages, 2, offsets, s.experts, s.rows, [] {},
          [per](int n) { return ADD && n == 0 ? 0 : per; });
    const uint32_t tmem = bars->tmem_base;
    const int units = tab.unit0[s.experts];

    if (warp == 0) {
        // Producer.  A stage's products wait for both blocks: for the bytes of both on the
        // first block's barrier, and for an arrival of each.  A tail (less than 64 rows) lands on
        // its block's own barrier, for warp 2 to clear the rest and arrive.
        if (lane == 0) {
            tma_prefetch_desc(&tmap_dy);
            tma_prefetch_desc(&tmap_x);
            int it = 0, e = 0;
            Ring at;
            uint32_t tail_phases = 0;  // of the stages' `landed`
            bool run = true;
            for (int u = pair; run && u < units; u += pairs) {
                const DwUnit w = dw_unit(tab, s, u, e);
                const int m0 = w.m0 + (int)rank * kHalfM, n0 = w.n0 + (int)rank * kHalfM;
                for (int k0 = 0; k0 < w.count; k0 += kBK, ++it, at.next(stages)) {
                    const int st = at.st;
                    if (it >= stages &&
                        !mbar_wait(&bars->empty[st], at.phase ^ 1, kSiteEmpty, abort)) {
                        run = false;
                        break;
                    }
                    uint8_t* sa = smem + st * kDwStageBytes;
                    const bool tail = w.count - k0 < kBK;
                    const uint32_t bar = tail ? smem_u32(&bars->landed[st])
                                              : cluster_addr(&bars->full[st], 0);
                    if (tail) tail_phases ^= 1u << st;
                    mbar_arrive_expect_tx_at(bar, kDwStageBytes);
                    for (int c = 0; c < kHalfM / 64; ++c) {
                        tma_load_2d_pair(sa + c * (kBK * 128), &tmap_dy, bar, m0 + 64 * c, w.r0 + k0);
                        tma_load_2d_pair(sa + kDwHalfBytes + c * (kBK * 128), &tmap_x, bar,
                                         n0 + 64 * c, w.r0 + k0);
                    }
                    *begun = it + 1;
                }
            }
            if (*abort)  // let copies already issued land before the pair ends
                for (int k = max(0, it - stages); k < it; ++k) {
                    const int st = k % stages;
                    if (rank == 0) mbar_wait_drain(&bars->full[st], (k / stages) & 1);
                    mbar_wait_drain(&bars->landed[st], ((tail_phases >> st) & 1) ^ 1);
                }
        }
    } else if (warp == 2) {
        // Clears the tails.
        uint32_t tail_phases = 0;
        int it = 0, e = 0;
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs) {
            const DwUnit w = dw_unit(tab, s, u, e);
            const int blocks = (w.count + kBK - 1) / kBK, valid = w.count % kBK;
            it += blocks;
            if (valid == 0) continue;
            const int st = (it - 1) % stages;
            ok = __all_sync(0xffffffffu,
                            wait_landed(&bars->landed[st], (tail_phases >> st) & 1, begun, abort));
            if (!ok) break;
            tail_phases ^= 1u << st;
            clear_rows(smem + st * kDwStageBytes, valid, lane);
            fence_proxy_async_smem();
            fence_cluster();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(cluster_addr(&bars->full[st], 0));
        }
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t kIdesc = idesc_f16kind_f32(2 * kHalfM, 2 * kHalfM, true, true, F16);
        Ring at;
        int n_acc = 0, e = 0;
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs) {
            const DwUnit w = dw_unit(tab, s, u, e);
            const int blocks = (w.count + kBK - 1) / kBK;
            for (int kb0 = 0; ok && kb0 < blocks; kb0 += kChunk32, ++n_acc) {
                const int kb1 = min(kb0 + kChunk32, blocks);
                const int buf = n_acc & 1, use = n_acc >> 1;
                if (use > 0 &&
                    !warp_wait(&bars->acc_empty[buf], (use - 1) & 1, kSiteAccEmpty, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tacc = tmem + buf * kAccCols;
                for (int kb = kb0; kb < kb1; ++kb, at.next(stages)) {
                    const int st = at.st;
                    if (!warp_wait(&bars->full[st], at.phase, kSiteFull, abort)) {
                        ok = false;
                        break;
                    }
                    if (w.count - kb * kBK < kBK) fence_cluster();  // rows that were cleared
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + st * kDwStageBytes), b = a + kDwHalfBytes;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        mma_ss_pair_warp(tacc, sdesc_sw128(a + kk * 2048, kBK * 128, 1024),
                                         sdesc_sw128(b + kk * 2048, kBK * 128, 1024), kIdesc,
                                         (kb > kb0 || kk > 0) ? 1u : 0u);
                    mma_commit_pair_warp(&bars->empty[st]);
                }
                if (ok) mma_commit_pair_warp(&bars->acc_full[buf]);
            }
        }
        mma_commit_pair_warp(&bars->mma_final);
    } else if (warp >= 4) {
        // Epilogue.  A thread adds up its row's 128 columns over the chunks in registers; then
        // a warp stages its 32 rows in boxes of 32 columns (128-byte swizzle) and one lane
        // hands them to the copy engine, which clips them at the expert's last row and column
        // and, when accumulating, adds them (one addition per element).
        const uint32_t quarter = warp & 3, half = (warp >> 2) - 1;
        const uint32_t lane_off = (quarter * 32u) << 16;
        uint8_t* box = staging0 + (warp - 4) * 2 * kDwBoxBytes;
        const uint32_t empty_bar[2] = {cluster_addr(&bars->acc_empty[0], 0),
                                       cluster_addr(&bars->acc_empty[1], 0)};
        int n_acc = 0, e = 0;
        bool ok = true;
        for (int u = pair; ok && u < units; u += pairs) {
            const DwUnit w = dw_unit(tab, s, u, e);
            const int chunks = (w.count + kChunk32 * kBK - 1) / (kChunk32 * kBK);
            float sum[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) sum[j] = 0.f;
            for (int c = 0; c < chunks; ++c, ++n_acc) {
                const int buf = n_acc & 1;
                if (!warp_wait(&bars->acc_full[buf], (n_acc >> 1) & 1, kSiteAccFull, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint32_t r[16];
                    tmem_ld16(tmem + lane_off + buf * kAccCols + half * 128 + 16 * q, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[16 * q + j] += __uint_as_float(r[j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(empty_bar[buf]);
            }
            if (!ok) break;
            const int row = w.m0 + (int)(rank * kHalfM + quarter * 32);
            const int col = w.n0 + (int)half * 128;
            if (row >= s.m) continue;
#pragma unroll
            for (int c = 0; c < 4; c += 2) {  // two boxes to a fence and a wait
                if (col + 32 * c >= s.n) break;
                if (lane == 0) tma_store_wait_all_read();
                __syncwarp();
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float* v = sum + 32 * (c + b) + 4 * j;
                        *reinterpret_cast<float4*>(box + b * kDwBoxBytes + sw128_offset(lane, j)) =
                            make_float4(v[0], v[1], v[2], v[3]);
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    for (int b = 0; b < 2 && col + 32 * (c + b) < s.n; ++b) {
                        const uint8_t* src = box + b * kDwBoxBytes;
                        if constexpr (ADD)
                            tma_reduce_add_3d(&tmap_dw, src, col + 32 * (c + b), row, w.e);
                        else tma_store_3d(&tmap_dw, src, col + 32 * (c + b), row, w.e);
                    }
                    tma_store_commit();
                }
            }
        }
        if (lane == 0) tma_store_wait_all();
    }
    finish(bars);
}

// ------------------------------------------------------------------------- host ----
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dims(int rows, int experts, int in_f, int out_f) {
    if (rows < 0 || experts < 1 || in_f < 1 || out_f < 1) return FORGE_ATTN_ERR_INVALID_ARG;
    if (experts > kMaxExperts || in_f % 8 || out_f % 8) return FORGE_ATTN_ERR_UNSUPPORTED;
    // (the range that the sums' errors are stated and tested for)
    if (in_f > kMaxFeatures || out_f > kMaxFeatures) return FORGE_ATTN_ERR_UNSUPPORTED;
    if ((long long)rows * in_f >= (1ll << 31) || (long long)rows * out_f >= (1ll << 31) ||
        (long long)out_f * in_f >= (1ll << 31))
        return FORGE_ATTN_ERR_UNSUPPORTED;
    return FORGE_ATTN_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? FORGE_ATTN_OK : FORGE_ATTN_ERR_CUDA; }

// Blocks of a launch: two to a pair, as many pairs as there are units or SMs for.
int grid_of(long long units) {
    const int pairs = sm_count() / 2;
    return 2 * (units < 1 ? 1 : (units < pairs ? (int)units : pairs));
}

template <int BN, bool W_MN, bool OUT32, bool F16, bool LONG>
cudaError_t launch_rows_t(const CUtensorMap& tw, const TokenMaps& tx, const int* offsets,
                          void* out, const RowsShape& s, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured{0};
    auto* kernel = grouped_rows_kernel<BN, W_MN, OUT32, F16, LONG>;
    using C = RowsCfg<BN, OUT32, LONG>;
    cudaError_t e = set_max_dynamic_smem(kernel, kMaxSmem, configured);
    if (e != cudaSuccess) return e;
    RowsShape shape = s;
    shape.stages = C::stages(s.experts);
    const int smem = shape.stages * C::kStageBytes + C::kRest + tables_bytes(s.experts);
    // units: at most one partly filled tile to an expert on top of the full ones, with tiles of
    // BN / 2 and more
    const long long units = ((long long)s.rows / (BN / 2) + s.experts) * s.feature_tiles;
    return launch_dependent(kernel, dim3(grid_of(units)), dim3(kThreads), smem, stream, tw, tx, offsets,
                            out, shape);
}

template <int BN, bool W_MN>
cudaError_t launch_rows_n(const CUtensorMap& tw, const TokenMaps& tx, const int* offsets,
                          void* out, const RowsShape& s, bool f32, bool f16, cudaStream_t cs) {
    if (f32)
        return f16 ? launch_rows_t<BN, W_MN, true, true, false>(tw, tx, offsets, out, s, cs)
                   : launch_rows_t<BN, W_MN, true, false, false>(tw, tx, offsets, out, s, cs);
    if (s.k_blocks > kChunk16)
        return f16 ? launch_rows_t<BN, W_MN, false, true, true>(tw, tx, offsets, out, s, cs)
                   : launch_rows_t<BN, W_MN, false, false, true>(tw, tx, offsets, out, s, cs);
    return f16 ? launch_rows_t<BN, W_MN, false, true, false>(tw, tx, offsets, out, s, cs)
               : launch_rows_t<BN, W_MN, false, false, false>(tw, tx, offsets, out, s, cs);
}

template <bool W_MN>
int launch_rows(const void* x, const void* w, void* out, const int* offsets, int rows, int experts,
                int in_f, int out_f, int flags, void* stream) {
    if (!w || !offsets) return FORGE_ATTN_ERR_INVALID_ARG;
    int st = check_dims(rows, experts, in_f, out_f);
    if (st != FORGE_ATTN_OK) return st;
    if (flags & ~(FORGE_ATTN_OUT_F32 | FORGE_ATTN_FP16)) return FORGE_ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(offsets) & 3u) return FORGE_ATTN_ERR_MISALIGNED;
    if (rows == 0) return FORGE_ATTN_OK;
    if (!x || !out) return FORGE_ATTN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(out)) return FORGE_ATTN_ERR_MISALIGNED;
    const bool f16 = (flags & FORGE_ATTN_FP16) != 0, f32 = (flags & FORGE_ATTN_OUT_F32) != 0;
    const int k = W_MN ? out_f : in_f, features = W_MN ? in_f : out_f;
    // Tokens of a tile: the host knows the rows but not who has them, so it goes by the
    // experts' mean.  A tile wider than an expert's rows copies rows that it does not need; a
    // narrower one reads the expert's weights once for each of its tiles.  Where even tiles half
    // as wide leave pairs of SMs without any, they are halved.
    const int feature_tiles = (features + 2 * kHalfM - 1) / (2 * kHalfM);
    const int mean = (rows + experts - 1) / experts, busy = rows < experts ? rows : experts;
    int bn = mean <= 64 ? 64 : (mean <= 128 ? 128 : 256);
    while (bn > 64 && (long long)feature_tiles * busy * ((2 * mean + bn - 1) / bn) <= sm_count() / 2)
        bn /= 2;
    CUtensorMap tw;
    TokenMaps tx;
    if (encode_map_3d(&tw, w, in_f, out_f, experts, 64, W_MN ? 64 : kHalfM,
                      f16 ? kMapF16 : kMapBf16) != cudaSuccess)
        return FORGE_ATTN_ERR_CUDA;
    for (int n = 0; n < bn / 32; ++n)
        if (encode_map_2d16(&tx.box[n], x, k, rows, 64, 16 * (n + 1), f16) != cudaSuccess)
            return FORGE_ATTN_ERR_CUDA;
    const RowsShape s{rows, experts, features, (k + kBK - 1) / kBK, feature_tiles, 0};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return status_of(bn == 64    ? launch_rows_n<64, W_MN>(tw, tx, offsets, out, s, f32, f16, cs)
                     : bn == 128 ? launch_rows_n<128, W_MN>(tw, tx, offsets, out, s, f32, f16, cs)
                                 : launch_rows_n<256, W_MN>(tw, tx, offsets, out, s, f32, f16, cs));
}

template <bool ADD, bool F16>
cudaError_t launch_dw_t(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td,
                        const int* offsets, const DwShape& s, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured{0};
    auto* kernel = grouped_dw_kernel<ADD, F16>;
    cudaError_t e = set_max_dynamic_smem(kernel, kMaxSmem, configured);
    if (e != cudaSuccess) return e;
    const int smem = s.stages * kDwStageBytes + kDwStagingBytes + kBarBytes + 1024 +
                     tables_bytes(s.experts);
    const long long units = (long long)s.experts * s.tiles_m * s.tiles_n;
    return launch_dependent(kernel, dim3(grid_of(units)), dim3(kThreads), smem, stream, ta, tb, td,
                            offsets, s);
}

}  // namespace

cudaError_t read_and_clear_device_error_grouped(unsigned int* value) {
    return read_and_clear_unit_error(value);
}

}  // namespace forge

using namespace forge;

extern "C" {

int forge_linear_grouped_fwd(const void* x, const void* w, void* y, const int* offsets, int rows,
                             int experts, int in_features, int out_features, int flags,
                             void* stream) {
    return launch_rows<false>(x, w, y, offsets, rows, experts, in_features, out_features, flags,
                              stream);
}

int forge_linear_grouped_bwd_dx(const void* dy, const void* w, void* dx, const int* offsets,
                                int rows, int experts, int in_features, int out_features, int flags,
                                void* stream) {
    return launch_rows<true>(dy, w, dx, offsets, rows, experts, in_features, out_features, flags,
                             stream);
}

int forge_linear_grouped_bwd_dw(const void* dy, const void* x, float* dw, const int* offsets,
                                int rows, int experts, int in_features, int out_features,
                                int accumulate, int flags, void* stream) {
    if (!dw || !offsets) return FORGE_ATTN_ERR_INVALID_ARG;
    int st = check_dims(rows, experts, in_features, out_features);
    if (st != FORGE_ATTN_OK) return st;
    if (accumulate != 0 && accumulate != 1) return FORGE_ATTN_ERR_INVALID_ARG;
    if (flags & ~FORGE_ATTN_FP16) return FORGE_ATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(offsets) & 3u) || !aligned16(dw))
        return FORGE_ATTN_ERR_MISALIGNED;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // every expert is empty
        if (accumulate) return FORGE_ATTN_OK;
        return status_of(cudaMemsetAsync(
            dw, 0, (size_t)experts * in_features * out_features * sizeof(float), cs));
    }
    if (!dy || !x) return FORGE_ATTN_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x)) return FORGE_ATTN_ERR_MISALIGNED;
    const bool f16 = (flags & FORGE_ATTN_FP16) != 0;
    CUtensorMap ta, tb, td;
    if (encode_map_2d16(&ta, dy, out_features, rows, 64, kBK, f16) != cudaSuccess ||
        encode_map_2d16(&tb, x, in_features, rows, 64, kBK, f16) != cudaSuccess ||
        encode_map_3d(&td, dw, in_features, out_features, experts, 32, 32, kMapF32) != cudaSuccess)
        return FORGE_ATTN_ERR_CUDA;
    const DwShape s{rows, experts, out_features, in_features,
                    (out_features + 2 * kHalfM - 1) / (2 * kHalfM),
                    (in_features + 2 * kHalfM - 1) / (2 * kHalfM),
                    dw_stages(experts)};
    if (accumulate)
        return status_of(f16 ? launch_dw_t<true, true>(ta, tb, td, offsets, s, cs)
                             : launch_dw_t<true, false>(ta, tb, td, offsets, s, cs));
    return status_of(f16 ? launch_dw_t<false, true>(ta, tb, td, offsets, s, cs)
                         : launch_dw_t<false, false>(ta, tb, td, offsets, s, cs));
}

}  // extern "C"
