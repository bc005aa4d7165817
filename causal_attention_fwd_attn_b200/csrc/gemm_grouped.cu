// gemm_grouped.cu -- the three products of a linear layer, grouped by expert, on tcgen05
// tensor cores: the rows [o_e, o_{e+1}) of the token matrices belong to expert e, and the
// offsets are read on the device, so that a router's counts never visit the host.
//   forward   y  = x w_e^T       backward  dx = dy w_e,   dw_e (+)= dy_e^T x_e
//
// Forward and dX are one kernel (grouped_rows_kernel).  It computes the transposed product:
// the weights' features are the 128 rows of a tile and the expert's tokens its columns, so
// that the ragged dimension is the one whose width a tcgen05 product can vary (any
// multiple of 16): an expert's rows are cut into equal tiles of at most BN tokens and
// each product is as wide as its tile.  Rows of a neighbouring expert that the last copy of
// a tile brings along only feed columns that are never stored.
// dW (grouped_dw_kernel) reduces over an expert's tokens, 64 to a step.  In the last step
// the rows after the expert's end are cleared in shared memory, in both operands (a
// neighbour's row may hold infinities, which a zero in one operand would not remove).
//
// Both are persistent, one block per SM.  Every block reads the offsets into shared
// memory (each clamped to the rows there are, so that no offsets can lead outside the
// tensors) and walks the (expert, tile) units in one common order.
#include <cmath>

#include "forge_attn.h"
#include "forge_internal.h"
#include "forge_linear.h"
#include "sm100_grouped_ptx.cuh"
#include "sm100_ptx.cuh"

namespace forge {
namespace {

constexpr int kMaxExperts = FORGE_LINEAR_MAX_EXPERTS;
constexpr int kThreads = 192;
constexpr int kBM = 128, kBK = 64, kBN = 256;

enum : uint32_t { kSiteFull = 1, kSiteEmpty, kSiteAccFull, kSiteAccEmpty };

struct Barriers {
    uint64_t full[8], empty[8];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_final;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Barriers) <= 256, "barrier block");

// The experts' rows and units: first[e] the first row, unit0[e] the first unit.
struct Tables {
    int first[kMaxExperts + 1];
    int count[kMaxExperts];
    int unit0[kMaxExperts + 1];
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t site,
                                          volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, site, abort));
}

// Fills the tables: `units_of(rows)` units to an expert.  Called by the whole block; ends
// with a barrier.
template <typename F>
__device__ __forceinline__ void fill_tables(Tables* t, const int* offsets, int experts, int rows,
                                            F units_of) {
    for (int e = threadIdx.x; e <= experts; e += blockDim.x)
        t->first[e] = min(max(offsets[e], 0), rows);
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += blockDim.x)
        t->count[e] = max(t->first[e + 1] - t->first[e], 0);
    __syncthreads();
    if (warp_id() == 0) {
        int base = 0;
        for (int e0 = 0; e0 < experts; e0 += 32) {
            const int e = e0 + (int)lane_id();
            int u = e < experts ? units_of(t->count[e]) : 0;
            int sum = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int below = __shfl_up_sync(0xffffffffu, sum, o);
                if ((int)lane_id() >= o) sum += below;
            }
            if (e < experts) t->unit0[e] = base + sum - u;
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane_id() == 0) t->unit0[experts] = base;
    }
    __syncthreads();
}

// ------------------------------------------------------------------ forward and dX ----
constexpr int kRowsStages = 4;
constexpr int kRowsABytes = kBM * kBK * 2, kRowsBBytes = kBN * kBK * 2;
constexpr int kRowsStageBytes = kRowsABytes + kRowsBBytes;
constexpr int kStageRows = 32;  // token rows of one staging buffer of the epilogue
constexpr int kRowsStagingBytes = kStageRows * kBM * 4;
constexpr int kRowsOffStaging = kRowsStages * kRowsStageBytes;
constexpr int kRowsOffTables = kRowsOffStaging + kRowsStagingBytes;
constexpr int kRowsOffBar = kRowsOffTables + (int)((sizeof(Tables) + 127) / 128 * 128);
constexpr int kRowsSmem = kRowsOffBar + 256 + 1024;
static_assert(kRowsSmem <= 232448, "shared memory budget");

struct RowsShape {
    int rows, experts, features, k_blocks, feature_tiles;
};

// One unit: features [fm, fm + 128) of expert e for the token rows [r0, r0 + n).
struct RowsUnit {
    int e, fm, r0, n;
};
__device__ __forceinline__ RowsUnit rows_unit(const Tables* t, const RowsShape& s, int u, int& e) {
    while (u >= t->unit0[e + 1]) ++e;
    const int local = u - t->unit0[e], cnt = t->count[e];
    const int tiles = (cnt + kBN - 1) / kBN;
    const int f = local / tiles, tn = local - f * tiles;
    const int width = ((cnt + tiles - 1) / tiles + 15) / 16 * 16;
    return RowsUnit{e, f * kBM, t->first[e] + tn * width, min(width, cnt - tn * width)};
}

template <bool W_MN, bool OUT32, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_rows_kernel(const __grid_constant__ CUtensorMap tmap_w,
                        const __grid_constant__ CUtensorMap tmap_x,
                        const int* __restrict__ offsets, void* __restrict__ out, const RowsShape s) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Tables* tab = reinterpret_cast<Tables*>(smem + kRowsOffTables);
    Barriers* bars = reinterpret_cast<Barriers*>(smem + kRowsOffBar);
    volatile int* abort = &bars->abort;
    const uint32_t warp = warp_id(), lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRowsStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 4);
        }
        mbar_init(&bars->mma_final, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    const int ft = s.feature_tiles;
    fill_tables(tab, offsets, s.experts, s.rows,
                [ft](int n) { return (n + kBN - 1) / kBN * ft; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const int units = tab->unit0[s.experts];

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmap_w);
            tma_prefetch_desc(&tmap_x);
            int it = 0, e = 0;
            int last_use[kRowsStages];
            for (int i = 0; i < kRowsStages; ++i) last_use[i] = -1;
            bool run = true;
            for (int u = blockIdx.x; run && u < units; u += gridDim.x) {
                const RowsUnit w = rows_unit(tab, s, u, e);
                for (int kb = 0; kb < s.k_blocks; ++kb, ++it) {
                    const int st = it % kRowsStages, use = it / kRowsStages;
                    if (use > 0 && !mbar_wait(&bars->empty[st], (use - 1) & 1, kSiteEmpty, abort)) {
                        run = false;
                        break;
                    }
                    uint8_t* sa = smem + st * kRowsStageBytes;
                    mbar_arrive_expect_tx(&bars->full[st], kRowsStageBytes);
                    if constexpr (W_MN) {
                        for (int c = 0; c < kBM / 64; ++c)
                            tma_load_3d(sa + c * (kBK * 128), &tmap_w, &bars->full[st],
                                        w.fm + 64 * c, kb * kBK, w.e);
                    } else {
                        tma_load_3d(sa, &tmap_w, &bars->full[st], kb * kBK, w.fm, w.e);
                    }
                    tma_load_2d(sa + kRowsABytes, &tmap_x, &bars->full[st], kb * kBK, w.r0);
                    last_use[st] = use;
                }
            }
            if (*abort)
                for (int i = 0; i < kRowsStages; ++i)
                    if (last_use[i] >= 0) mbar_wait_drain(&bars->full[i], last_use[i] & 1);
        }
    } else if (warp == 1) {
        // --------------------------------------------------------- MMA issuer
        constexpr uint32_t kIdesc0 = idesc_f16kind_f32(kBM, 0, W_MN, false, F16);
        int it = 0, n_unit = 0, e = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++n_unit) {
            const RowsUnit w = rows_unit(tab, s, u, e);
            const int buf = n_unit & 1, use = n_unit >> 1;
            if (use > 0 &&
                !warp_wait(&bars->acc_empty[buf], (use - 1) & 1, kSiteAccEmpty, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem + buf * kBN;
            const uint32_t idesc = kIdesc0 | ((uint32_t)((w.n + 15) / 16 * 2) << 17);
            for (int kb = 0; kb < s.k_blocks; ++kb, ++it) {
                const int st = it % kRowsStages;
                if (!warp_wait(&bars->full[st], (it / kRowsStages) & 1, kSiteFull, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t a = smem_u32(smem + st * kRowsStageBytes), b = a + kRowsABytes;
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) {
                    const uint64_t ad = W_MN ? sdesc_sw128(a + kk * 2048, kBK * 128, 1024)
                                             : sdesc_sw128(a + kk * 32, 16, 1024);
                    mma_ss_warp(tacc, ad, sdesc_sw128(b + kk * 32, 16, 1024), idesc,
                                (kb > 0 || kk > 0) ? 1u : 0u);
                }
                mma_commit_warp(&bars->empty[st]);
            }
            if (ok) mma_commit_warp(&bars->acc_full[buf]);
        }
        mma_commit_warp(&bars->mma_final);
        mbar_wait_drain(&bars->mma_final, 0);
    } else {
        // ------------------------------------------------------------ epilogue
        // A thread reads its feature's accumulators 32 tokens at a time; the four warps
        // turn them into rows of 128 features in shared memory and store those whole.
        const uint32_t quarter = warp & 3;
        const uint32_t lane_off = (quarter * 32u) << 16;
        const int tid = (int)threadIdx.x - 64;
        constexpr int kEl = OUT32 ? 4 : 2, kRowBytes = kBM * kEl, kChunks = kRowBytes / 16;
        uint8_t* staging = smem + kRowsOffStaging;
        int n_unit = 0, e = 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x, ++n_unit) {
            const RowsUnit w = rows_unit(tab, s, u, e);
            const int buf = n_unit & 1, use = n_unit >> 1;
            // the four warps go on, or give up, together: they meet at barriers below
            if (!named_barrier_all(
                    1, 128, warp_wait(&bars->acc_full[buf], use & 1, kSiteAccFull, abort)))
                break;
            tc_fence_after();
            const int steps = (w.n + kStageRows - 1) / kStageRows;
            for (int c = 0; c < steps; ++c) {
                uint32_t r[32];
                tmem_ld32(tmem + lane_off + buf * kBN + c * kStageRows, r);
                tmem_wait_ld();
                if (c == steps - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->acc_empty[buf]);
                }
                named_barrier_sync(1, 128);  // the staging rows have been read
#pragma unroll
                for (int j = 0; j < kStageRows; ++j) {
                    uint8_t* dst = staging + j * kRowBytes + (quarter * 32 + lane) * kEl;
                    if constexpr (OUT32) *reinterpret_cast<uint32_t*>(dst) = r[j];
                    else
                        *reinterpret_cast<uint16_t*>(dst) =
                            (uint16_t)pack16x2<F16>(__uint_as_float(r[j]), 0.f);
                }
                named_barrier_sync(1, 128);
                const int live = min(kStageRows, w.n - c * kStageRows);
                for (int k = tid; k < live * kChunks; k += 128) {
                    const int row = k / kChunks, col = (k - row * kChunks) * (16 / kEl);
                    if (w.fm + col >= s.features) continue;
                    const uint4 v = *reinterpret_cast<const uint4*>(staging + k * 16);
                    const long long off =
                        (long long)(w.r0 + c * kStageRows + row) * s.features + w.fm + col;
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + off * kEl) = v;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------- dW ----
constexpr int kDwStages = 4;
constexpr int kDwABytes = kBM * kBK * 2, kDwBBytes = kBN * kBK * 2;
constexpr int kDwStageBytes = kDwABytes + kDwBBytes;
constexpr int kDwOffStaging = kDwStages * kDwStageBytes;
constexpr int kDwBoxBytes = 32 * 128;  // one warp's 32 x 32 fp32 box
constexpr int kDwOffTables = kDwOffStaging + 4 * kDwBoxBytes;
constexpr int kDwOffBar = kDwOffTables + (int)((sizeof(Tables) + 127) / 128 * 128);
constexpr int kDwSmem = kDwOffBar + 256 + 1024;
static_assert(kDwSmem <= 232448, "shared memory budget");

struct DwShape {
    int rows, experts, m, n, tiles_m, tiles_n;
};

struct DwUnit {
    int e, m0, n0, r0, count;
};
__device__ __forceinline__ DwUnit dw_unit(const Tables* t, const DwShape& s, int u, int& e) {
    while (u >= t->unit0[e + 1]) ++e;
    const int local = u - t->unit0[e];
    const int tn = local / s.tiles_m, tm = local - tn * s.tiles_m;
    return DwUnit{e, tm * kBM, tn * kBN, t->first[e], t->count[e]};
}

// Clears rows [valid, 64) of the 64-row chunks of a stage (each row is 128 bytes, whatever
// the swizzle does inside it).
__device__ __forceinline__ void clear_rows(uint8_t* stage, int chunks, int valid, uint32_t lane) {
    const int per = (kBK - valid) * 8;
    for (int k = lane; k < chunks * per; k += 32) {
        const int c = k / per, r = k - c * per;
        *reinterpret_cast<uint4*>(stage + c * (kBK * 128) + valid * 128 + r * 16) =
            make_uint4(0, 0, 0, 0);
    }
}

template <bool ADD, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_dw_kernel(const __grid_constant__ CUtensorMap tmap_dy,
                      const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ CUtensorMap tmap_dw,
                      const int* __restrict__ offsets, const DwShape s) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Tables* tab = reinterpret_cast<Tables*>(smem + kDwOffTables);
    Barriers* bars = reinterpret_cast<Barriers*>(smem + kDwOffBar);
    volatile int* abort = &bars->abort;
    const uint32_t warp = warp_id(), lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kDwStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 4);
        }
        mbar_init(&bars->mma_final, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    // an expert without rows has a zero gradient: written, or nothing to add
    const int per = s.tiles_m * s.tiles_n;
    fill_tables(tab, offsets, s.experts, s.rows,
                [per](int n) { return ADD && n == 0 ? 0 : per; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const int units = tab->unit0[s.experts];

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&tmap_dy);
            tma_prefetch_desc(&tmap_x);
            int it = 0, e = 0;
            int last_use[kDwStages];
            for (int i = 0; i < kDwStages; ++i) last_use[i] = -1;
            bool run = true;
            for (int u = blockIdx.x; run && u < units; u += gridDim.x) {
                const DwUnit w = dw_unit(tab, s, u, e);
                for (int k0 = 0; k0 < w.count; k0 += kBK, ++it) {
                    const int st = it % kDwStages, use = it / kDwStages;
                    if (use > 0 && !mbar_wait(&bars->empty[st], (use - 1) & 1, kSiteEmpty, abort)) {
                        run = false;
                        break;
                    }
                    uint8_t* sa = smem + st * kDwStageBytes;
                    mbar_arrive_expect_tx(&bars->full[st], kDwStageBytes);
                    for (int c = 0; c < kBM / 64; ++c)
                        tma_load_2d(sa + c * (kBK * 128), &tmap_dy, &bars->full[st],
                                    w.m0 + 64 * c, w.r0 + k0);
                    for (int c = 0; c < kBN / 64; ++c)
                        tma_load_2d(sa + kDwABytes + c * (kBK * 128), &tmap_x, &bars->full[st],
                                    w.n0 + 64 * c, w.r0 + k0);
                    last_use[st] = use;
                }
            }
            if (*abort)
                for (int i = 0; i < kDwStages; ++i)
                    if (last_use[i] >= 0) mbar_wait_drain(&bars->full[i], last_use[i] & 1);
        }
    } else if (warp == 1) {
        constexpr uint32_t kIdesc = idesc_f16kind_f32(kBM, kBN, true, true, F16);
        int it = 0, n_unit = 0, e = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const DwUnit w = dw_unit(tab, s, u, e);
            if (w.count == 0) continue;
            const int buf = n_unit & 1, use = n_unit >> 1;
            ++n_unit;
            if (use > 0 &&
                !warp_wait(&bars->acc_empty[buf], (use - 1) & 1, kSiteAccEmpty, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem + buf * kBN;
            for (int k0 = 0; k0 < w.count; k0 += kBK, ++it) {
                const int st = it % kDwStages;
                if (!warp_wait(&bars->full[st], (it / kDwStages) & 1, kSiteFull, abort)) {
                    ok = false;
                    break;
                }
                uint8_t* stage = smem + st * kDwStageBytes;
                if (w.count - k0 < kBK) {
                    clear_rows(stage, (kBM + kBN) / 64, w.count - k0, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                const uint32_t a = smem_u32(stage), b = a + kDwABytes;
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                    mma_ss_warp(tacc, sdesc_sw128(a + kk * 2048, kBK * 128, 1024),
                                sdesc_sw128(b + kk * 2048, kBK * 128, 1024), kIdesc,
                                (k0 > 0 || kk > 0) ? 1u : 0u);
                mma_commit_warp(&bars->empty[st]);
            }
            if (ok) mma_commit_warp(&bars->acc_full[buf]);
        }
        mma_commit_warp(&bars->mma_final);
        mbar_wait_drain(&bars->mma_final, 0);
    } else {
        // A warp stages its 32 rows 32 columns at a time (128-byte swizzle) and one lane
        // hands the box to the copy engine, which clips it at the expert's last row and
        // column and, when accumulating, adds it (one addition per element).
        const uint32_t quarter = warp & 3;
        const uint32_t lane_off = (quarter * 32u) << 16;
        uint8_t* box = smem + kDwOffStaging + quarter * kDwBoxBytes;
        int n_unit = 0, e = 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            const DwUnit w = dw_unit(tab, s, u, e);
            const bool empty = w.count == 0;
            const int buf = n_unit & 1, use = n_unit >> 1;
            if (!empty) {
                ++n_unit;
                if (!warp_wait(&bars->acc_full[buf], use & 1, kSiteAccFull, abort)) break;
                tc_fence_after();
            }
            const int row = w.m0 + (int)quarter * 32;
            for (int c = 0; c < kBN / 32; ++c) {
                uint32_t r[32];
                if (empty) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                } else {
                    tmem_ld32(tmem + lane_off + buf * kBN + c * 32, r);
                    tmem_wait_ld();
                    if (c == kBN / 32 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->acc_empty[buf]);
                    }
                }
                if (row >= s.m || w.n0 + 32 * c >= s.n) continue;
                if (lane == 0) tma_store_wait_all_read();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(box + sw128_offset(lane, j)) =
                        make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (ADD) tma_reduce_add_3d(&tmap_dw, box, w.n0 + 32 * c, row, w.e);
                    else tma_store_3d(&tmap_dw, box, w.n0 + 32 * c, row, w.e);
                    tma_store_commit();
                }
            }
        }
        if (lane == 0) tma_store_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------- host ----
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dims(int rows, int experts, int in_f, int out_f) {
    if (rows < 0 || experts < 1 || in_f < 1 || out_f < 1) return FORGE_ATTN_ERR_INVALID_ARG;
    if (experts > kMaxExperts || in_f % 8 || out_f % 8) return FORGE_ATTN_ERR_UNSUPPORTED;
    if ((long long)rows * in_f >= (1ll << 31) || (long long)rows * out_f >= (1ll << 31) ||
        (long long)out_f * in_f >= (1ll << 31))
        return FORGE_ATTN_ERR_UNSUPPORTED;
    return FORGE_ATTN_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? FORGE_ATTN_OK : FORGE_ATTN_ERR_CUDA; }

template <bool W_MN, bool OUT32, bool F16>
cudaError_t launch_rows_t(const CUtensorMap& tw, const CUtensorMap& tx, const int* offsets,
                          void* out, const RowsShape& s, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured{0};
    auto* kernel = grouped_rows_kernel<W_MN, OUT32, F16>;
    cudaError_t e = set_max_dynamic_smem(kernel, kRowsSmem, configured);
    if (e != cudaSuccess) return e;
    // units: at most one partly filled tile to an expert on top of the full ones
    const long long units = ((long long)s.rows / kBN + s.experts) * s.feature_tiles;
    const int grid = units < sm_count() ? (int)units : sm_count();
    kernel<<<grid, kThreads, kRowsSmem, stream>>>(tw, tx, offsets, out, s);
    return cudaGetLastError();
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
    CUtensorMap tw, tx;
    if (encode_map_3d(&tw, w, in_f, out_f, experts, 64, W_MN ? 64 : kBM, f16 ? kMapF16 : kMapBf16) !=
            cudaSuccess ||
        encode_map_2d16(&tx, x, k, rows, 64, kBN, f16) != cudaSuccess)
        return FORGE_ATTN_ERR_CUDA;
    const RowsShape s{rows, experts, features, (k + kBK - 1) / kBK, (features + kBM - 1) / kBM};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (f32)
        return status_of(f16 ? launch_rows_t<W_MN, true, true>(tw, tx, offsets, out, s, cs)
                             : launch_rows_t<W_MN, true, false>(tw, tx, offsets, out, s, cs));
    return status_of(f16 ? launch_rows_t<W_MN, false, true>(tw, tx, offsets, out, s, cs)
                         : launch_rows_t<W_MN, false, false>(tw, tx, offsets, out, s, cs));
}

template <bool ADD, bool F16>
cudaError_t launch_dw_t(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td,
                        const int* offsets, const DwShape& s, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured{0};
    auto* kernel = grouped_dw_kernel<ADD, F16>;
    cudaError_t e = set_max_dynamic_smem(kernel, kDwSmem, configured);
    if (e != cudaSuccess) return e;
    const long long units = (long long)s.experts * s.tiles_m * s.tiles_n;
    const int grid = units < sm_count() ? (int)units : sm_count();
    kernel<<<grid, kThreads, kDwSmem, stream>>>(ta, tb, td, offsets, s);
    return cudaGetLastError();
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
    const DwShape s{rows, experts, out_features, in_features, (out_features + kBM - 1) / kBM,
                    (in_features + kBN - 1) / kBN};
    if (accumulate)
        return status_of(f16 ? launch_dw_t<true, true>(ta, tb, td, offsets, s, cs)
                             : launch_dw_t<true, false>(ta, tb, td, offsets, s, cs));
    return status_of(f16 ? launch_dw_t<false, true>(ta, tb, td, offsets, s, cs)
                         : launch_dw_t<false, false>(ta, tb, td, offsets, s, cs));
}

}  // extern "C"
