// grad.cu -- the global norm of many gradient tensors, and their clipping at it.
//
//   norm = sqrt(sum over tensors and elements of g^2),  c = max_norm / norm if
//   norm > max_norm, else 1,  out = c g
// over fp32, bf16 and fp16 tensors mixed.  The Forge paper folds this factor into the
// optimizer's read of the gradient (section "Training details"), as forge_adamw_step
// does; the entry points here are for gradients that another consumer reads, and for
// 16-bit ones.
//
// Both passes are bound by HBM: every value is read for the norm, and read and written
// to be scaled (124.4M fp32 values: 76 us at 6.6 TB/s, and 168 us at 5.9; 246 together).  As in the AdamW step the tensor table travels in the kernel parameters
// and the blocks of one grid walk fixed chunks of all tensors.  The norm pass leaves one
// 64-bit partial per block; every block of the clip pass adds all of them itself, in the
// same order, so that no counter, atomic or third launch is needed and the result does
// not depend on which block ends last.  The clip pass walks the chunks backwards: what
// the norm pass read last is still in L2.
//
// Squares are summed in fp32 within a thread's share of a chunk (at most 128 values) and
// in fp64 from there on.  A share whose fp32 sum left the range where that is exact enough
// (above 2^120, or below 2^-80 with a value that is not zero) is summed again in fp64.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "forge_adamw.h"
#include "forge_attn.h"
#include "forge_internal.h"
#include "sm100_ptx.cuh"

namespace forge {
namespace {

constexpr int kThreads = 512;
constexpr int kBlocksPerSm = 2;
constexpr int kMaxPerLaunch = FORGE_ADAMW_MAX_TENSORS_PER_LAUNCH;
// Elements per chunk: a power of two between these, so that small sets still give every
// block a chunk and large ones walk long contiguous runs.
constexpr int kMinChunk = 1 << 12, kMaxChunk = 1 << 16;

struct Table {
    const void* grad[kMaxPerLaunch];
    void* out[kMaxPerLaunch];
    long long n[kMaxPerLaunch];
    int chunk0[kMaxPerLaunch + 1];  // first chunk of each tensor; chunk0[count] = all
    unsigned char dtype[kMaxPerLaunch];
    int count, chunk;
};
static_assert(sizeof(Table) < 16384, "kernel parameter space");

__device__ __forceinline__ int tensor_of(const Table& t, int c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {  // last tensor whose first chunk is <= c
        const int mid = (lo + hi + 1) >> 1;
        if (t.chunk0[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Sum over the block, valid in every thread.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double red[kThreads / 32];
    __shared__ double total;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane_id() == 0) red[warp_id()] = x;
    __syncthreads();
    if (warp_id() == 0) {
        x = lane_id() < kThreads / 32 ? red[lane_id()] : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane_id() == 0) total = x;
    }
    __syncthreads();
    return total;
}

// A 16-byte load as floats: 4 of fp32, 8 of bf16 or fp16.
template <int DT>
__device__ __forceinline__ void values(const uint4& u, float* f) {
    if constexpr (DT == FORGE_GRAD_F32) {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = unpack16x2<DT == FORGE_GRAD_F16>(w[j]);
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
        }
    }
}
template <int DT>
__device__ __forceinline__ float value(const void* p, long long e) {
    if constexpr (DT == FORGE_GRAD_F32) return static_cast<const float*>(p)[e];
    if constexpr (DT == FORGE_GRAD_BF16)
        return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[e] << 16);
    return __half2float(static_cast<const __half*>(p)[e]);
}

template <int DT>
constexpr int kPer = DT == FORGE_GRAD_F32 ? 4 : 8;  // values of a 16-byte load

constexpr int kFly = 8;  // 16-byte loads a thread has in flight

// Sum of squares of elements [e0, e1) over the thread's share of them.  KEEP: leave them in L2
// for the clip pass.
template <int DT, bool KEEP>
__device__ __forceinline__ double chunk_squares(const void* g, long long e0, long long e1) {
    constexpr int P = kPer<DT>;
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(g) + e0 * (16 / P));
    const int n = (int)((e1 - e0) / P);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t any = 0;
    auto take = [&](const uint4& u, float& a) {
        any |= u.x | u.y | u.z | u.w;
        float f[P];
        values<DT>(u, f);
#pragma unroll
        for (int j = 0; j < P; ++j) a = fmaf(f[j], f[j], a);
    };
    int k = threadIdx.x;
    for (; k + (kFly - 1) * kThreads < n; k += kFly * kThreads) {
        uint4 u[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j)
            u[j] = KEEP ? v[k + j * kThreads] : __ldcs(v + k + j * kThreads);
#pragma unroll
        for (int j = 0; j < kFly; ++j) take(u[j], acc[j % 4]);
    }
    for (; k < n; k += kThreads) take(v[k], acc[0]);
    float tail = 0.f;
    const long long e = e0 + (long long)n * P + threadIdx.x;
    if (e < e1) {
        tail = value<DT>(g, e);
        any |= __float_as_uint(tail);
        acc[0] = fmaf(tail, tail, acc[0]);
    }
    const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    any &= DT == FORGE_GRAD_F32 ? 0x7fffffffu : 0x7fff7fffu;
    // fine: every square that matters is a normal number and nothing overflowed (a NaN
    // fails both comparisons and stays one below)
    if ((sum >= 0x1p-80f && sum <= 0x1p120f) || any == 0) return (double)sum;
    double s = (double)tail * (double)tail;
    for (int q = threadIdx.x; q < n; q += kThreads) {
        float f[P];
        values<DT>(v[q], f);
#pragma unroll
        for (int j = 0; j < P; ++j) s = fma((double)f[j], (double)f[j], s);
    }
    return s;
}

template <bool KEEP>
__device__ __forceinline__ double squares(int dtype, const void* g, long long e0, long long e1) {
    if (dtype == FORGE_GRAD_F32) return chunk_squares<FORGE_GRAD_F32, KEEP>(g, e0, e1);
    if (dtype == FORGE_GRAD_BF16) return chunk_squares<FORGE_GRAD_BF16, KEEP>(g, e0, e1);
    return chunk_squares<FORGE_GRAD_F16, KEEP>(g, e0, e1);
}

// Chunks from `keep` on stay in L2.
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_norm_kernel(const __grid_constant__ Table t, double* partials, int keep) {
    allow_dependents_launch();
    grid_dependency_wait();
    const int chunks = t.chunk0[t.count];
    double sum = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const long long e0 = (long long)(c - t.chunk0[i]) * t.chunk;
        const long long e1 = min(e0 + t.chunk, t.n[i]);
        sum += c >= keep ? squares<true>(t.dtype[i], t.grad[i], e0, e1)
                         : squares<false>(t.dtype[i], t.grad[i], e0, e1);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) partials[blockIdx.x] = sum;
}

// The norm of all partials, the same in every thread of every block.
__device__ __forceinline__ double norm_of(const double* partials, int n) {
    double x = 0.0;
    for (int k = threadIdx.x; k < n; k += kThreads) x += partials[k];
    return sqrt(block_sum(x));
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_sum_kernel(const double* partials, int n, float* norm_out) {
    allow_dependents_launch();
    grid_dependency_wait();
    const double norm = norm_of(partials, n);
    if (threadIdx.x == 0) *norm_out = (float)norm;
}

// out = c g over elements [e0, e1).  In 16-bit types the product is rounded once, to
// nearest; c = 1 copies the values.  F: c in fp32, or in 64 bits where fp32 has no normal number
// for it while the products may well be ordinary ones.
template <int DT, typename F>
__device__ __forceinline__ void chunk_scale(const void* g, void* out, long long e0, long long e1,
                                            F c) {
    constexpr int P = kPer<DT>;
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(g) + e0 * (16 / P));
    uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(out) + e0 * (16 / P));
    const int n = (int)((e1 - e0) / P);
    auto put = [&](int k, const uint4& u) {
        float f[P];
        values<DT>(u, f);
#pragma unroll
        for (int j = 0; j < P; ++j) f[j] = (float)(f[j] * c);
        uint4 r;
        if constexpr (DT == FORGE_GRAD_F32) {
            r = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                           __float_as_uint(f[3]));
        } else {
            constexpr bool F16 = DT == FORGE_GRAD_F16;
            r = make_uint4(pack16x2<F16>(f[0], f[1]), pack16x2<F16>(f[2], f[3]),
                           pack16x2<F16>(f[4], f[5]), pack16x2<F16>(f[6], f[7]));
        }
        __stcs(o + k, r);  // (not kept in L2: what the norm pass left there is still needed)
    };
    int k = threadIdx.x;
    for (; k + (kFly - 1) * kThreads < n; k += kFly * kThreads) {
        uint4 u[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j) u[j] = __ldcs(v + k + j * kThreads);
#pragma unroll
        for (int j = 0; j < kFly; ++j) put(k + j * kThreads, u[j]);
    }
    for (; k < n; k += kThreads) put(k, __ldcs(v + k));
    const long long e = e0 + (long long)n * P + threadIdx.x;
    if (e < e1) {
        const float r = (float)(value<DT>(g, e) * c);
        if constexpr (DT == FORGE_GRAD_F32) static_cast<float*>(out)[e] = r;
        else if constexpr (DT == FORGE_GRAD_BF16)
            static_cast<__nv_bfloat16*>(out)[e] = __float2bfloat16_rn(r);
        else static_cast<__half*>(out)[e] = __float2half_rn(r);
    }
}

template <typename F>
__device__ __forceinline__ void scale(int dtype, const void* g, void* out, long long e0, long long e1,
                                      F c) {
    if (dtype == FORGE_GRAD_F32) chunk_scale<FORGE_GRAD_F32>(g, out, e0, e1, c);
    else if (dtype == FORGE_GRAD_BF16) chunk_scale<FORGE_GRAD_BF16>(g, out, e0, e1, c);
    else chunk_scale<FORGE_GRAD_F16>(g, out, e0, e1, c);
}

__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_clip_kernel(const __grid_constant__ Table t, const double* partials, int n,
                     float max_norm, float* norm_out) {
    allow_dependents_launch();
    grid_dependency_wait();
    const double norm = norm_of(partials, n);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    const double wide = norm > (double)max_norm ? (double)max_norm / norm : 1.0;
    const float c = (float)wide;
    const bool tiny = wide < 0x1p-126 && wide > 0.0;  // (an infinite norm makes it 0)
    for (int ch = t.chunk0[t.count] - 1 - (int)blockIdx.x; ch >= 0; ch -= (int)gridDim.x) {
        const int i = tensor_of(t, ch);
        if (c == 1.f && t.out[i] == t.grad[i]) continue;  // nothing to change in place
        const long long e0 = (long long)(ch - t.chunk0[i]) * t.chunk;
        const long long e1 = min(e0 + t.chunk, t.n[i]);
        if (tiny) scale(t.dtype[i], t.grad[i], t.out[i], e0, e1, wide);
        else scale(t.dtype[i], t.grad[i], t.out[i], e0, e1, c);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_tensors(const forge_grad_tensor* tensors, int n_tensors, bool clip) {
    if (!tensors || n_tensors < 1) return FORGE_ATTN_ERR_INVALID_ARG;
    for (int k = 0; k < n_tensors; ++k) {
        const forge_grad_tensor& x = tensors[k];
        if (x.n < 0 || x.dtype < FORGE_GRAD_F32 || x.dtype > FORGE_GRAD_F16)
            return FORGE_ATTN_ERR_INVALID_ARG;
        if (x.n == 0) continue;
        if (x.n > (1ll << 44)) return FORGE_ATTN_ERR_UNSUPPORTED;
        if (!x.grad || (clip && !x.out)) return FORGE_ATTN_ERR_INVALID_ARG;
        if (!aligned16(x.grad) || (clip && !aligned16(x.out))) return FORGE_ATTN_ERR_MISALIGNED;
        if (clip && x.out != x.grad) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(x.grad),
                            b = reinterpret_cast<uintptr_t>(x.out);
            const uintptr_t bytes = (uintptr_t)x.n * (x.dtype == FORGE_GRAD_F32 ? 4 : 2);
            if (a < b + bytes && b < a + bytes) return FORGE_ATTN_ERR_INVALID_ARG;
        }
    }
    return FORGE_ATTN_OK;
}

// First chunk of a launch's table whose values are to stay in L2 for the clip pass, which
// walks the chunks backwards: the last kKeepBytes (of 126 MB of L2).  124.4M fp32 values took
// 244 us this way, 249 with everything streamed and 251 with everything kept.
constexpr long long kKeepBytes = 80ll << 20;
int first_kept(const Table& t) {
    long long bytes = 0;
    int c = t.chunk0[t.count];
    for (int k = t.count - 1; k >= 0 && bytes < kKeepBytes; --k) {
        const long long chunk = (long long)t.chunk * (t.dtype[k] == FORGE_GRAD_F32 ? 4 : 2);
        const long long want = (kKeepBytes - bytes + chunk - 1) / chunk;
        const int n = t.chunk0[k + 1] - t.chunk0[k];
        const int take = n < want ? n : (int)want;
        c -= take;
        bytes += take * chunk;
    }
    return c;
}

// Chunk size of a set: about four chunks to a block, within the limits.
int chunk_for(const forge_grad_tensor* tensors, int n_tensors) {
    long long all = 0;
    for (int k = 0; k < n_tensors; ++k) all += tensors[k].n;
    const long long want = all / (4ll * kBlocksPerSm * sm_count());
    int c = kMinChunk;
    while (c < kMaxChunk && c < want) c *= 2;
    return c;
}

int fill(Table* t, const forge_grad_tensor* tensors, int first, int count, int chunk) {
    t->count = count;
    t->chunk = chunk;
    long long chunks = 0;
    for (int k = 0; k < count; ++k) {
        const forge_grad_tensor& x = tensors[first + k];
        t->grad[k] = x.grad;
        t->out[k] = x.out;
        t->n[k] = x.n;
        t->dtype[k] = (unsigned char)x.dtype;
        t->chunk0[k] = (int)chunks;
        chunks += (x.n + chunk - 1) / chunk;
        if (chunks > 0x3fffffff) return FORGE_ATTN_ERR_UNSUPPORTED;
    }
    t->chunk0[count] = (int)chunks;
    return FORGE_ATTN_OK;
}

int grid_for(const Table& t) {
    const int chunks = t.chunk0[t.count], cap = kBlocksPerSm * sm_count();
    return chunks < 1 ? 1 : (chunks < cap ? chunks : cap);
}

// Norm pass, then the clip pass (clip) or the norm alone.  One launch of each per
// kMaxPerLaunch tensors.
int run(const forge_grad_tensor* tensors, int n_tensors, bool clip, float max_norm,
        float* norm_out, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_tensors(tensors, n_tensors, clip);
    if (st != FORGE_ATTN_OK) return st;
    if (!workspace || workspace_bytes < forge_grad_workspace_size(n_tensors))
        return FORGE_ATTN_ERR_WORKSPACE;
    if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(norm_out) & 3u))
        return FORGE_ATTN_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    double* partials = static_cast<double*>(workspace);
    const int chunk = chunk_for(tensors, n_tensors);
    Table t;  // the parameters are copied at launch
    for (int first = 0; first < n_tensors; first += kMaxPerLaunch)  // before any launch
        if ((st = fill(&t, tensors, first, n_tensors - first < kMaxPerLaunch ? n_tensors - first
                                                                             : kMaxPerLaunch,
                       chunk)) != FORGE_ATTN_OK)
            return st;
    cudaError_t e = cudaSuccess;
    int parts = 0;
    for (int pass = 0; pass < (clip ? 2 : 1); ++pass)
        for (int first = 0; first < n_tensors && e == cudaSuccess; first += kMaxPerLaunch) {
            const int count = n_tensors - first < kMaxPerLaunch ? n_tensors - first : kMaxPerLaunch;
            if (n_tensors > kMaxPerLaunch) fill(&t, tensors, first, count, chunk);
            const int grid = grid_for(t);
            if (pass == 0) {
                e = launch_dependent(grad_norm_kernel, dim3(grid), dim3(kThreads), 0, s, t,
                                     partials + parts, clip ? first_kept(t) : t.chunk0[t.count]);
                parts += grid;
            } else {
                e = launch_dependent(grad_clip_kernel, dim3(grid), dim3(kThreads), 0, s, t,
                                     (const double*)partials, parts, max_norm,
                                     first == 0 ? norm_out : (float*)nullptr);
            }
        }
    if (!clip && e == cudaSuccess) {
        e = launch_dependent(grad_norm_sum_kernel, dim3(1), dim3(kThreads), 0, s,
                             (const double*)partials, parts, norm_out);
    }
    return e == cudaSuccess ? FORGE_ATTN_OK : FORGE_ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

size_t forge_grad_workspace_size(int n_tensors) {
    if (n_tensors < 1) return 0;
    const size_t launches = ((size_t)n_tensors + kMaxPerLaunch - 1) / kMaxPerLaunch;
    // a launch has at most two blocks to an SM; 1024 SMs is far beyond any part
    return launches * kBlocksPerSm * 1024 * sizeof(double);
}

int forge_grad_norm(const forge_grad_tensor* tensors, int n_tensors, float* norm_out,
                    void* workspace, size_t workspace_bytes, void* stream) {
    if (!norm_out) return FORGE_ATTN_ERR_INVALID_ARG;
    return run(tensors, n_tensors, false, 0.f, norm_out, workspace, workspace_bytes, stream);
}

int forge_grad_clip(const forge_grad_tensor* tensors, int n_tensors, float max_norm,
                    float* norm_out, void* workspace, size_t workspace_bytes, void* stream) {
    if (!std::isfinite(max_norm) || max_norm <= 0.f) return FORGE_ATTN_ERR_INVALID_ARG;
    return run(tensors, n_tensors, true, max_norm, norm_out, workspace, workspace_bytes, stream);
}

}  // extern "C"
