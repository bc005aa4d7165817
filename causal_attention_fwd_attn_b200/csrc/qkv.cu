// qkv.cu -- the stage between the QKV projection and the attention: per-head RMS norm of
// queries and keys, rotary positions (one or several axes) and the change of layout from
// the projection's token-major rows to the attention's [B][H][T][d], in one pass each way.
//
// Forward, per token and head of q and k (v is only moved):
//   r = 1 / sqrt(mean_i x_i^2 + eps),  n = r x o w       (no weight: n = x)
//   the pair (a, b) of frequency j:  phi = pos[axis_j] f_j,
//   (a, b) -> (a cos phi - b sin phi, a sin phi + b cos phi)
// and key / value head g goes to the attention's heads [g H / Hkv, (g + 1) H / Hkv).
// Backward, with g = the rotation's inverse on the sum of dy over the shared heads:
//   dw += g o (r x),  u = g o w,  dx = r (u - r x mean(u o r x))
//
// Bound by HBM: each value is read once and written once (a shared head is written once
// for each of its copies).  D / 16 threads hold a head of a token, 16 values each: two
// 16-byte chunks placed so that both members of every rotated pair are in one thread.
// A block takes 8 consecutive tokens and a run of heads, computes the tokens' sines and
// cosines once into shared memory, and keeps a thread at its token, so that the angles
// stay in registers while it walks the heads.  Angles are reduced in 64 bits (turns =
// position * f / 2 pi, minus the nearest integer): a 32-bit product would lose the phase
// of far positions altogether.
#include <cmath>

#include "forge_attn.h"
#include "forge_internal.h"
#include "sm100_ptx.cuh"

namespace forge {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 8;   // tokens per block
constexpr int kUnroll = 4;  // head rows a thread has in flight

struct Rope {
    const double* freq;  // [pairs]
    const int* pos;      // [axes][B * T], or null: the token's index t
    const int* axis;     // [pairs], or null: axis 0
    int pairs, axes, adjacent;
};

// One of q, k, v: `heads` heads in the projection's layout, each going to `rep` heads of
// the attention's.
struct Part {
    const void* x;  // projection side (forward: source; backward: source of the norm)
    void* y;        // forward: attention side; backward: gradient, projection side
    const void* g;  // backward: gradient, attention side
    const float* w;
    long long sb, st, sh;     // strides of x, in elements
    long long gsb, gst, gsh;  // backward: strides of y
    int heads, rep;
};

struct Parts {
    Part part[3];  // q, k, v
};

struct Shape {
    int B, T, H;
    long long tokens;
    float eps;
};

template <int D>
struct Cfg {
    static constexpr int kLanes = D / 16;              // threads of a head row
    static constexpr int kGroups = kThreads / kLanes;  // rows at a time
    static constexpr int kSlots = kGroups / kTok;      // heads at a time
};

// First elements of the two 8-element chunks of thread i of a row: the halves of the
// same eight pairs while those last, then neighbours (elements that are not rotated).
__device__ __forceinline__ void chunks_of(int i, const Rope& r, int& a, int& b) {
    const int half = r.pairs >> 3;
    if (r.adjacent) {
        a = 16 * i;
        b = a + 8;
    } else if (i < half) {
        a = 8 * i;
        b = a + r.pairs;
    } else {
        a = 16 * i;
        b = a + 8;
    }
}

// (cos, sin) of the block's tokens and all pairs, [kTok][pairs].
__device__ __forceinline__ void fill_angles(const Rope& r, const Shape& s, long long tok0,
                                            float2* cs) {
    const int n = kTok * r.pairs;
    for (int k = threadIdx.x; k < n; k += kThreads) {
        const int t = k / r.pairs, j = k - t * r.pairs;
        const long long tok = tok0 + t;
        if (tok >= s.tokens) break;
        const int ax = r.axis ? min(max(r.axis[j], 0), r.axes - 1) : 0;
        const int p = r.pos ? r.pos[ax * s.tokens + tok] : (int)(tok % s.T);
        double turns = (double)p * (r.freq[j] * 0.15915494309189533577);
        turns -= rint(turns);
        float sn, c;
        sincospif(2.f * (float)turns, &sn, &c);
        cs[k] = make_float2(c, sn);
    }
}

// The (cos, sin) of the thread's pairs; returns how many of its eight there are.
__device__ __forceinline__ int load_angles(const Rope& r, const float2* cs, int t, int i,
                                           float2* c8) {
    const int n = min(max(r.pairs - 8 * i, 0), 8);
    const float2* p = cs + t * r.pairs + 8 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) c8[j] = p[j];
    return n;
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = unpack16x2<F16>(w[j]);
        f[2 * j] = p.x;
        f[2 * j + 1] = p.y;
    }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack16x2<F16>(f[0], f[1]), pack16x2<F16>(f[2], f[3]),
                      pack16x2<F16>(f[4], f[5]), pack16x2<F16>(f[6], f[7]));
}

// Rotates the thread's first n pairs (inverse: by -phi); the other values stay as they are.
template <bool INVERSE>
__device__ __forceinline__ void rotate(float* x, const float2* c8, int n, int adjacent) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= n) break;
        const float c = c8[j].x, s = INVERSE ? -c8[j].y : c8[j].y;
        if (adjacent) {
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = a * c - b * s;
            x[2 * j + 1] = a * s + b * c;
        } else {
            const float a = x[j], b = x[8 + j];
            x[j] = a * c - b * s;
            x[8 + j] = a * s + b * c;
        }
    }
}

// Sum over the threads of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A block to each (token tile, run of heads); runs of `per` heads of q, then k, then v.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads)
    qkv_fwd_kernel(const __grid_constant__ Parts parts, const Rope rope, const Shape s, int nq, int nk,
                   int runs, int per) {
    using C = Cfg<D>;
    __shared__ float2 cs[kTok * D / 2];
    const int tile = (int)(blockIdx.x / (unsigned)runs);
    int run = (int)(blockIdx.x % (unsigned)runs);
    const int kind = run < nq ? 0 : (run < nq + nk ? 1 : 2);
    const Part& p = parts.part[kind];
    run -= kind == 0 ? 0 : (kind == 1 ? nq : nq + nk);
    const long long tok0 = (long long)tile * kTok;
    const int i = threadIdx.x % C::kLanes, g = threadIdx.x / C::kLanes;
    const int t = g % kTok, slot = g / kTok;
    const long long tok = tok0 + t;
    const bool live = tok < s.tokens;
    const bool turn = kind < 2 && rope.pairs > 0;
    int ea, eb;
    chunks_of(i, rope, ea, eb);
    const long long b = tok / s.T, tt = tok - b * s.T;
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + b * p.sb + tt * p.st;
    uint16_t* y = static_cast<uint16_t*>(p.y) + (b * s.H * s.T + tt) * D;
    if (turn) fill_angles(rope, s, tok0, cs);
    float2 c8[8];
    float w[16];
    if (kind < 2 && p.w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = p.w[ea + j];
            w[8 + j] = p.w[eb + j];
        }
    }
    __syncthreads();
    const int n8 = turn ? load_angles(rope, cs, t, i, c8) : 0;
    const int h1 = min((run + 1) * per, p.heads);
    for (int h0 = run * per + slot; h0 - slot < h1; h0 += C::kSlots * kUnroll) {
        uint4 in[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * C::kSlots;
            in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
            if (live && h < h1) {
                in[u][0] = __ldg(reinterpret_cast<const uint4*>(x + h * p.sh + ea));
                in[u][1] = __ldg(reinterpret_cast<const uint4*>(x + h * p.sh + eb));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * C::kSlots;
            uint4 oa = in[u][0], ob = in[u][1];
            if (kind < 2) {
                float f[16];
                unpack8<F16>(oa, f);
                unpack8<F16>(ob, f + 8);
                if (p.w) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) ss = fmaf(f[j], f[j], ss);
                    const float r = rsqrtf(row_sum<C::kLanes>(ss) * (1.f / D) + s.eps);
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[j] = f[j] * r * w[j];
                }
                if (turn) rotate<false>(f, c8, n8, rope.adjacent);
                oa = pack8<F16>(f);
                ob = pack8<F16>(f + 8);
            }
            if (live && h < h1) {
                for (int c = 0; c < p.rep; ++c) {
                    uint16_t* o = y + (long long)(h * p.rep + c) * s.T * D;
                    *reinterpret_cast<uint4*>(o + ea) = oa;
                    *reinterpret_cast<uint4*>(o + eb) = ob;
                }
            }
        }
    }
}

// The thread's 16 gradients of a row on the attention's side, in 32 bits.
template <bool F16, bool G32>
__device__ __forceinline__ void add_grad(const void* g, long long off, int ea, int eb, float* f) {
    if constexpr (G32) {
        const float* p = static_cast<const float*>(g) + off;
        const float4 v[4] = {__ldg(reinterpret_cast<const float4*>(p + ea)),
                             __ldg(reinterpret_cast<const float4*>(p + ea) + 1),
                             __ldg(reinterpret_cast<const float4*>(p + eb)),
                             __ldg(reinterpret_cast<const float4*>(p + eb) + 1)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[4 * j] += v[j].x;
            f[4 * j + 1] += v[j].y;
            f[4 * j + 2] += v[j].z;
            f[4 * j + 3] += v[j].w;
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(g) + off;
        float a[16];
        unpack8<F16>(__ldg(reinterpret_cast<const uint4*>(p + ea)), a);
        unpack8<F16>(__ldg(reinterpret_cast<const uint4*>(p + eb)), a + 8);
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] += a[j];
    }
}

// Blocks [0, nq) walk q's (token tile, run of heads) units, the next nk k's, the rest v's.
// Each block of q and k sums its share of the norm weight's gradient in registers and
// writes it to partials[block][D].
template <int D, bool F16, bool G32>
__global__ void __launch_bounds__(kThreads)
    qkv_bwd_kernel(const __grid_constant__ Parts parts, const Rope rope, const Shape s, int nq, int nk,
                   int per, float* __restrict__ partials) {
    using C = Cfg<D>;
    __shared__ float2 cs[kTok * D / 2];
    int blk = blockIdx.x;
    const int kind = blk < nq ? 0 : (blk < nq + nk ? 1 : 2);
    const Part& p = parts.part[kind];
    blk -= kind == 0 ? 0 : (kind == 1 ? nq : nq + nk);
    const int blocks = kind == 0 ? nq : (kind == 1 ? nk : (int)gridDim.x - nq - nk);
    const int i = threadIdx.x % C::kLanes, g = threadIdx.x / C::kLanes;
    const int t = g % kTok, slot = g / kTok;
    const bool turn = kind < 2 && rope.pairs > 0;
    const bool norm = kind < 2 && p.w != nullptr;
    int ea, eb;
    chunks_of(i, rope, ea, eb);
    float w[16], dw[16];
    if (norm) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = p.w[ea + j];
            w[8 + j] = p.w[eb + j];
        }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) dw[j] = 0.f;
    const int runs = (p.heads + per - 1) / per;
    const long long tiles = (s.tokens + kTok - 1) / kTok;
    for (long long unit = blk; unit < tiles * runs; unit += blocks) {
        const long long tok0 = unit / runs * kTok;
        const int run = (int)(unit % runs);
        const long long tok = tok0 + t;
        const bool live = tok < s.tokens;
        const long long b = tok / s.T, tt = tok - b * s.T;
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + b * p.sb + tt * p.st;
        uint16_t* y = static_cast<uint16_t*>(p.y) + b * p.gsb + tt * p.gst;
        const long long grow = (b * s.H * s.T + tt) * D;
        float2 c8[8];
        int n8 = 0;
        if (turn) {
            __syncthreads();  // the previous unit's angles have been read
            fill_angles(rope, s, tok0, cs);
            __syncthreads();
            n8 = load_angles(rope, cs, t, i, c8);
        }
        const int h1 = min((run + 1) * per, p.heads);
        for (int h0 = run * per + slot; h0 - slot < h1; h0 += C::kSlots) {
            const bool on = live && h0 < h1;
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = 0.f;
            uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
            if (on) {
                if (norm) {
                    xa = __ldg(reinterpret_cast<const uint4*>(x + h0 * p.sh + ea));
                    xb = __ldg(reinterpret_cast<const uint4*>(x + h0 * p.sh + eb));
                }
                for (int c = 0; c < p.rep; ++c)
                    add_grad<F16, G32>(p.g, grow + (long long)(h0 * p.rep + c) * s.T * D, ea, eb, f);
            }
            if (turn) rotate<true>(f, c8, n8, rope.adjacent);
            if (norm) {
                float n[16];
                unpack8<F16>(xa, n);
                unpack8<F16>(xb, n + 8);
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    ss = fmaf(n[j], n[j], ss);
                    dot = fmaf(f[j] * w[j], n[j], dot);
                }
                const float r = rsqrtf(row_sum<C::kLanes>(ss) * (1.f / D) + s.eps);
                const float m = row_sum<C::kLanes>(dot) * r * (1.f / D);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    n[j] *= r;
                    dw[j] = fmaf(f[j], n[j], dw[j]);
                    f[j] = r * (f[j] * w[j] - n[j] * m);
                }
            }
            if (on) {
                *reinterpret_cast<uint4*>(y + h0 * p.gsh + ea) = pack8<F16>(f);
                *reinterpret_cast<uint4*>(y + h0 * p.gsh + eb) = pack8<F16>(f + 8);
            }
        }
    }
    if (norm) {
        // the block's sum, always added in the same order
        __shared__ float red[kThreads / 32][D];
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int o = C::kLanes; o < 32; o <<= 1)
                dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
        if ((threadIdx.x & 31) < C::kLanes) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                red[threadIdx.x >> 5][ea + j] = dw[j];
                red[threadIdx.x >> 5][eb + j] = dw[8 + j];
            }
        }
        __syncthreads();
        if (threadIdx.x < D) {
            float sum = 0.f;
#pragma unroll
            for (int wv = 0; wv < kThreads / 32; ++wv) sum += red[wv][threadIdx.x];
            partials[(long long)blockIdx.x * D + threadIdx.x] = sum;
        }
    }
}

// dw (+)= sum of the blocks' partials, in 64 bits and in a fixed order.  Block x: eight
// elements; block y: q or k (partials [first, first + n)).
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(8 * kSumRows)
    qkv_dw_kernel(const float* __restrict__ partials, float* dwq, float* dwk, int nq, int nk, int D,
                  int accumulate) {
    float* out = blockIdx.y == 0 ? dwq : dwk;
    if (!out) return;
    const int first = blockIdx.y == 0 ? 0 : nq, n = blockIdx.y == 0 ? nq : nk;
    const int col = threadIdx.x & 7, row = threadIdx.x >> 3;
    const int e = blockIdx.x * 8 + col;
    double sum = 0.0;
    for (int k = row; k < n; k += kSumRows) sum += (double)partials[(long long)(first + k) * D + e];
    __shared__ double red[kSumRows][8];
    red[row][col] = sum;
    __syncthreads();
    if (row == 0) {
        for (int k = 1; k < kSumRows; ++k) sum += red[k][col];
        out[e] = accumulate ? (float)((double)out[e] + sum) : (float)sum;
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A gradient tensor's rows must not overlap: each stride (of a dimension longer than one)
// at least the extent of the dimensions inside it.
bool distinct(const forge_qkv_tensor& t, int B, int T, int heads, int d) {
    long long size[3] = {B, T, heads}, stride[3] = {t.stride_b, t.stride_t, t.stride_h};
    long long extent = d;
    bool used[3] = {size[0] == 1, size[1] == 1, size[2] == 1};
    for (int round = 0; round < 3; ++round) {
        int best = -1;
        for (int j = 0; j < 3; ++j)
            if (!used[j] && (best < 0 || stride[j] < stride[best])) best = j;
        if (best < 0) break;
        if (stride[best] < extent) return false;
        extent = stride[best] * (size[best] - 1) + extent;
        used[best] = true;
    }
    return true;
}

// Strides of dimensions of size one are never used, and may be anything.
int check_strides(const forge_qkv_tensor& t, int B, int T, int heads) {
    if (!t.data) return FORGE_ATTN_ERR_INVALID_ARG;
    const long long size[3] = {B, T, heads}, stride[3] = {t.stride_b, t.stride_t, t.stride_h};
    for (int j = 0; j < 3; ++j) {
        if (size[j] == 1) continue;
        if (stride[j] < 0) return FORGE_ATTN_ERR_INVALID_ARG;
        if (stride[j] % 8) return FORGE_ATTN_ERR_MISALIGNED;
    }
    return aligned(t.data, 16) ? FORGE_ATTN_OK : FORGE_ATTN_ERR_MISALIGNED;
}

int check_config(const forge_qkv_config* c, int flags, int allowed) {
    if (!c) return FORGE_ATTN_ERR_INVALID_ARG;
    if (flags & ~allowed) return FORGE_ATTN_ERR_INVALID_ARG;
    if (c->B < 1 || c->T < 1 || c->H < 1 || c->Hkv < 1 || c->H % c->Hkv)
        return FORGE_ATTN_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return FORGE_ATTN_ERR_UNSUPPORTED;
    if ((long long)c->B * c->T > 0x7fffffffll ||
        (long long)c->B * c->T * c->H * c->d >= (1ll << 31))
        return FORGE_ATTN_ERR_UNSUPPORTED;
    if (!std::isfinite(c->eps) || c->eps < 0.f) return FORGE_ATTN_ERR_INVALID_ARG;
    if (c->rot < 0 || c->rot > c->d || c->rot % 2 || c->axes < 1) return FORGE_ATTN_ERR_INVALID_ARG;
    if (!(flags & FORGE_QKV_ADJACENT) && c->rot % 16) return FORGE_ATTN_ERR_UNSUPPORTED;
    if (c->rot > 0) {
        if (!c->inv_freq) return FORGE_ATTN_ERR_INVALID_ARG;
        if (!aligned(c->inv_freq, 8) || !aligned(c->positions, 4) || !aligned(c->pair_axis, 4))
            return FORGE_ATTN_ERR_MISALIGNED;
    }
    if (!aligned(c->q_weight, 4) || !aligned(c->k_weight, 4)) return FORGE_ATTN_ERR_MISALIGNED;
    return FORGE_ATTN_OK;
}

Rope make_rope(const forge_qkv_config& c, int flags) {
    Rope r;
    r.freq = c.inv_freq;
    r.pos = c.positions;
    r.axis = c.pair_axis;
    r.pairs = c.rot / 2;
    r.axes = c.axes;
    r.adjacent = (flags & FORGE_QKV_ADJACENT) != 0;
    return r;
}

Part make_part(const forge_qkv_tensor* x, const float* w, int heads, int rep) {
    Part p{};
    if (x) {
        p.x = x->data;
        p.sb = x->stride_b;
        p.st = x->stride_t;
        p.sh = x->stride_h;
    }
    p.w = w;
    p.heads = heads;
    p.rep = rep;
    return p;
}

// Blocks of the backward: two to an SM, shared out among q, k and v by the bytes each
// moves, at least one to a part that is there and no more than it has units.
constexpr int kBwdBlocksPerSm = 2;
struct Blocks {
    int n[3];
};
Blocks share_out(const double* bytes, const long long* units) {
    const int all = kBwdBlocksPerSm * sm_count();
    const double sum = bytes[0] + bytes[1] + bytes[2];
    Blocks r;
    for (int j = 0; j < 3; ++j) {
        long long n = units[j] ? (long long)(all * bytes[j] / sum) : 0;
        if (units[j] && n < 1) n = 1;
        r.n[j] = (int)(n < units[j] ? n : units[j]);
    }
    return r;
}

int max_bwd_blocks() { return kBwdBlocksPerSm * sm_count() + 3; }

int status_of(cudaError_t e) { return e == cudaSuccess ? FORGE_ATTN_OK : FORGE_ATTN_ERR_CUDA; }

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

int forge_qkv_fwd(const forge_qkv_config* c, const forge_qkv_tensor* q, const forge_qkv_tensor* k,
                  const forge_qkv_tensor* v, void* q_out, void* k_out, void* v_out, int flags,
                  void* stream) {
    int st = check_config(c, flags, FORGE_ATTN_FP16 | FORGE_QKV_ADJACENT);
    if (st != FORGE_ATTN_OK) return st;
    if (!q && !k && !v) return FORGE_ATTN_ERR_INVALID_ARG;
    const forge_qkv_tensor* in[3] = {q, k, v};
    void* out[3] = {q_out, k_out, v_out};
    const int heads[3] = {c->H, c->Hkv, c->Hkv};
    const float* weight[3] = {c->q_weight, c->k_weight, nullptr};
    for (int j = 0; j < 3; ++j) {
        if ((in[j] != nullptr) != (out[j] != nullptr)) return FORGE_ATTN_ERR_INVALID_ARG;
        if (!in[j]) continue;
        if ((st = check_strides(*in[j], c->B, c->T, heads[j])) != FORGE_ATTN_OK) return st;
        if (!aligned(out[j], 16)) return FORGE_ATTN_ERR_MISALIGNED;
    }
    const int per = (c->d == 64 ? Cfg<64>::kSlots : Cfg<128>::kSlots) * kUnroll;
    Parts parts;
    Part* p = parts.part;
    int n[3];
    for (int j = 0; j < 3; ++j) {
        p[j] = make_part(in[j], weight[j], heads[j], c->H / heads[j]);
        p[j].y = out[j];
        n[j] = in[j] ? (heads[j] + per - 1) / per : 0;
    }
    const Shape s{c->B, c->T, c->H, (long long)c->B * c->T, c->eps};
    const Rope rope = make_rope(*c, flags);
    const int runs = n[0] + n[1] + n[2];
    const long long blocks = (s.tokens + kTok - 1) / kTok * runs;
    if (blocks > 0x7fffffffll) return FORGE_ATTN_ERR_UNSUPPORTED;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool f16 = (flags & FORGE_ATTN_FP16) != 0;
    auto* kernel = c->d == 64 ? (f16 ? qkv_fwd_kernel<64, true> : qkv_fwd_kernel<64, false>)
                              : (f16 ? qkv_fwd_kernel<128, true> : qkv_fwd_kernel<128, false>);
    kernel<<<(unsigned)blocks, kThreads, 0, cs>>>(parts, rope, s, n[0], n[1], runs, per);
    return status_of(cudaGetLastError());
}

size_t forge_qkv_bwd_workspace_size(int d) {
    if (d != 64 && d != 128) return 0;
    return (size_t)max_bwd_blocks() * d * sizeof(float);
}

int forge_qkv_bwd(const forge_qkv_config* c, const void* dq, const void* dk, const void* dv,
                  const forge_qkv_tensor* q, const forge_qkv_tensor* k,
                  const forge_qkv_tensor* q_grad, const forge_qkv_tensor* k_grad,
                  const forge_qkv_tensor* v_grad, float* dq_weight, float* dk_weight,
                  int accumulate, void* workspace, size_t workspace_bytes, int flags,
                  void* stream) {
    int st = check_config(c, flags, FORGE_ATTN_FP16 | FORGE_QKV_ADJACENT | FORGE_QKV_GRAD_F32);
    if (st != FORGE_ATTN_OK) return st;
    if (accumulate != 0 && accumulate != 1) return FORGE_ATTN_ERR_INVALID_ARG;
    if (!q_grad && !k_grad && !v_grad) return FORGE_ATTN_ERR_INVALID_ARG;
    const forge_qkv_tensor* x[3] = {q, k, nullptr};
    const forge_qkv_tensor* out[3] = {q_grad, k_grad, v_grad};
    const void* dy[3] = {dq, dk, dv};
    float* dw[3] = {dq_weight, dk_weight, nullptr};
    const float* weight[3] = {c->q_weight, c->k_weight, nullptr};
    const int heads[3] = {c->H, c->Hkv, c->Hkv};
    bool any_norm = false;
    for (int j = 0; j < 3; ++j) {
        if ((out[j] != nullptr) != (dy[j] != nullptr)) return FORGE_ATTN_ERR_INVALID_ARG;
        if (!out[j]) continue;
        if ((st = check_strides(*out[j], c->B, c->T, heads[j])) != FORGE_ATTN_OK) return st;
        if (!distinct(*out[j], c->B, c->T, heads[j], c->d)) return FORGE_ATTN_ERR_INVALID_ARG;
        if (!aligned(dy[j], 16)) return FORGE_ATTN_ERR_MISALIGNED;
        if (!weight[j]) continue;
        any_norm = true;
        if (!x[j] || !dw[j]) return FORGE_ATTN_ERR_INVALID_ARG;
        if ((st = check_strides(*x[j], c->B, c->T, heads[j])) != FORGE_ATTN_OK) return st;
        if (!aligned(dw[j], 4)) return FORGE_ATTN_ERR_MISALIGNED;
    }
    if (any_norm) {
        if (!workspace || workspace_bytes < forge_qkv_bwd_workspace_size(c->d))
            return FORGE_ATTN_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return FORGE_ATTN_ERR_MISALIGNED;
    }
    const bool f16 = (flags & FORGE_ATTN_FP16) != 0, g32 = (flags & FORGE_QKV_GRAD_F32) != 0;
    const Shape s{c->B, c->T, c->H, (long long)c->B * c->T, c->eps};
    const Rope rope = make_rope(*c, flags);
    const int per = (c->d == 64 ? Cfg<64>::kSlots : Cfg<128>::kSlots) * kUnroll;
    const long long tiles = (s.tokens + kTok - 1) / kTok;
    Parts parts;
    Part* p = parts.part;
    double bytes[3];
    long long units[3];
    for (int j = 0; j < 3; ++j) {
        const bool norm = out[j] && weight[j];
        p[j] = make_part(norm ? x[j] : nullptr, norm ? weight[j] : nullptr, heads[j],
                         c->H / heads[j]);
        p[j].g = dy[j];
        if (out[j]) {
            p[j].y = const_cast<void*>(out[j]->data);
            p[j].gsb = out[j]->stride_b;
            p[j].gst = out[j]->stride_t;
            p[j].gsh = out[j]->stride_h;
        }
        units[j] = out[j] ? tiles * ((heads[j] + per - 1) / per) : 0;
        bytes[j] = out[j] ? (double)c->H * (g32 ? 4 : 2) + heads[j] * (norm ? 4.0 : 2.0) : 0.0;
    }
    const Blocks n = share_out(bytes, units);
    const int blocks = n.n[0] + n.n[1] + n.n[2];
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    float* ws = static_cast<float*>(workspace);
#define FORGE_QKV_BWD(D_)                                                                       \
    (f16 ? (g32 ? qkv_bwd_kernel<D_, true, true> : qkv_bwd_kernel<D_, true, false>)             \
         : (g32 ? qkv_bwd_kernel<D_, false, true> : qkv_bwd_kernel<D_, false, false>))
    auto* kernel = c->d == 64 ? FORGE_QKV_BWD(64) : FORGE_QKV_BWD(128);
#undef FORGE_QKV_BWD
    kernel<<<blocks, kThreads, 0, cs>>>(parts, rope, s, n.n[0], n.n[1], per, ws);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && any_norm) {
        float* wq = p[0].w ? dq_weight : nullptr;
        float* wk = p[1].w ? dk_weight : nullptr;
        qkv_dw_kernel<<<dim3(c->d / 8, 2), 8 * kSumRows, 0, cs>>>(ws, wq, wk, n.n[0], n.n[1], c->d,
                                                                  accumulate);
        e = cudaGetLastError();
    }
    return status_of(e);
}

}  // extern "C"
