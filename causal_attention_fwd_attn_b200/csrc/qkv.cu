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
// A block takes 16 or 32 consecutive tokens and a run of heads of q, k or v, computes the tokens'
// sines and cosines once into shared memory, and keeps each thread at its token while it
// walks the heads.  Angles are reduced in 64 bits (turns =
// position * f / 2 pi, minus the nearest integer): a 32-bit product would lose the phase
// of far positions altogether.
#include <cmath>

#include "forge_attn.h"
#include "forge_internal.h"
#include "sm100_ptx.cuh"

namespace forge {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 2;  // heads that a block takes at a time

struct Rope {
    const double* freq;  // [pairs]
    const int* pos;      // [axes][B * T], or null: the token's index t
    const int* axis;     // [pairs], or null: axis 0
    int pairs, axes;
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
    int T, H;
    unsigned tokens;
    float eps;
};

template <int D>
struct Cfg {
    static constexpr int kLanes = D / 16;              // threads of a head row
    static constexpr int kGroups = kThreads / kLanes;  // rows at a time
    static constexpr int kTok = kGroups / kSlots;      // tokens of a block: 32 or 16
};

// First elements of the two 8-element chunks of thread i of a row.  Where whole heads are
// rotated by halves, or pairs are neighbours, they lie half a head apart, so that each of a
// warp's accesses covers half heads without gaps (with the chunks side by side, every
// second 16 bytes, B8 T1024 H12 d64 took 23.0 us instead of 18.9).  Where only the first 2 * pairs
// elements are rotated by halves: the halves of the same eight pairs while those last, then
// neighbours.
template <int D, bool ADJ>
__device__ __forceinline__ void chunks_of(int i, int pairs, int& a, int& b) {
    if (ADJ || pairs == 0) {
        a = 8 * i;
        b = a + D / 2;
    } else if (8 * i < pairs) {
        a = 8 * i;
        b = a + pairs;
    } else {
        a = 16 * i;
        b = a + 8;
    }
}

// Where (cos, sin) of pair j goes: thread, and its place among the thread's eight.
template <int D, bool ADJ>
__device__ __forceinline__ void place_of_pair(int j, int& thread, int& place) {
    if (ADJ) {  // chunk a holds pairs [4 i, 4 i + 4), chunk b those half a head further
        const int half = j >= D / 4, in = half ? j - D / 4 : j;
        thread = in / 4;
        place = 4 * half + in % 4;
    } else {
        thread = j / 8;
        place = j % 8;
    }
}
// How many of the thread's eight places hold a pair: all of the first `a` and of [4, 4 + b).
template <int D, bool ADJ>
__device__ __forceinline__ void pairs_of(int i, int pairs, int& a, int& b) {
    if (ADJ) {
        a = min(max(pairs - 4 * i, 0), 4);
        b = min(max(pairs - D / 4 - 4 * i, 0), 4);
    } else {
        a = b = 8 * i < pairs ? 4 : 0;
    }
}

// Ordinary loads, issued where they stand.  What they read may have been written by the kernel
// ahead, so that the read-only path is not theirs; loads that the compiler places took up to 8 %
// longer (backward B2 T4096 H16 d128 50.4 us against 49.0, B3 T1468 H16 d64 19.1 against 17.6).
// Volatile, or they could be moved out of the conditions that keep them inside their tables.
__device__ __forceinline__ int load(const int* p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ double load(const double* p) {
    double v;
    asm volatile("ld.global.f64 %0, [%1];" : "=d"(v) : "l"(p));
    return v;
}

// Tables in shared memory: what thread i of a row reads lies in four 16-byte columns, each
// with the threads of a row side by side.
// Angles, [kTok][4][kLanes] of (cos, cos, sin, sin) of two pairs.  A warp takes every eighth token.
// Past the last token the turn is none: rows that are not there are rotated too, and their
// zeros have to stay zeros in the sums over the rows.
template <int D, bool ADJ>
__device__ __forceinline__ void fill_angles(const Rope& r, const Shape& s, unsigned tok0,
                                            float* cs) {
    constexpr int L = Cfg<D>::kLanes, kTok = Cfg<D>::kTok;
    // The warp's tokens and the lane's pairs at once: the loads, then the long chains of
    // arithmetic, side by side.
    constexpr int N = kTok / (kThreads / 32), M = D / 2 / 32 > 0 ? D / 2 / 32 : 1;
    double f[M], turns[N][M];
    int ax[M];
    bool on[N][M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int j = lane_id() + 32 * m;
        ax[m] = r.axis && j < r.pairs ? min(max(load(r.axis + j), 0), r.axes - 1) : 0;
        f[m] = j < r.pairs ? load(r.freq + j) : 0.0;
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const unsigned tok = tok0 + warp_id() + n * (kThreads / 32);
            on[n][m] = (int)lane_id() + 32 * m < r.pairs && tok < s.tokens;
            int p = 0;
            if (on[n][m])
                p = r.pos ? load(r.pos + (size_t)ax[m] * s.tokens + tok)
                          : (int)(tok % (unsigned)s.T);
            turns[n][m] = (double)p;
        }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if ((int)lane_id() + 32 * m >= r.pairs) continue;
            double v = on[n][m] ? turns[n][m] * (f[m] * 0.15915494309189533577) : 0.;
            v -= rint(v);
            float sn, c;
            sincospif(2.f * (float)v, &sn, &c);
            int thread, place;
            place_of_pair<D, ADJ>(lane_id() + 32 * m, thread, place);
            const unsigned t = warp_id() + n * (kThreads / 32);
            float* at = cs + ((t * 4 + place / 2) * L + thread) * 4 + (place & 1);
            at[0] = c;
            at[2] = sn;
        }
}
// Norm weights, [4][kLanes] of four: the thread's chunks a and b.
template <int D, bool ADJ>
__device__ __forceinline__ void fill_weights(const float* w, int pairs, float* out) {
    constexpr int L = Cfg<D>::kLanes;
    if (threadIdx.x < D) {
        const int i = threadIdx.x % L, c = threadIdx.x / L;  // element c of the 16 of thread i
        int a, b;
        chunks_of<D, ADJ>(i, pairs, a, b);
        out[((c / 4) * L + i) * 4 + c % 4] = w[(c < 8 ? a : b - 8) + c];
    }
}

// A thread's 16 values of a row: chunk a in the first four pairs, chunk b in the others.
// Arithmetic goes by pairs (f32x2 instructions): the kernels are close to the issue limit.
template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& u, float2* f) {
    f[0] = unpack16x2<F16>(u.x);
    f[1] = unpack16x2<F16>(u.y);
    f[2] = unpack16x2<F16>(u.z);
    f[3] = unpack16x2<F16>(u.w);
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float2* f) {
    return make_uint4(pack16x2<F16>(f[0].x, f[0].y), pack16x2<F16>(f[1].x, f[1].y),
                      pack16x2<F16>(f[2].x, f[2].y), pack16x2<F16>(f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Rotates the thread's pairs (inverse: by -phi), na of its first four and nb of the others; other
// values stay as they are (not multiplied by one and zero: a neighbour may be infinite).  cs:
// the thread's first column of its token, the others STEP apart.
template <int STEP, bool ADJ, bool INVERSE>
__device__ __forceinline__ void rotate(float2* x, const float4* cs, int na, int nb) {
    if (na + nb == 0) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 v = cs[c * STEP];
        const float2 co = make_float2(v.x, v.y);
        const float2 up = INVERSE ? make_float2(-v.z, -v.w) : make_float2(v.z, v.w);
        const float2 dn = INVERSE ? make_float2(v.z, v.w) : make_float2(-v.z, -v.w);
        if constexpr (ADJ) {
            const int n = c < 2 ? na : nb + 4;
            const float2 p = x[2 * c], q = x[2 * c + 1];
            const float2 p2 = ffma2(make_float2(p.y, p.x), make_float2(dn.x, up.x),
                                    fmul2(p, both(co.x)));
            const float2 q2 = ffma2(make_float2(q.y, q.x), make_float2(dn.y, up.y),
                                    fmul2(q, both(co.y)));
            if (2 * c < n) x[2 * c] = p2;
            if (2 * c + 1 < n) x[2 * c + 1] = q2;
        } else {  // halves come in eights: all of the thread's pairs or none
            const float2 a = x[c], b = x[4 + c];
            x[c] = ffma2(b, dn, fmul2(a, co));
            x[4 + c] = ffma2(a, up, fmul2(b, co));
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

// Copies go through a ring in shared memory, each thread's own 16-byte slots: kDepth rows
// are in flight without a register or a barrier spent on them.  Where there is no row (on = false) the slot gets zeros and nothing is read.
__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's share of one head of q or k: norm, weights, rotation.
template <int D, bool F16, bool ADJ>
__device__ __forceinline__ void forward_row(uint4& oa, uint4& ob, bool norm, const float4* my_w,
                                            const float4* my_cs, int na, int nb, float eps) {
    float2 f[8];
    unpack8<F16>(oa, f);
    unpack8<F16>(ob, f + 4);
    if (norm) {
        float2 ss = fmul2(f[0], f[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) ss = ffma2(f[j], f[j], ss);
        const float2 r = both(rsqrtf(row_sum<Cfg<D>::kLanes>(ss.x + ss.y) * (1.f / D) + eps));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 w = my_w[c];
            f[2 * c] = fmul2(fmul2(f[2 * c], r), make_float2(w.x, w.y));
            f[2 * c + 1] = fmul2(fmul2(f[2 * c + 1], r), make_float2(w.z, w.w));
        }
    }
    rotate<1, ADJ, false>(f, my_cs, na, nb);
    oa = pack8<F16>(f);
    ob = pack8<F16>(f + 4);
}

constexpr int kFwdDepth = 4;
constexpr int kFwdBlocksPerSm = 3;

// Forward.  HBM is the bound of large calls: B1 T8000 H32 d128 (393 MB) takes 64.7 us, 6.08 TB/s or
// 0.93 of the copy rate; loads, arithmetic and stores in one thread without the ring, and
// scalar fp32 arithmetic, took 104.5.  Smaller ones wait for their chains (positions, angles,
// rows): B8 T1024 H12 d64 (75 MB) 17.7 us, where a plain copy of as many bytes takes 13.1; 48 tokens of
// a decoding step 3.7 us, a launch.  Blocks come and go (a persistent form with the next unit's
// rows and angles under way spent more on keeping its place: 79 us at the first size).
// Runs of heads that the blocks of a token tile take: nq runs of q's heads, nk of k's and the
// rest of v's, `per` heads to a run.
template <int D, bool F16, bool ADJ>
__global__ void __launch_bounds__(kThreads, kFwdBlocksPerSm)
    qkv_fwd_kernel(const __grid_constant__ Parts parts, const Rope rope, const Shape s, int nq, int nk,
                   int runs, int per) {
    using C = Cfg<D>;
    constexpr int L = C::kLanes, kTok = C::kTok;
    __shared__ float4 cs[kTok * 4 * L];
    __shared__ float4 wt[4 * L];
    __shared__ uint4 ring[kFwdDepth][2][kThreads];
    allow_dependents_launch();
    grid_dependency_wait();
    const unsigned tile = blockIdx.x / (unsigned)runs;
    int run = (int)(blockIdx.x - tile * (unsigned)runs);
    const int kind = run < nq ? 0 : (run < nq + nk ? 1 : 2);
    run -= kind == 0 ? 0 : (kind == 1 ? nq : nq + nk);
    const Part& p = parts.part[kind];
    const unsigned tok0 = tile * kTok;
    const int i = threadIdx.x % L, g = threadIdx.x / L;
    const int t = g % kTok, slot = g / kTok;
    const unsigned tok = min(tok0 + t, s.tokens - 1);
    const unsigned b = tok / (unsigned)s.T, tt = tok - b * (unsigned)s.T;
    int ea, eb;
    chunks_of<D, ADJ>(i, rope.pairs, ea, eb);
    const int first = run * per + slot;
    // heads this thread may take, counted from `first` (none where its token is not there)
    const int mine = tok0 + t < s.tokens ? min((run + 1) * per, p.heads) - first : 0;
    const int rows = (min((run + 1) * per, p.heads) - run * per + kSlots - 1) / kSlots;

    const uint16_t* x =
        static_cast<const uint16_t*>(p.x) + b * p.sb + tt * p.st + (mine > 0 ? first * p.sh : 0);
    const long long x_step = kSlots * p.sh;
    int fetched = 0;  // heads, in steps of kSlots
    auto prefetch = [&](int at) {
        const bool on = fetched < mine;
        copy16(&ring[at][0][threadIdx.x], x + ea, on);
        copy16(&ring[at][1][threadIdx.x], x + eb, on);
        copies_commit();
        fetched += kSlots;
        if (fetched < mine) x += x_step;  // (past the last row the address stays valid)
    };
#pragma unroll
    for (int n = 0; n < kFwdDepth; ++n) prefetch(n);
    const bool norm = kind < 2 && p.w != nullptr;
    if (kind < 2 && rope.pairs > 0) fill_angles<D, ADJ>(rope, s, tok0, reinterpret_cast<float*>(cs));
    if (norm) fill_weights<D, ADJ>(p.w, rope.pairs, reinterpret_cast<float*>(wt));
    __syncthreads();
    int na, nb;  // the thread's rotated pairs
    pairs_of<D, ADJ>(i, rope.pairs, na, nb);
    // the thread's angles and weights stay in registers: shared memory's pipe is the busiest
    float4 my_cs[4], my_w[4];
    if (kind < 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            my_cs[c] = cs[(t * 4 + c) * L + i];
            my_w[c] = wt[c * L + i];
        }
    }
    const long long head = (long long)s.T * D;
    uint16_t* y = static_cast<uint16_t*>(p.y) +
                  (((long long)b * s.H + (long long)first * p.rep) * s.T + tt) * D;

    for (int n = 0; n < rows; ++n) {
        copies_wait<kFwdDepth - 1>();
        uint4* at = &ring[n % kFwdDepth][0][threadIdx.x];
        uint4 oa = at[0], ob = at[kThreads];
        if (kind < 2) {
            forward_row<D, F16, ADJ>(oa, ob, norm, my_w, my_cs, na, nb, s.eps);
        }
        if (n * kSlots < mine) {
            for (int c = 0; c < p.rep; ++c, y += head) {
                *reinterpret_cast<uint4*>(y + ea) = oa;
                *reinterpret_cast<uint4*>(y + eb) = ob;
            }
            y += (kSlots - 1) * p.rep * head;
        }
        prefetch(n % kFwdDepth);  // into the slots just read
    }
    copies_wait<0>();
}

// The same where q, k and v are few heads (a tensor-parallel rank's): a block takes a token tile's
// heads of all three, so that they share its start and its angles.  A row is kSlots heads of
// one part; rows are q's (the first `qe`), k's (up to `ke`), then v's (up to `ve`).
// Chosen for up to kFewRows rows where there are two such blocks and more for every resident one:
// B16 T2048 H4 Hkv1 d128 (2048 tiles) 35.1 us against 43.8 with a block to each part, B64 T2048 H3 d64
// 69.5 against 89.6, H16 Hkv2 d128 (ten rows) 346 against 368 there and 91.7 against 92.1 at B16; with
// 512 tiles (B8 T1024 H8 Hkv1 d128) 18.0 against 17.3, with 188 (B1 T3000) 9.4 against 7.6.  Walking
// the parts costs registers and instructions: runs of a larger list of rows, across the
// parts, took 36.6 where the kernel above takes 34.3 (B2 T4096 H16 d128).
constexpr int kFewRows = 10;
template <int D, bool F16, bool ADJ>
__global__ void __launch_bounds__(kThreads, kFwdBlocksPerSm)
    qkv_fwd_few_kernel(const __grid_constant__ Parts parts, const Rope rope, const Shape s, int qe,
                       int ke, int ve) {
    using C = Cfg<D>;
    constexpr int L = C::kLanes, kTok = C::kTok;
    __shared__ float4 cs[kTok * 4 * L];
    __shared__ float4 wt[2][4 * L];
    __shared__ uint4 ring[kFwdDepth][2][kThreads];
    allow_dependents_launch();
    grid_dependency_wait();
    const unsigned tok0 = blockIdx.x * kTok;
    const int i = threadIdx.x % L, g = threadIdx.x / L;
    const int t = g % kTok, slot = g / kTok;
    const bool here = tok0 + t < s.tokens;
    const unsigned tok = min(tok0 + t, s.tokens - 1);
    const unsigned b = tok / (unsigned)s.T, tt = tok - b * (unsigned)s.T;
    int ea, eb;
    chunks_of<D, ADJ>(i, rope.pairs, ea, eb);
    auto kind_of = [&](int row) { return row < qe ? 0 : (row < ke ? 1 : 2); };
    auto end_of = [&](int kind) { return kind == 0 ? qe : (kind == 1 ? ke : ve); };

    // What is fetched next: the row, its part's end, the thread's head of how many.
    int f_row = 0, f_end, f_head, f_heads;
    const uint16_t* x;
    long long x_step;
    auto fetch_part = [&]() {  // from its first row on
        const int kind = kind_of(f_row);
        const Part& p = parts.part[kind];
        f_end = end_of(kind);
        f_head = slot;
        f_heads = here ? p.heads : 0;
        x_step = kSlots * p.sh;
        x = static_cast<const uint16_t*>(p.x) + b * p.sb + tt * p.st +
            (slot < p.heads ? slot * p.sh : 0);
    };
    auto prefetch = [&](int at) {
        const bool on = f_row < ve && f_head < f_heads;
        copy16(&ring[at][0][threadIdx.x], x + ea, on);
        copy16(&ring[at][1][threadIdx.x], x + eb, on);
        copies_commit();
        if (++f_row == f_end && f_row < ve) {
            fetch_part();
        } else {
            f_head += kSlots;
            if (f_head < f_heads) x += x_step;  // (past the last row the address stays valid)
        }
    };
    fetch_part();
#pragma unroll
    for (int n = 0; n < kFwdDepth; ++n) prefetch(n);
    if (rope.pairs > 0 && ke > 0) fill_angles<D, ADJ>(rope, s, tok0, reinterpret_cast<float*>(cs));
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
        if (parts.part[kind].w)
            fill_weights<D, ADJ>(parts.part[kind].w, rope.pairs, reinterpret_cast<float*>(wt[kind]));
    __syncthreads();
    int na, nb;  // the thread's rotated pairs
    pairs_of<D, ADJ>(i, rope.pairs, na, nb);
    float4 my_cs[4], my_w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) my_cs[c] = cs[(t * 4 + c) * L + i];
    const long long head = (long long)s.T * D;

    int row = 0, at_now = 0;
    for (int kind = 0; kind < 3; ++kind) {
        const Part& p = parts.part[kind];
        const int end = end_of(kind), heads = here ? p.heads : 0;
        const bool norm = p.w != nullptr;
        if (norm) {
#pragma unroll
            for (int c = 0; c < 4; ++c) my_w[c] = wt[kind][c * L + i];
        }
        uint16_t* y = static_cast<uint16_t*>(p.y) +
                      (((long long)b * s.H + (long long)slot * p.rep) * s.T + tt) * D;
        for (int h = slot; row < end; ++row, h += kSlots) {
            copies_wait<kFwdDepth - 1>();
            uint4* at = &ring[at_now][0][threadIdx.x];
            uint4 oa = at[0], ob = at[kThreads];
            if (kind < 2) forward_row<D, F16, ADJ>(oa, ob, norm, my_w, my_cs, na, nb, s.eps);
            if (h < heads) {
                for (int c = 0; c < p.rep; ++c, y += head) {
                    *reinterpret_cast<uint4*>(y + ea) = oa;
                    *reinterpret_cast<uint4*>(y + eb) = ob;
                }
                y += (kSlots - 1) * p.rep * head;
            }
            prefetch(at_now);  // into the slots just read
            at_now = (at_now + 1) % kFwdDepth;
        }
    }
    copies_wait<0>();
}

// The ring of the backward: per step one gradient row (16 values: two or four slots) and the
// row of x (two slots).
template <bool G32>
struct Bwd {
    static constexpr int kG = G32 ? 4 : 2;
    static constexpr int kDepth = G32 ? 3 : 4;
    static constexpr int kRingBytes = kDepth * (kG + 2) * kThreads * 16;
    static constexpr int kBlocksPerSm = G32 ? 2 : 3;  // what shared memory holds
};

// Backward.  B2 T4096 H16 d128 (268 MB) takes 49 us, 5.4 TB/s or 0.83 of the copy rate, with fp32
// gradients (369 MB) 63 us, 0.89 of it; B3 T1023 H12 Hkv4 d64 with fp32 gradients (42 MB) 15 us, most of
// it latencies.  Two thirds of the issue slots are busy (a third of them with the norm), so angles and
// weights are read from shared memory and three blocks fit on an SM (in registers, with two
// blocks: 62 us at the first size).
// Blocks [0, nq) walk q's (token tile, run of heads) units, the next nk k's, the rest v's.
// A head row takes p.rep steps, one for each of the attention's heads that share it; the
// norm's backward follows the last.  Each block of q and k sums its share of the norm
// weight's gradient in registers and writes it to partials[block][D].
template <int D, bool F16, bool G32, bool ADJ>
__global__ void __launch_bounds__(kThreads, Bwd<G32>::kBlocksPerSm)
    qkv_bwd_kernel(const __grid_constant__ Parts parts, const Rope rope, const Shape s, int nq, int nk,
                   int per, float* partials) {
    using C = Cfg<D>;
    using R = Bwd<G32>;
    constexpr int L = C::kLanes, kTok = C::kTok;
    constexpr int kStep = (R::kG + 2) * kThreads;
    extern __shared__ uint4 ring[];  // [kDepth][kG + 2][kThreads]
    __shared__ float4 cs[kTok * 4 * L];
    __shared__ float4 wt[4 * L];
    allow_dependents_launch();
    grid_dependency_wait();
    unsigned blk = blockIdx.x;
    const int kind = (int)blk < nq ? 0 : ((int)blk < nq + nk ? 1 : 2);
    const Part& p = parts.part[kind];
    blk -= kind == 0 ? 0 : (kind == 1 ? nq : nq + nk);
    const unsigned blocks = kind == 0 ? nq : (kind == 1 ? nk : gridDim.x - nq - nk);
    const int i = threadIdx.x % L, g = threadIdx.x / L;
    const int t = g % kTok, slot = g / kTok;
    const bool turn = kind < 2 && rope.pairs > 0;
    const bool norm = kind < 2 && p.w != nullptr;
    int ea, eb;
    chunks_of<D, ADJ>(i, rope.pairs, ea, eb);
    if (norm) fill_weights<D, ADJ>(p.w, rope.pairs, reinterpret_cast<float*>(wt));
    float2 dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = both(0.f);
    const unsigned runs = (unsigned)((p.heads + per - 1) / per);
    const unsigned units = (s.tokens + kTok - 1) / kTok * runs;
    int na, nb;  // the thread's rotated pairs
    pairs_of<D, ADJ>(i, turn ? rope.pairs : 0, na, nb);
    const float4* my_cs = cs + t * 4 * L + i;
    const long long head = (long long)s.T * D;  // from one of the attention's heads to the next
    const long long x_step = kSlots * p.sh, y_step = kSlots * p.gsh;
    uint4* const ring0 = ring + threadIdx.x;

    for (unsigned unit = blk; unit < units; unit += blocks) {
        const unsigned tok0 = unit / runs * kTok;
        const int h0 = (int)(unit % runs) * per, first = h0 + slot;
        const int last = min(h0 + per, p.heads);
        const unsigned tok = min(tok0 + t, s.tokens - 1);
        const unsigned b = tok / (unsigned)s.T, tt = tok - b * (unsigned)s.T;
        const int mine = tok0 + t < s.tokens ? last - first : 0;
        const long long at_first = mine > 0 ? first : 0;
        const uint16_t* x =
            static_cast<const uint16_t*>(p.x) + b * p.sb + tt * p.st + at_first * p.sh;
        uint16_t* y = static_cast<uint16_t*>(p.y) + b * p.gsb + tt * p.gst + at_first * p.gsh;
        const char* dy = static_cast<const char*>(p.g) +
                         (((long long)b * s.H + at_first * p.rep) * s.T + tt) * (D * (G32 ? 4 : 2));
        int fetched = 0, shared_head = 0;  // heads in steps of kSlots; which of the rep rows
        int pf_at = 0;
        auto prefetch = [&]() {
            uint4* at = ring0 + pf_at;
            pf_at = pf_at == (R::kDepth - 1) * kStep ? 0 : pf_at + kStep;
            const bool on = fetched < mine;
            if constexpr (G32) {
                // the row's threads side by side, each 16 bytes: whole sectors, which other
                // threads of the row will read (a thread's own 32 bytes at a time, every sector
                // came twice: 90.7 us at B2 T4096 H16 d128)
                uint4* row = at - i + 3 * (threadIdx.x - i);  // [4 L] of the row's own
                const float* src = reinterpret_cast<const float*>(dy) + 4 * i;
                __syncwarp();  // the row's threads have read the slots
#pragma unroll
                for (int q = 0; q < 4; ++q) copy16(row + q * L + i, src + q * 4 * L, on);
            } else {
                const uint16_t* src = reinterpret_cast<const uint16_t*>(dy);
                copy16(at, src + ea, on);
                copy16(at + kThreads, src + eb, on);
            }
            // the row's last step brings its x, and goes on to the next row
            if (++shared_head == p.rep) {
                if (norm) {
                    copy16(at + R::kG * kThreads, x + ea, on);
                    copy16(at + (R::kG + 1) * kThreads, x + eb, on);
                }
                shared_head = 0;
                fetched += kSlots;
                if (fetched < mine) {  // (past the last row the addresses stay valid)
                    dy += ((kSlots - 1) * p.rep + 1) * head * (G32 ? 4 : 2);
                    x += x_step;
                }
            } else if (on) {
                dy += head * (G32 ? 4 : 2);
            }
            copies_commit();
        };
        copies_wait<0>();  // (a slot's zeros past the last unit's end come before what follows)
#pragma unroll
        for (int n = 0; n < R::kDepth; ++n) prefetch();
        if (turn) {
            __syncthreads();  // the previous unit's angles have been read
            fill_angles<D, ADJ>(rope, s, tok0, reinterpret_cast<float*>(cs));
        }
        __syncthreads();
        int at_now = 0;
        const int rows = (last - h0 + kSlots - 1) / kSlots;
        for (int row = 0; row < rows; ++row) {
            float2 f[8];
            const uint4* at = ring0 + at_now;
            auto step = [&](float2* a) {  // the next gradient row
                copies_wait<R::kDepth - 1>();
                at = ring0 + at_now;
                at_now = at_now == (R::kDepth - 1) * kStep ? 0 : at_now + kStep;
                if constexpr (G32) {
                    __syncwarp();  // the row's threads have waited for their copies
                    const uint4* row = at - i + 3 * (threadIdx.x - i);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 v = row[(q < 2 ? ea / 4 + q : eb / 4 + q - 2)];
                        a[2 * q] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
                        a[2 * q + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
                    }
                } else {
                    unpack8<F16>(at[0], a);
                    unpack8<F16>(at[kThreads], a + 4);
                }
            };
            step(f);
            for (int c = 1; c < p.rep; ++c) {
                prefetch();
                float2 a[8];
                step(a);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = fadd2(f[j], a[j]);
            }
            rotate<L, ADJ, true>(f, my_cs, na, nb);
            if (norm) {
                // dx = r (u - n mean(u n)) with n = r x, u = g w: both row sums at once
                float2 x2[8];
                unpack8<F16>(at[R::kG * kThreads], x2);
                unpack8<F16>(at[(R::kG + 1) * kThreads], x2 + 4);
                float2 ss = both(0.f), ux = both(0.f), u[8];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 w = wt[c * L + i];
                    u[2 * c] = fmul2(f[2 * c], make_float2(w.x, w.y));
                    u[2 * c + 1] = fmul2(f[2 * c + 1], make_float2(w.z, w.w));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss = ffma2(x2[j], x2[j], ss);
                    ux = ffma2(u[j], x2[j], ux);
                }
                // (a row that is not there holds zeros: with eps = 0 its r would be infinite)
                const float mean = row_sum<L>(ss.x + ss.y) * (1.f / D) + s.eps;
                const float r = row * kSlots < mine ? rsqrtf(mean) : 0.f;
                const float m = row_sum<L>(ux.x + ux.y) * r * (1.f / D);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 n = fmul2(x2[j], both(r));
                    dw[j] = ffma2(f[j], n, dw[j]);
                    f[j] = fmul2(ffma2(n, both(-m), u[j]), both(r));
                }
            }
            if (row * kSlots < mine) {
                *reinterpret_cast<uint4*>(y + ea) = pack8<F16>(f);
                *reinterpret_cast<uint4*>(y + eb) = pack8<F16>(f + 4);
                y += y_step;
            }
            prefetch();
        }
    }
    copies_wait<0>();
    if (norm) {
        // the block's sum, always added in the same order
        __syncthreads();
        float* red = reinterpret_cast<float*>(ring);  // [warps][D]
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int o = L; o < 32; o <<= 1) {
                dw[j].x += __shfl_xor_sync(0xffffffffu, dw[j].x, o);
                dw[j].y += __shfl_xor_sync(0xffffffffu, dw[j].y, o);
            }
            if (lane_id() < L) {
                const int e = j < 4 ? ea + 2 * j : eb + 2 * (j - 4);
                red[warp_id() * D + e] = dw[j].x;
                red[warp_id() * D + e + 1] = dw[j].y;
            }
        }
        __syncthreads();
        if (threadIdx.x < D) {
            float sum = 0.f;
#pragma unroll
            for (int wv = 0; wv < kThreads / 32; ++wv) sum += red[wv * D + threadIdx.x];
            partials[(size_t)blockIdx.x * D + threadIdx.x] = sum;
        }
    }
}

// dw (+)= sum of the blocks' partials, in 64 bits and in a fixed order.  Block x: eight
// elements; block y: q or k (partials [first, first + n)).
constexpr int kSumRows = 128;
__global__ void __launch_bounds__(8 * kSumRows)
    qkv_dw_kernel(const float* partials, float* dwq, float* dwk, int nq, int nk, int D,
                  int accumulate) {
    allow_dependents_launch();
    grid_dependency_wait();
    float* out = blockIdx.y == 0 ? dwq : dwk;
    if (!out) return;
    const int first = blockIdx.y == 0 ? 0 : nq, n = blockIdx.y == 0 ? nq : nk;
    const int col = threadIdx.x & 7, row = threadIdx.x >> 3;
    const int e = blockIdx.x * 8 + col;
    double sum = 0.0;
    for (int k = row; k < n; k += kSumRows) sum += (double)partials[(long long)(first + k) * D + e];
    // rows of a warp, then of the warps
    constexpr int kWarps = 8 * kSumRows / 32;
    __shared__ double red[kWarps][8];
    auto over_rows = [](double v) {
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        return v + __shfl_xor_sync(0xffffffffu, v, 16);
    };
    sum = over_rows(sum);
    if (lane_id() < 8) red[warp_id()][col] = sum;
    __syncthreads();
    if (warp_id() == 0) {
        sum = 0.0;
        for (int w = lane_id() / 8; w < kWarps; w += 4) sum += red[w][col];
        sum = over_rows(sum);
        if (lane_id() < 8) out[e] = accumulate ? (float)((double)out[e] + sum) : (float)sum;
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Two ranges of `n` bytes.
bool overlap(const void* a, const void* b, long long n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)n && y < x + (uintptr_t)n;
}

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

Rope make_rope(const forge_qkv_config& c) {
    Rope r;
    r.freq = c.inv_freq;
    r.pos = c.positions;
    r.axis = c.pair_axis;
    r.pairs = c.rot / 2;
    r.axes = c.axes;
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

// Heads of a run, and the units (token tile, run) of each part.  A unit costs kStart (its
// latencies and its angles) and its rows, in the time of one row of eight to a thread or
// fewer: the choice is the one with the least work for a resident block plus one unit, the
// wait for the last.
struct Split {
    long long units[3];
    int per;
};
constexpr double kStart = 4.5;
Split split_heads(const double* row_cost, const int* heads, long long tiles, int resident) {
    Split best{};
    double best_time = 0.0;
    for (int rows = 8; rows >= 1; rows /= 2) {
        Split b{};
        b.per = rows * kSlots;
        double sum = 0.0, most = 0.0;
        for (int j = 0; j < 3; ++j) {
            if (row_cost[j] <= 0.0) continue;
            b.units[j] = tiles * ((heads[j] + b.per - 1) / b.per);
            const int used = heads[j] < b.per ? (heads[j] + kSlots - 1) / kSlots : rows;
            const double cost = kStart + used * row_cost[j];
            sum += b.units[j] * cost;
            most = cost > most ? cost : most;
        }
        const double time = sum / resident + most;
        if (rows == 8 || time < best_time) {
            best = b;
            best_time = time;
        }
    }
    return best;
}

// Blocks of the backward: one to a unit while that keeps the partial sums of the weights'
// gradients few.
constexpr int kMaxPartials = 1024;  // of q, and of k
struct Blocks {
    int n[3], per;
};

template <int D, bool F16, bool G32, bool ADJ>
cudaError_t launch_bwd_t(const Parts& parts, const Rope& rope, const Shape& s, const Blocks& n,
                         float* ws, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured{0};
    auto* kernel = qkv_bwd_kernel<D, F16, G32, ADJ>;
    cudaError_t e = set_max_dynamic_smem(kernel, Bwd<G32>::kRingBytes, configured);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(n.n[0] + n.n[1] + n.n[2]), dim3(kThreads),
                            Bwd<G32>::kRingBytes, stream, parts, rope, s, n.n[0], n.n[1], n.per, ws);
}
template <int D, bool F16, bool G32>
cudaError_t launch_bwd(bool adj, const Parts& parts, const Rope& rope, const Shape& s,
                       const Blocks& n, float* ws, cudaStream_t stream) {
    return adj ? launch_bwd_t<D, F16, G32, true>(parts, rope, s, n, ws, stream)
               : launch_bwd_t<D, F16, G32, false>(parts, rope, s, n, ws, stream);
}

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
    for (int j = 0; j < 3; ++j)
        if (out[j] && out[(j + 1) % 3] &&
            overlap(out[j], out[(j + 1) % 3], 2ll * c->B * c->T * c->H * c->d))
            return FORGE_ATTN_ERR_INVALID_ARG;
    const long long tokens = (long long)c->B * c->T, tok = c->d == 64 ? Cfg<64>::kTok : Cfg<128>::kTok,
                    tiles = (tokens + tok - 1) / tok;
    Parts parts;
    double row_cost[3];
    for (int j = 0; j < 3; ++j) {
        parts.part[j] = make_part(in[j], weight[j], heads[j], c->H / heads[j]);
        parts.part[j].y = out[j];
        row_cost[j] = in[j] ? 0.5 + 0.5 * parts.part[j].rep : 0.0;
    }
    const Split split = split_heads(row_cost, heads, tiles, kFwdBlocksPerSm * sm_count());
    const int per = split.per;
    int n[3];
    for (int j = 0; j < 3; ++j) n[j] = in[j] ? (heads[j] + per - 1) / per : 0;
    const Shape s{c->T, c->H, (unsigned)tokens, c->eps};
    const Rope rope = make_rope(*c);
    const int runs = n[0] + n[1] + n[2];
    const long long blocks = tiles * runs;
    if (blocks > 0x7fffffffll) return FORGE_ATTN_ERR_UNSUPPORTED;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool f16 = (flags & FORGE_ATTN_FP16) != 0;
    const bool adj = (flags & FORGE_QKV_ADJACENT) != 0;
    int ends[3], rows = 0;
    for (int j = 0; j < 3; ++j)
        ends[j] = rows += in[j] ? (heads[j] + kSlots - 1) / kSlots : 0;
    if (rows <= kFewRows && tiles >= 2 * kFwdBlocksPerSm * sm_count()) {
#define FORGE_QKV_FWD(D_)                                                                       \
    (f16 ? (adj ? qkv_fwd_few_kernel<D_, true, true> : qkv_fwd_few_kernel<D_, true, false>)     \
         : (adj ? qkv_fwd_few_kernel<D_, false, true> : qkv_fwd_few_kernel<D_, false, false>))
        auto* kernel = c->d == 64 ? FORGE_QKV_FWD(64) : FORGE_QKV_FWD(128);
#undef FORGE_QKV_FWD
        return status_of(launch_dependent(kernel, dim3((unsigned)tiles), dim3(kThreads), 0, cs, parts,
                                          rope, s, ends[0], ends[1], ends[2]));
    }
#define FORGE_QKV_FWD(D_)                                                                 \
    (f16 ? (adj ? qkv_fwd_kernel<D_, true, true> : qkv_fwd_kernel<D_, true, false>)       \
         : (adj ? qkv_fwd_kernel<D_, false, true> : qkv_fwd_kernel<D_, false, false>))
    auto* kernel = c->d == 64 ? FORGE_QKV_FWD(64) : FORGE_QKV_FWD(128);
#undef FORGE_QKV_FWD
    return status_of(launch_dependent(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, cs, parts, rope,
                                      s, n[0], n[1], runs, per));
}

size_t forge_qkv_bwd_workspace_size(int d) {
    if (d != 64 && d != 128) return 0;
    return (size_t)(2 * kMaxPartials) * d * sizeof(float);
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
    // (each is read, added to and written by its own blocks of the second kernel)
    if (out[0] && weight[0] && out[1] && weight[1] && overlap(dw[0], dw[1], 4ll * c->d))
        return FORGE_ATTN_ERR_INVALID_ARG;
    const bool f16 = (flags & FORGE_ATTN_FP16) != 0, g32 = (flags & FORGE_QKV_GRAD_F32) != 0;
    const long long tokens = (long long)c->B * c->T, tok = c->d == 64 ? Cfg<64>::kTok : Cfg<128>::kTok,
                    tiles = (tokens + tok - 1) / tok;
    const Shape s{c->T, c->H, (unsigned)tokens, c->eps};
    const Rope rope = make_rope(*c);
    const bool adj = (flags & FORGE_QKV_ADJACENT) != 0;
    const int resident = (g32 ? Bwd<true>::kBlocksPerSm : Bwd<false>::kBlocksPerSm) * sm_count();
    Parts parts;
    Part* p = parts.part;
    double row_cost[3];
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
        row_cost[j] = out[j] ? 0.5 * p[j].rep + (norm ? 0.5 : 0.0) : 0.0;
    }
    const Split split = split_heads(row_cost, heads, tiles, resident);
    Blocks n;
    n.per = split.per;
    for (int j = 0; j < 3; ++j)
        n.n[j] = (int)(split.units[j] < kMaxPartials ? split.units[j] : kMaxPartials);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    float* ws = static_cast<float*>(workspace);
#define FORGE_QKV_BWD(D_)                                                                \
    (c->d != D_   ? cudaErrorInvalidValue                                                \
     : f16 && g32 ? launch_bwd<D_, true, true>(adj, parts, rope, s, n, ws, cs)      \
     : f16        ? launch_bwd<D_, true, false>(adj, parts, rope, s, n, ws, cs)     \
     : g32        ? launch_bwd<D_, false, true>(adj, parts, rope, s, n, ws, cs)     \
                  : launch_bwd<D_, false, false>(adj, parts, rope, s, n, ws, cs))
    cudaError_t e = c->d == 64 ? FORGE_QKV_BWD(64) : FORGE_QKV_BWD(128);
#undef FORGE_QKV_BWD
    if (e == cudaSuccess && any_norm)
        e = launch_dependent(qkv_dw_kernel, dim3(c->d / 8, 2), dim3(8 * kSumRows), 0, cs,
                             (const float*)ws, p[0].w ? dq_weight : nullptr,
                             p[1].w ? dk_weight : nullptr, n.n[0], n.n[1], c->d, accumulate);
    return status_of(e);
}

}  // extern "C"
