// Rotary positions, and the RMS norm of each head with the rotation in the same pass (formulas
// and layout in include/anchor_attn.h), forward and backward.
//
// Both are bound by memory: every element is read and written once, with about ten operations in
// between.  The angle of a (token, pair) is shared by all heads, and costs about forty operations
// (a 64-bit product for each axis, sincospi), so a thread keeps a token and a set of pairs and
// walks the heads: its sines and cosines stay in registers.  The angle is taken as a 64-bit
// fraction of a turn; the product position * phase wraps at whole turns by itself, which is the
// exact reduction that fp32 (or even fp64) angles lack at far positions, and costs no fp64.
//
// A group of d / (2 V) threads of one warp holds a row: V first and V second elements of its pairs
// for each thread (V = 16 bytes of elements), so loads and stores are 16 bytes wide:
//   halves       two chunks rot / 2 apart (columns behind rot: (d - rot) / 2 apart)
//   neighbours   two adjacent chunks
//   odd halves   rot / 2 or (d - rot) / 2 not a multiple of V: adjacent chunks, the partners come
//                through shared memory
// Few tokens: the heads are cut into groups so that the SMs are filled (heads_per, below).
//
// Backward: dz = R^T dy; with a norm, xhat = x r, r = 1 / sqrt(mean x^2 + eps):
//   dw += dz o xhat,  dx = r (w o dz - xhat mean(w o dz o xhat)).
// dw: each thread sums its columns over its rows, the block adds its groups in order, and a second
// launch adds the blocks in order; the grid depends on the shapes alone, so the bits do too.
#include "common.cuh"
#include "views.cuh"

#include <math.h>
#include <stdlib.h>

namespace anchor {
namespace {

constexpr int kThreads = 128;
constexpr int kFill = 152 * 12;      // blocks that fill the GPU, below which heads are cut into groups
// Most blocks of a backward whose dweight is summed: bf16, all tensors together as many as are resident
// at once (three an SM), so that no tail is left and few blocks' sums remain (8 x 24 x 4200 rows of 64: 61
// us against 70 with 1216 a tensor); fp32, whose threads have more in flight, 1216 a tensor (101 us
// against 111).
constexpr int kBwdBlocks16 = 152 * 3, kBwdBlocks32 = 152 * 8;

enum Mode { kHalves = 0, kNeighbours = 1, kOddHalves = 2 };

struct Rows {
    const void *x, *dy, *w, *pos;
    void *y;        // forward: Y; backward: dX
    float *part;    // backward: the blocks' dweight sums [blocks][d], or null
    long long xb, xh, xn, yb, yh, yn, gb, gh, gn;  // strides of x, y, dy
    long long pos_batch, start;
    int heads, n, tokens;      // tokens = B * n
    int heads_per, groups;     // heads per thread and groups of them
    int blocks, token_blocks;  // blocks of this tensor: groups * token_blocks
};

struct Params {
    Rows r[2];
    const unsigned long long *phases;
    int d, rot, axes, norm, w_f32, pos64;
    float eps, magnitude;
};

template <typename T> constexpr int kV = 16 / sizeof(T);

__device__ __forceinline__ void store_chunk(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16 *p, const float *v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
// raw 16 bytes, kept until they are used: the loads of several heads are in flight together
template <typename T> struct Raw {
    uint4 a, b;
};
template <typename T> __device__ __forceinline__ void unpack(const uint4 &a, float *v);
template <> __device__ __forceinline__ void unpack<float>(const uint4 &a, float *v) {
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4 &a, float *v) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// This thread's columns and the sines of its pairs for one token.
template <typename T, int MODE>
struct Turn {
    static constexpr int V = kV<T>;
    static constexpr int NS = MODE == kOddHalves ? 2 * V : V;
    int a, b;           // first element of the two chunks
    float c[NS], s[NS];
    unsigned on;        // bit i: pair (odd halves: element) i is rotated

    __device__ __forceinline__ void place(const Params &p, int t) {
        if (MODE == kHalves) {
            const int rc = p.rot / (2 * V);
            a = t < rc ? t * V : p.rot + (t - rc) * V;
            b = t < rc ? a + p.rot / 2 : a + (p.d - p.rot) / 2;
        } else {
            a = t * 2 * V, b = a + V;
        }
        on = 0;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const bool r = MODE == kHalves ? a < p.rot / 2 : MODE == kNeighbours ? a + 2 * i < p.rot : a + i < p.rot;
            on |= r ? 1u << i : 0u;
        }
    }
    // pair of slot i
    __device__ __forceinline__ int pair(const Params &p, int i) const {
        if (MODE == kHalves) return a + i;
        if (MODE == kNeighbours) return a / 2 + i;
        return a + i < p.rot / 2 ? a + i : a + i - p.rot / 2;
    }
    __device__ __forceinline__ void angles(const Params &p, const Rows &r, int bi, int row) {
        if (!on) return;
        unsigned long long at[3] = {0, 0, 0};
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (x >= p.axes) continue;
            if (!r.pos) {
                at[x] = (unsigned long long)(r.start + row);
            } else {
                const long long o = (long long)bi * r.pos_batch + (long long)row * p.axes + x;
                at[x] = p.pos64 ? (unsigned long long)reinterpret_cast<const long long *>(r.pos)[o]
                                : (unsigned long long)(long long)reinterpret_cast<const int *>(r.pos)[o];
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (!(on >> i & 1u)) continue;
            const unsigned long long *ph = p.phases + pair(p, i);
            unsigned long long t = at[0] * __ldg(ph);
            if (p.axes > 1) t += at[1] * __ldg(ph + p.rot / 2);
            if (p.axes > 2) t += at[2] * __ldg(ph + p.rot);
            // the upper 32 bits as half turns in [-1, 1]: 2^-32 of a turn is cut off at most, and rounding to fp32 moves
            // it by up to 2^-26 (near half a turn; 1e-7 rad)
            const float half_turns = (float)(int)(t >> 32) * 0x1p-31f;
            sincospif(half_turns, &s[i], &c[i]);
            s[i] *= p.magnitude, c[i] *= p.magnitude;
            if (MODE == kOddHalves && a + i < p.rot / 2) s[i] = -s[i];
        }
    }
    // v[0..V) the first chunk, v[V..2V) the second; sign: 1 turns, -1 turns back (both scaled)
    __device__ __forceinline__ void apply(const Params &p, float *v, float sign, float *row) const {
        if constexpr (MODE == kOddHalves) {
            // the group's row through shared memory (the group is part of one warp)
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) row[a + i] = v[i];
            __syncwarp();
            float o[2 * V];
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) {
                const int e = a + i;
                o[i] = (on >> i & 1u) ? row[e < p.rot / 2 ? e + p.rot / 2 : e - p.rot / 2] : 0.f;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2 * V; ++i)
                if (on >> i & 1u) v[i] = fmaf(v[i], c[i], sign * s[i] * o[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!(on >> i & 1u)) continue;
                float &x = MODE == kHalves ? v[i] : v[2 * i];
                float &y = MODE == kHalves ? v[V + i] : v[2 * i + 1];
                const float u = x * c[i] - y * (sign * s[i]), w = x * (sign * s[i]) + y * c[i];
                x = u, y = w;
            }
        }
    }
};

__device__ __forceinline__ float group_sum(float v, int threads) {
    for (int o = threads / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__device__ __forceinline__ void load_weight(const Params &p, const void *w, int a, float *v) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < kV<T>; ++i) v[i] = 1.f;
        return;
    }
#pragma unroll
    for (int i = 0; i < kV<T>; ++i)
        v[i] = p.w_f32 ? reinterpret_cast<const float *>(w)[a + i] : to_f32(reinterpret_cast<const T *>(w)[a + i]);
}

// BWD: y receives dx; with a norm x is read too.  Every lane of a warp runs every step (the
// shuffles and __syncwarp), lanes without a token or head on row 0 without loads and stores.
template <typename T, int MODE, bool BWD>
__global__ void __launch_bounds__(kThreads, MODE == kOddHalves ? (BWD ? 3 : 4) : BWD ? (sizeof(T) == 2 ? 3 : 4) : 5) norm_rope_kernel(const Params p) {
    constexpr int V = kV<T>;
    // Heads whose rows are on their way.  bf16: a head's place is refilled as soon as it is unpacked
    // (4 x 32 heads x 16384 rows of 128: 170 us against 179 for three at a time).  fp32 is not unpacked,
    // its place stays in use: refilled behind the batch (67 us against 80, 8 x 24 x 4200 rows of 64).
    constexpr bool kRefill = sizeof(T) == 2;
    constexpr int kAhead = MODE == kOddHalves ? 2 : kRefill ? 3 : 4;
    extern __shared__ float sh[];  // odd halves: [groups][d + 4]; backward: the block's dweight [groups][d]
    grid_dependency_wait();
    grid_dependents_launch();
    const bool second = (int)blockIdx.x >= p.r[0].blocks;
    const Rows &r = p.r[second ? 1 : 0];
    const int block = (int)blockIdx.x - (second ? p.r[0].blocks : 0);
    const int tpr = p.d / (2 * V), per_block = kThreads / tpr;
    const int g = threadIdx.x / tpr, t = threadIdx.x % tpr;
    float *row = sh + g * (p.d + 4);
    Turn<T, MODE> turn;
    turn.place(p, t);
    float w[2 * V], dw[BWD ? 2 * V : 1];
    load_weight<T>(p, p.norm ? r.w : nullptr, turn.a, w);
    load_weight<T>(p, p.norm ? r.w : nullptr, turn.b, w + V);
    if (BWD) {
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) dw[i] = 0.f;
    }
    const int group = block / r.token_blocks;
    const int h0 = group * r.heads_per, h1 = min(h0 + r.heads_per, r.heads);
    const float inv_d = 1.f / (float)p.d;
    const T *X = reinterpret_cast<const T *>(r.x), *DY = reinterpret_cast<const T *>(r.dy);
    T *Y = reinterpret_cast<T *>(r.y);
    // all threads of the block make the same number of steps
    for (long long base = (long long)(block % r.token_blocks) * per_block; base < r.tokens;
         base += (long long)r.token_blocks * per_block) {
        const bool live = base + g < r.tokens;
        const int tok = live ? (int)(base + g) : 0;
        const int bi = tok / r.n, i = tok - bi * r.n;
        turn.angles(p, r, bi, i);
        const long long xo = bi * r.xb + i * r.xn, yo = bi * r.yb + i * r.yn, go = bi * r.gb + i * r.gn;
        const bool need_x = !BWD || p.norm;
        Raw<T> xr[kAhead], gr[BWD ? kAhead : 1];
        auto fetch = [&](int k, int h) {
            if (!live || h >= h1) return;
            if (need_x) {
                const T *x = X + xo + (long long)h * r.xh;
                xr[k].a = *reinterpret_cast<const uint4 *>(x + turn.a);
                xr[k].b = *reinterpret_cast<const uint4 *>(x + turn.b);
            }
            if (BWD) {
                const T *y = DY + go + (long long)h * r.gh;
                gr[k].a = *reinterpret_cast<const uint4 *>(y + turn.a);
                gr[k].b = *reinterpret_cast<const uint4 *>(y + turn.b);
            }
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            xr[k].a = xr[k].b = make_uint4(0, 0, 0, 0);
            if (BWD) gr[k].a = gr[k].b = make_uint4(0, 0, 0, 0);
            fetch(k, h0 + k);
        }
        for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (h + k >= h1) break;  // the same for all lanes
                float v[2 * V];
                unpack<T>(xr[k].a, v);
                unpack<T>(xr[k].b, v + V);
                float z[BWD ? 2 * V : 1];
                if (BWD) {
                    unpack<T>(gr[k].a, z);
                    unpack<T>(gr[k].b, z + V);
                }
                if (kRefill) fetch(k, h + k + kAhead);
                float rs = 1.f;
                if (p.norm) {
                    float q = 0.f;
#pragma unroll
                    for (int j = 0; j < 2 * V; ++j) q = fmaf(v[j], v[j], q);
                    rs = rsqrtf(fmaf(group_sum(q, tpr), inv_d, p.eps));
                }
                if (!BWD) {
                    if (p.norm) {
#pragma unroll
                        for (int j = 0; j < 2 * V; ++j) v[j] = v[j] * rs * w[j];
                    }
                    turn.apply(p, v, 1.f, row);
                } else {
                    turn.apply(p, z, -1.f, row);
                    if (p.norm) {
                        float q = 0.f;
#pragma unroll
                        for (int j = 0; j < 2 * V; ++j) {
                            v[j] *= rs;                       // xhat
                            if (live) dw[j] = fmaf(z[j], v[j], dw[j]);
                            z[j] *= w[j];
                            q = fmaf(z[j], v[j], q);
                        }
                        q = group_sum(q, tpr) * inv_d;
#pragma unroll
                        for (int j = 0; j < 2 * V; ++j) v[j] = rs * (z[j] - v[j] * q);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2 * V; ++j) v[j] = z[j];
                    }
                }
                if (live) {
                    T *y = Y + yo + (long long)(h + k) * r.yh;
                    store_chunk(y + turn.a, v);
                    store_chunk(y + turn.b, v + V);
                }
            }
            if (!kRefill) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) fetch(k, h + k + kAhead);
            }
        }
    }
    if (BWD && r.part) {
        __syncthreads();
        float *acc = sh + (size_t)g * p.d;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[turn.a + j] = dw[j], acc[turn.b + j] = dw[V + j];
        __syncthreads();
        for (int e = threadIdx.x; e < p.d; e += kThreads) {
            float s = 0.f;
            for (int q = 0; q < per_block; ++q) s += sh[(size_t)q * p.d + e];
            r.part[(size_t)block * p.d + e] = s;
        }
    }
}

// dweight[e] = sum over the blocks' sums: 4 columns of one tensor per CTA, 64 runs of blocks each added
// in order, then the runs in order.  Bound by the latency of a run's loads, of which eight are in
// flight.
__global__ void __launch_bounds__(256)
norm_weight_kernel(const float *part0, int blocks0, void *out0, const float *part1, int blocks1, void *out1, int d, int f32) {
    __shared__ float run[64][4];
    grid_dependency_wait();
    grid_dependents_launch();
    const float *part = blockIdx.y ? part1 : part0;
    void *out = blockIdx.y ? out1 : out0;
    const int blocks = blockIdx.y ? blocks1 : blocks0;
    if (!out) return;
    const int e = blockIdx.x * 4 + (threadIdx.x & 3), q = threadIdx.x >> 2;
    const int each = (blocks + 63) / 64, from = min(q * each, blocks), to = min(from + each, blocks);
    float s = 0.f;
    for (int b = from; b < to; b += 8) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = b + k < to ? part[(size_t)(b + k) * d + e] : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += x[k];
    }
    run[q][threadIdx.x & 3] = s;
    __syncthreads();
    if (q == 0) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < 64; ++k) a += run[k][threadIdx.x];
        if (f32) reinterpret_cast<float *>(out)[e] = a;
        else reinterpret_cast<__nv_bfloat16 *>(out)[e] = __float2bfloat16_rn(a);
    }
}

template <typename T>
cudaError_t launch(const Params &p, int mode, bool bwd, cudaStream_t stream) {
    const int blocks = p.r[0].blocks + p.r[1].blocks;
    const int per_block = kThreads / (p.d / (2 * kV<T>));
    const size_t smem = std::max(mode == kOddHalves ? (size_t)per_block * (p.d + 4) * 4 : (size_t)0,
                                 bwd ? (size_t)per_block * p.d * 4 : (size_t)0);
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(blocks), dim3(kThreads), smem, stream, p); };
    if (bwd) {
        return mode == kHalves       ? go(norm_rope_kernel<T, kHalves, true>)
               : mode == kNeighbours ? go(norm_rope_kernel<T, kNeighbours, true>)
                                     : go(norm_rope_kernel<T, kOddHalves, true>);
    }
    return mode == kHalves       ? go(norm_rope_kernel<T, kHalves, false>)
           : mode == kNeighbours ? go(norm_rope_kernel<T, kNeighbours, false>)
                                 : go(norm_rope_kernel<T, kOddHalves, false>);
}

bool finite_not_negative(float x) { return isfinite(x) && x >= 0.f; }

// The checks of one tensor, and its part of the launch.
anchor_attn_status_t check_rows(const anchor_attn_rope_t &how, const anchor_attn_rows_t &t, bool bwd, int tensors, Rows &r, View *in,
                                int &nin, View *out, int &nout) {
    if (t.B < 0 || t.heads < 0 || t.n < 0 || t.positions_batch < 0) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (t.dweight && (!bwd || !how.norm)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    const int es = how.dtype ? 4 : 2, ws = how.weight_f32 ? 4 : es;
    if (((uintptr_t)t.weight | (uintptr_t)t.dweight) & (ws - 1)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    r = Rows{};
    if (t.B == 0 || t.heads == 0 || t.n == 0) return ANCHOR_ATTN_OK;
    if ((long long)t.B * t.n > 0x7fffffffLL - kThreads || t.heads > 1 << 20) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (t.positions && ((uintptr_t)t.positions & (how.positions64 ? 7u : 3u))) return ANCHOR_ATTN_ERR_INVALID_ARG;
    auto view = [&](const anchor_attn_view_t &v) { return make_view(v, t.B, t.heads, t.n, how.d, es); };
    const bool reads_x = !bwd || how.norm;
    const View x = reads_x ? view(t.X) : View{}, g = bwd ? view(t.dY) : View{}, y = view(bwd ? t.dX : t.Y);
    anchor_attn_status_t st = check_view(y, true);
    if (st == ANCHOR_ATTN_OK && reads_x) st = check_view(x, false);
    if (st == ANCHOR_ATTN_OK && bwd) st = check_view(g, false);
    if (st != ANCHOR_ATTN_OK) return st;
    if (reads_x) in[nin++] = x;
    if (bwd) in[nin++] = g;
    out[nout++] = y;
    r.x = x.ptr, r.dy = g.ptr, r.y = (void *)y.ptr, r.w = t.weight, r.pos = how.rot ? t.positions : nullptr;
    r.xb = x.sb, r.xh = x.sh, r.xn = x.sn, r.yb = y.sb, r.yh = y.sh, r.yn = y.sn, r.gb = g.sb, r.gh = g.sh, r.gn = g.sn;
    r.pos_batch = t.positions_batch, r.start = t.start;
    r.heads = t.heads, r.n = t.n, r.tokens = t.B * t.n;
    // One group of heads walks all of them where the tokens alone make kFill blocks; fewer tokens
    // cut the heads, down to one a thread (the sines are then made once for each group).
    const int per_block = kThreads / (how.d / (2 * (16 / es)));
    r.token_blocks = (int)(((long long)r.tokens + per_block - 1) / per_block);
    r.groups = std::min(r.heads, std::max(1, kFill / r.token_blocks));
    r.heads_per = (r.heads + r.groups - 1) / r.groups;
    r.groups = (r.heads + r.heads_per - 1) / r.heads_per;
    if (t.dweight) {
        const int most = how.dtype ? kBwdBlocks32 : kBwdBlocks16 / tensors;
        r.token_blocks = std::min(r.token_blocks, std::max(1, most / r.groups));
    }
    if ((long long)r.token_blocks * r.groups > 0x3fffffffLL) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    r.blocks = r.token_blocks * r.groups;
    return ANCHOR_ATTN_OK;
}

anchor_attn_status_t norm_rope(const anchor_attn_rope_t *how, const anchor_attn_rows_t *first,
                               const anchor_attn_rows_t *second, bool bwd, void *stream_v) {
    if (!how || !first) return ANCHOR_ATTN_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_v;
    const anchor_attn_rope_t &a = *how;
    auto flag = [](int v) { return v == 0 || v == 1; };
    if (!flag(a.dtype) || !flag(a.interleaved) || !flag(a.norm) || !flag(a.weight_f32) || !flag(a.positions64))
        return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (a.d != 16 && a.d != 32 && a.d != 64 && a.d != 128) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (a.rot < 0 || a.rot > a.d || a.rot % 2 || a.axes < 1 || a.axes > 3) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (!finite_not_negative(a.eps) || !isfinite(a.magnitude)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (a.rot && (!a.phases || ((uintptr_t)a.phases & 7u))) return ANCHOR_ATTN_ERR_INVALID_ARG;

    Params p = {};
    View in[4], out[2];
    int nin = 0, nout = 0;
    const anchor_attn_rows_t *t[2] = {first, second};
    for (int i = 0; i < 2; ++i) {
        if (!t[i]) continue;
        const anchor_attn_status_t st = check_rows(a, *t[i], bwd, second ? 2 : 1, p.r[i], in, nin, out, nout);
        if (st != ANCHOR_ATTN_OK) return st;
    }
    // an output may be its own tensor's X (forward): a row is read whole before it is written
    const int es = a.dtype ? 4 : 2;
    const size_t wbytes = (size_t)a.d * (a.weight_f32 ? 4 : es);
    for (int o = 0; o < nout; ++o) {
        for (int k = 0; k < nin; ++k)
            if (!(!bwd && k == o && out[o].same(in[k])) && views_overlap(out[o], in[k])) return ANCHOR_ATTN_ERR_ALIAS;
        if (o == 1 && views_overlap(out[0], out[1])) return ANCHOR_ATTN_ERR_ALIAS;
        for (const anchor_attn_rows_t *q : t) {
            if (!q) continue;
            const View &v = out[o];
            if (q->weight && bytes_overlap(v.ptr, (size_t)v.extent(), q->weight, wbytes)) return ANCHOR_ATTN_ERR_ALIAS;
            if (q->dweight && bytes_overlap(v.ptr, (size_t)v.extent(), q->dweight, wbytes)) return ANCHOR_ATTN_ERR_ALIAS;
            if (a.rot && bytes_overlap(v.ptr, (size_t)v.extent(), a.phases, (size_t)a.axes * a.rot / 2 * 8))
                return ANCHOR_ATTN_ERR_ALIAS;
            if (a.rot && q->positions && q->n > 0 && q->B > 0 &&
                bytes_overlap(v.ptr, (size_t)v.extent(), q->positions,
                              ((size_t)(q->B - 1) * q->positions_batch + (size_t)q->n * a.axes) * (a.positions64 ? 8 : 4)))
                return ANCHOR_ATTN_ERR_ALIAS;
        }
    }
    for (int i = 0; i < 2; ++i) {
        if (!t[i] || !t[i]->dweight) continue;
        for (int k = 0; k < nin; ++k)
            if (bytes_overlap(t[i]->dweight, wbytes, in[k].ptr, (size_t)in[k].extent())) return ANCHOR_ATTN_ERR_ALIAS;
        for (const anchor_attn_rows_t *q : t)
            if (q && q->weight && bytes_overlap(t[i]->dweight, wbytes, q->weight, wbytes)) return ANCHOR_ATTN_ERR_ALIAS;
        if (i == 1 && first->dweight && bytes_overlap(first->dweight, wbytes, second->dweight, wbytes))
            return ANCHOR_ATTN_ERR_ALIAS;
    }
    p.phases = reinterpret_cast<const unsigned long long *>(a.phases);
    p.d = a.d, p.rot = a.rot, p.axes = a.axes, p.norm = a.norm, p.w_f32 = a.weight_f32 || a.dtype, p.pos64 = a.positions64;
    p.eps = a.eps, p.magnitude = a.magnitude;
    const int V = 16 / es;
    const int mode = a.interleaved                                              ? kNeighbours
                     : (a.rot / 2) % V == 0 && ((a.d - a.rot) / 2) % V == 0 ? kHalves
                                                                                : kOddHalves;
    float *ws = nullptr;
    bool sums = false;
    for (int i = 0; i < 2; ++i) {
        if (!t[i] || !t[i]->dweight) continue;
        if (p.r[i].blocks) {
            sums = true;
        } else if (cudaMemsetAsync(t[i]->dweight, 0, wbytes, stream) != cudaSuccess) {
            cudaGetLastError();
            return ANCHOR_ATTN_ERR_CUDA;
        }
    }
    if (p.r[0].blocks + p.r[1].blocks == 0) return ANCHOR_ATTN_OK;
    cudaError_t e = cudaSuccess;
    if (sums) {
        if (getenv("ANCHOR_ATTN_TEST_FAIL_ALLOC") != nullptr) return ANCHOR_ATTN_ERR_ALLOC;
        const size_t bytes = (size_t)(p.r[0].blocks + p.r[1].blocks) * a.d * 4;
        if (workspace_alloc((void **)&ws, bytes, stream) != cudaSuccess) {
            cudaGetLastError();
            return ANCHOR_ATTN_ERR_ALLOC;
        }
        for (int i = 0; i < 2; ++i)
            if (t[i] && t[i]->dweight && p.r[i].blocks) p.r[i].part = ws + (i ? (size_t)p.r[0].blocks * a.d : 0);
    }
    e = a.dtype ? launch<float>(p, mode, bwd, stream) : launch<__nv_bfloat16>(p, mode, bwd, stream);
    if (sums) {
        if (e == cudaSuccess)
            e = launch_pdl(norm_weight_kernel, dim3(a.d / 4, 2), dim3(256), 0, stream, (const float *)p.r[0].part,
                           p.r[0].blocks, p.r[0].part ? first->dweight : nullptr, (const float *)p.r[1].part, p.r[1].blocks,
                           p.r[1].part ? second->dweight : nullptr, a.d, p.w_f32);
        const cudaError_t ef = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess) e = ef;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return ANCHOR_ATTN_ERR_CUDA;
    }
    return ANCHOR_ATTN_OK;
}

}  // namespace
}  // namespace anchor

extern "C" {

anchor_attn_status_t anchor_attn_norm_rope(const anchor_attn_rope_t *how, const anchor_attn_rows_t *first,
                                           const anchor_attn_rows_t *second, void *stream) {
    return anchor::norm_rope(how, first, second, false, stream);
}

anchor_attn_status_t anchor_attn_norm_rope_backward(const anchor_attn_rope_t *how, const anchor_attn_rows_t *first,
                                                    const anchor_attn_rows_t *second, void *stream) {
    return anchor::norm_rope(how, first, second, true, stream);
}

}  // extern "C"
