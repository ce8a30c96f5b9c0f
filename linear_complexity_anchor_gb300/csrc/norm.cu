// The RMS norm of a residual sum, with a result in the rows' type or in 8 bits with scales, and its
// backward (formulas and layout in include/anchor_attn.h).
//
// All of them are bound by memory: a row is read once, kept in registers, and written once. T threads
// hold a row, NC chunks of 8 neighbouring columns each, chunk c of thread t at column 8 (c T + t), so that
// a warp's loads are contiguous and the threads of a scale's group of columns are neighbours in a warp.
// Rows of up to 2048 columns (backward: 1024, whose registers end there) belong to a warp, which needs no barrier; longer ones
// to a block.  (bf16, 8 bits: 65536 x 1024 by a warp 73 us, by four 86; 65536 x 2048 139, by eight 170; in 16 bits the
// same to 1 %.  Backward: 65536 x 1024 93, by four 94; 65536 x 2048 by a warp 1236, by eight 178.)  65536 x 2048 in 8 bits:
// 138 us, 6.8 TB/s; 33600 x 768 backward: 40 us with the second launch, 5.2 TB/s.  (fp32, the same layouts: forward 32768 x 1024 81 us,
// 6.6 TB/s, 16384 x 2048 83; backward with ds and dw 32768 x 768 69 us, 5.8 TB/s, x 1024 102, 5.3, where a warp's columns do not fit its registers, x 1040
// 104, 16384 x 2048 86, 6.2, 4096 x 8192 96, 3000 x 16384 158, 5.0, which do not fit either.  bf16: 65536 x 1024 108 us, 5.0 TB/s, x 1040 159, 3.4:
// 130 of a block's 256 threads have columns; 6000 x 16384 166, 4.8.)
//
// Backward: xhat = s r, r = 1 / sqrt(mean s^2 + eps):
//   dx = r (w o dy - xhat mean(w o dy o xhat)) + ds,  dw += dy o xhat.
// dw: a thread sums its columns over the rows that it walks, the block adds its rows' threads in order, and a
// second launch adds the blocks in order; the grid depends on the shapes alone, so the bits do too.
#include "cross.cuh"
#include "ptx.cuh"

#include <cuda_fp8.h>
#include <math.h>
#include <stdlib.h>

namespace anchor {
namespace {

constexpr float kTop = 448.f;  // the largest e4m3 number

struct Rows {
    long long sb, sn;  // strides of a batch entry and a row, in elements
    void *ptr;
};

struct NormParams {
    Rows x, r, s, y, dy, ds, dx;
    const void *weight;
    float *scales;  // [rows][groups]
    float *part;    // backward: the blocks' dweight sums [blocks][D], or null
    int rows, n, D, groups;
    Divide by_n;
    float eps, inv_d;
    int w_f32;
};

template <typename T> __device__ __forceinline__ T *row_of(const NormParams &p, const Rows &v, int row) {
    const int b = p.by_n.of(row), i = row - b * p.n;
    return (T *)v.ptr + b * v.sb + (long long)i * v.sn;
}

// eight columns
struct Raw16 { uint4 a; };
struct Raw32 { uint4 a, b; };
template <typename T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> { using type = Raw16; };
template <> struct RawOf<float> { using type = Raw32; };
template <typename T> using Raw = typename RawOf<T>::type;

__device__ __forceinline__ Raw16 fetch(const __nv_bfloat16 *p) { return Raw16{*reinterpret_cast<const uint4 *>(p)}; }
__device__ __forceinline__ Raw32 fetch(const float *p) {
    return Raw32{reinterpret_cast<const uint4 *>(p)[0], reinterpret_cast<const uint4 *>(p)[1]};
}
__device__ __forceinline__ void unpack(const Raw16 &r, float *v) {
    const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw32 &r, float *v) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ Raw16 pack(const float *v, const __nv_bfloat16 *) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return Raw16{make_uint4(u[0], u[1], u[2], u[3])};
}
__device__ __forceinline__ Raw32 pack(const float *v, const float *) {
    const uint4 *u = reinterpret_cast<const uint4 *>(v);
    return Raw32{u[0], u[1]};
}
__device__ __forceinline__ void put(__nv_bfloat16 *p, const Raw16 &r) { *reinterpret_cast<uint4 *>(p) = r.a; }
__device__ __forceinline__ void put(float *p, const Raw32 &r) {
    reinterpret_cast<uint4 *>(p)[0] = r.a;
    reinterpret_cast<uint4 *>(p)[1] = r.b;
}

template <typename T>
__device__ __forceinline__ void load_weight(const NormParams &p, int e, float *w) {
    if (!p.weight) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
    } else if (p.w_f32) {
        unpack(fetch((const float *)p.weight + e), w);
    } else {
        unpack(fetch((const T *)p.weight + e), w);
    }
}

// the larger one, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
struct Sum {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
};

// v over a row's T threads; `slots`: T / 32 numbers of the block's, free before the call for T > 32
template <int T, typename Op>
__device__ __forceinline__ float over_row(float v, Op op, float *slots) {
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (T > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) slots[warp] = v;
        __syncthreads();
        v = slots[lane % (T / 32)];
#pragma unroll
        for (int o = T / 64; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    return v;
}

// Rows whose squares leave fp32's range: mean s^2 + eps is not above 2^-100 (squares below 2^-126 have lost bits) or not finite.  They are
// summed again, scaled by a power of two, 2^100 (numbers below 2^-43 by then) or 2^-72: both leave room for 16384 squares.  One test a
// row, and a branch that ordinary rows do not take.
struct Far {
    bool odd;
    float scale;
    __device__ __forceinline__ explicit Far(float mean) : odd(!(mean > 0x1p-100f && mean < INFINITY)), scale(!odd ? 1.f : mean < 1.f ? 0x1p100f : 0x1p-72f) {}
    // 1 / sqrt(mean + eps) of the scaled numbers, from the sum of their squares: 0 for a row of zeros and eps = 0
    __device__ __forceinline__ float root(float sum, float inv_d, float eps) const {
        const float mean = fmaf(sum, inv_d, eps * scale * scale);
        return mean == 0.f ? 0.f : rsqrtf(mean);
    }
};

// Threads of a block: a long row's, or those of several rows.
template <int T> constexpr int kBlock = T > 32 ? T : 128;

// BITS8: GROUP columns share a scale (0: the row).  Five blocks an SM where a thread holds 64 columns of bf16 (65536 x 1040 in 8 bits, scales
// of 128 columns: 109 us, 16 bytes spilt; four, with two registers a thread more: 122).
template <typename T, int TPR, int NC, bool BITS8, int GROUP>
__global__ void __launch_bounds__(kBlock<TPR>, NC == 8 && sizeof(T) == 2 ? 5 : 0) add_norm_kernel(const NormParams p) {
    __shared__ float slots[2][TPR > 32 ? TPR / 32 : 1];
    grid_dependency_wait();
    grid_dependents_launch();
    const int t = threadIdx.x % TPR;
    const int row = (int)(blockIdx.x * (kBlock<TPR> / TPR) + threadIdx.x / TPR);
    const bool live = row < p.rows;  // (a row of a block's own always exists)
    float v[NC][8];
    {
        Raw<T> x[NC], r[NC];
        const T *xp = live ? row_of<const T>(p, p.x, row) : nullptr, *rp = live && p.r.ptr ? row_of<const T>(p, p.r, row) : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = 8 * (c * TPR + t);
            x[c] = r[c] = Raw<T>{};
            if (live && e < p.D) {
                x[c] = fetch(xp + e);
                if (rp) r[c] = fetch(rp + e);
            }
        }
        T *sp = rp ? row_of<T>(p, p.s, row) : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            unpack(x[c], v[c]);
            if (rp) {
                // the norm is that of the sum as it is kept
                float a[8];
                unpack(r[c], a);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] += a[i];
                const Raw<T> s = pack(v[c], (const T *)nullptr);
                unpack(s, v[c]);
                const int e = 8 * (c * TPR + t);
                if (e < p.D) put(sp + e, s);
            }
        }
    }
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(v[c][i], v[c][i], q);
    q = fmaf(over_row<TPR>(q, Sum(), slots[0]), p.inv_d, p.eps);
    float rs = rsqrtf(q);
    const Far far(q);
    if (__any_sync(0xffffffffu, far.odd)) {  // (the same for all warps of a row)
        q = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = v[c][i] * far.scale;
                q = fmaf(x, x, q);
                if (far.scale > 1.f) v[c][i] = x;  // (1 / sqrt of the smallest numbers is none of fp32)
            }
        if (TPR > 32) __syncthreads();  // the slots are free again
        rs = far.root(over_row<TPR>(q, Sum(), slots[0]), p.inv_d, p.eps) * fminf(far.scale, 1.f);
    }
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int e = 8 * (c * TPR + t);
        if (e >= p.D) continue;
        float w[8];
        load_weight<T>(p, e, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * rs * w[i];
        if constexpr (!BITS8) {
            if (live) put(row_of<T>(p, p.y, row) + e, pack(v[c], (const T *)nullptr));
        } else if (GROUP == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(v[c][i]));
        }
    }
    if constexpr (BITS8) {
        if (GROUP == 0) top = over_row<TPR>(top, Max(), slots[1]);
        unsigned char *yp = live ? row_of<unsigned char>(p, p.y, row) : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = 8 * (c * TPR + t);
            const bool in = live && e < p.D;
            if (GROUP > 0) {
                top = 0.f;
                if (in)
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(v[c][i]));
#pragma unroll
                for (int o = (GROUP / 8 < TPR ? GROUP / 8 : TPR) / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            if (!in) continue;
            // y / scale as y (448 / top): two roundings of fp32, where the result has half a step of 2^-4.
            // A tiny top is lifted first, so that its reciprocal exists.
            const float up = top < 0x1p-100f ? 0x1p100f : 1.f, inv = top == 0.f ? 0.f : __fdiv_rn(kTop, top * up);
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[c][2 * i] * up * inv, v[c][2 * i + 1] * up * inv), __NV_SATFINITE, __NV_E4M3);
            *reinterpret_cast<uint2 *>(yp + e) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
            const float scale = __fdiv_rn(top, kTop);
            if (GROUP == 0 ? e == 0 : e % (GROUP ? GROUP : 1) == 0) p.scales[(long long)row * p.groups + (GROUP ? e / GROUP : 0)] = scale;
        }
    }
}

// Backward.  A block's rows are index, index + blocks, ...; each thread keeps its columns' dw and weights.  Short rows: sixteen
// at a time, so that few blocks' sums are left to be added.  16-bit rows are bound by instructions as much as by memory, so two
// columns go in one where they can (33600 x 768: 47 -> 40 us), and a row is unpacked once.
template <int T> constexpr int kBackBlock = T > 32 ? T : 512;
constexpr int kWays = 4;

// four pairs of columns
__device__ __forceinline__ void unpack2(const Raw16 &r, uint64_t *v) {
    const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ptx::f32x2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack2(const Raw32 &r, uint64_t *v) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ptx::f32x2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
}
__device__ __forceinline__ float sum2(uint64_t v) {
    float a, b;
    ptx::f32x2_split(v, a, b);
    return a + b;
}

template <typename T, int TPR, int NC>
__global__ void __launch_bounds__(kBackBlock<TPR>) add_norm_backward_kernel(const NormParams p) {
    using namespace ptx;
    constexpr int kRows = kBackBlock<TPR> / TPR;
    // weights, and what a row is unpacked to, stay in registers where they fit
    constexpr bool kKeep = NC <= (sizeof(T) == 2 ? 3 : 2);
    __shared__ float2 both[2][TPR > 32 ? TPR / 32 : 1];
    extern __shared__ float sum[];  // [kWays][D] where kRows > 1
    grid_dependency_wait();
    grid_dependents_launch();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    uint64_t dw2[NC][4], w_kept[kKeep ? NC : 1][4];
    auto weights = [&](int c, uint64_t *w2) {
        const int e = 8 * (c * TPR + t);
        float w[8] = {};
        if (e < p.D) load_weight<T>(p, e, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w2[i] = f32x2(w[2 * i], w[2 * i + 1]);
    };
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dw2[c][i] = 0ull;
        if constexpr (kKeep) weights(c, w_kept[c]);
    }
    int turn = 0;
    // (all threads of a block make the same number of steps)
    for (long long base = (long long)blockIdx.x * kRows; base < p.rows; base += (long long)gridDim.x * kRows, turn ^= 1) {
        const bool live = base + g < p.rows;
        const int row = live ? (int)(base + g) : 0;
        Raw<T> s[NC], y[NC], d[NC];
        const T *sp = row_of<const T>(p, p.s, row), *yp = row_of<const T>(p, p.dy, row), *dp = p.ds.ptr ? row_of<const T>(p, p.ds, row) : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = 8 * (c * TPR + t);
            s[c] = y[c] = d[c] = Raw<T>{};
            if (live && e < p.D) {
                s[c] = fetch(sp + e);
                y[c] = fetch(yp + e);
                if (dp) d[c] = fetch(dp + e);
            }
        }
        // sums of s^2 and of w dy s together: mean(w dy xhat) = r mean(w dy s)
        uint64_t a_kept[kKeep ? NC : 1][4], q2 = 0ull, z2 = 0ull;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            uint64_t b[4], w_here[4], *a = a_kept[kKeep ? c : 0], *w2 = kKeep ? w_kept[kKeep ? c : 0] : w_here;
            unpack2(s[c], a);
            unpack2(y[c], b);
            if constexpr (!kKeep) weights(c, w2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q2 = fma_f32x2(a[i], a[i], q2);
                z2 = fma_f32x2(mul_f32x2(a[i], w2[i]), b[i], z2);
            }
        }
        float q, z;
        auto total = [&](float q_here, float z_here, bool again) {
            q = q_here, z = z_here;
#pragma unroll
            for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
                q += __shfl_xor_sync(0xffffffffu, q, o);
                z += __shfl_xor_sync(0xffffffffu, z, o);
            }
            if (TPR > 32) {
                // both through one barrier; a step's slots are free again behind the next step's barrier
                if (again) __syncthreads();
                if ((threadIdx.x & 31) == 0) both[turn][threadIdx.x >> 5] = make_float2(q, z);
                __syncthreads();
                const float2 o2 = both[turn][(threadIdx.x & 31) % (TPR > 32 ? TPR / 32 : 1)];
                q = o2.x, z = o2.y;
#pragma unroll
                for (int o = TPR / 64; o > 0; o >>= 1) {
                    q += __shfl_xor_sync(0xffffffffu, q, o);
                    z += __shfl_xor_sync(0xffffffffu, z, o);
                }
            }
        };
        total(sum2(q2), sum2(z2), false);
        const float size = fmaf(q, p.inv_d, p.eps);
        float rs = rsqrtf(size), mean = -z * rs * p.inv_d;
        const Far far(size);
        if (__any_sync(0xffffffffu, far.odd)) {
            const uint64_t scale2 = f32x2(far.scale, far.scale);
            q2 = z2 = 0ull;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                uint64_t a[4], b[4], w_here[4], *w2 = kKeep ? w_kept[kKeep ? c : 0] : w_here;
                unpack2(s[c], a);
                unpack2(y[c], b);
                if constexpr (!kKeep) weights(c, w2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t x = mul_f32x2(a[i], scale2);
                    q2 = fma_f32x2(x, x, q2);
                    z2 = fma_f32x2(mul_f32x2(x, w2[i]), b[i], z2);
                }
            }
            total(sum2(q2), sum2(z2), true);
            // (of the warp's other rows these are the same numbers again)
            rs = far.root(q, p.inv_d, p.eps);
            if (far.scale > 1.f && rs > 0x1.fffffep27f) rs = 0x1.fffffep27f;  // (FLT_MAX / scale: 1 / sqrt counts as the largest number)
            mean = -z * rs * p.inv_d;
            rs *= far.scale;
        }
        const uint64_t rs2 = f32x2(rs, rs), mean2 = f32x2(mean, mean);
        T *xp = row_of<T>(p, p.dx, row);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = 8 * (c * TPR + t);
            if (e >= p.D || !live) continue;
            uint64_t b[4], o2[4], w_here[4], *a = a_kept[kKeep ? c : 0], *w2 = kKeep ? w_kept[kKeep ? c : 0] : w_here;
            float o[8];
            if constexpr (!kKeep) unpack2(s[c], a), weights(c, w2);
            unpack2(y[c], b);
            unpack2(d[c], o2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t hat = mul_f32x2(a[i], rs2);
                dw2[c][i] = fma_f32x2(b[i], hat, dw2[c][i]);
                f32x2_split(fma_f32x2(rs2, fma_f32x2(hat, mean2, mul_f32x2(w2[i], b[i])), o2[i]), o[2 * i], o[2 * i + 1]);
            }
            put(xp + e, pack(o, (const T *)nullptr));
        }
    }
    float dw[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) f32x2_split(dw2[c][i], dw[c][2 * i], dw[c][2 * i + 1]);
    if (!p.part) return;
    float *part = p.part + (size_t)blockIdx.x * p.D;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = 8 * (c * TPR + t);
            if (e < p.D) put(part + e, pack(dw[c], (const float *)nullptr));
        }
    } else {
        // by four ways, each a quarter of the rows in order, then the ways in order
        constexpr int kEach = kRows / kWays;
        float *mine = sum + g / kEach * p.D;
        for (int k = 0; k < kEach; ++k) {
            if (g % kEach == k) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int e = 8 * (c * TPR + t);
                    if (e >= p.D) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i) mine[e + i] = k > 0 ? mine[e + i] + dw[c][i] : dw[c][i];
                }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < p.D; e += kBackBlock<TPR>) {
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < kWays; ++k) a += sum[k * p.D + e];
            part[e] = a;
        }
    }
}

// dweight[e] = sum over the blocks' sums: 32 columns a CTA, 32 runs of blocks each added in order, then the
// runs in order.  Bound by the latency of a run's loads, of which eight are in flight.
__global__ void __launch_bounds__(1024) add_norm_weight_kernel(const float *part, int blocks, void *out, int D, int f32) {
    __shared__ float run[32][33];
    grid_dependency_wait();
    grid_dependents_launch();
    const int x = threadIdx.x & 31, q = threadIdx.x >> 5, e = blockIdx.x * 32 + x;
    const int each = (blocks + 31) / 32, from = min(q * each, blocks), to = min(from + each, blocks);
    float s = 0.f;
    if (e < D) {
        for (int b = from; b < to; b += 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = b + k < to ? part[(size_t)(b + k) * D + e] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    }
    run[q][x] = s;
    __syncthreads();
    if (q == 0 && e < D) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) a += run[k][x];
        if (f32) reinterpret_cast<float *>(out)[e] = a;
        else reinterpret_cast<__nv_bfloat16 *>(out)[e] = __float2bfloat16_rn(a);
    }
}

template <typename T, int TPR, int NC>
cudaError_t forward(const NormParams &p, int bits8, int group, cudaStream_t stream) {
    constexpr int kRows = kBlock<TPR> / TPR;
    const dim3 grid((unsigned)(((long long)p.rows + kRows - 1) / kRows));
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kBlock<TPR>), 0, stream, p); };
    if (!bits8) return go(add_norm_kernel<T, TPR, NC, false, 0>);
    return group == 0    ? go(add_norm_kernel<T, TPR, NC, true, 0>)
           : group == 32 ? go(add_norm_kernel<T, TPR, NC, true, 32>)
           : group == 64 ? go(add_norm_kernel<T, TPR, NC, true, 64>)
                         : go(add_norm_kernel<T, TPR, NC, true, 128>);
}

template <typename T>
cudaError_t forward(const NormParams &p, int bits8, int group, cudaStream_t stream) {
    const int D = p.D;
    return D <= 64      ? forward<T, 8, 1>(p, bits8, group, stream)
           : D <= 256   ? forward<T, 32, 1>(p, bits8, group, stream)
           : D <= 512   ? forward<T, 32, 2>(p, bits8, group, stream)
           : D <= 768   ? forward<T, 32, 3>(p, bits8, group, stream)
           : D <= 1024  ? forward<T, 32, 4>(p, bits8, group, stream)
           : D <= 2048  ? forward<T, 32, 8>(p, bits8, group, stream)
           : D <= 4096  ? forward<T, 256, 2>(p, bits8, group, stream)
           : D <= 8192  ? forward<T, 512, 2>(p, bits8, group, stream)
                        : forward<T, 512, 4>(p, bits8, group, stream);
}

template <typename T, int TPR, int NC>
cudaError_t backward(const NormParams &p, int blocks, cudaStream_t stream) {
    const size_t smem = kBackBlock<TPR> > TPR && p.part ? (size_t)kWays * p.D * 4 : 0;
    return launch_pdl(add_norm_backward_kernel<T, TPR, NC>, dim3(blocks), dim3(kBackBlock<TPR>), smem, stream, p);
}

template <typename T>
cudaError_t backward(const NormParams &p, int blocks, cudaStream_t stream) {
    const int D = p.D;
    return D <= 64      ? backward<T, 8, 1>(p, blocks, stream)
           : D <= 256   ? backward<T, 32, 1>(p, blocks, stream)
           : D <= 512   ? backward<T, 32, 2>(p, blocks, stream)
           : D <= 768   ? backward<T, 32, 3>(p, blocks, stream)
           : D <= 1024  ? backward<T, 32, 4>(p, blocks, stream)
           : D <= 2048  ? backward<T, 256, 1>(p, blocks, stream)
           : D <= 4096  ? backward<T, 256, 2>(p, blocks, stream)
           : D <= 8192  ? backward<T, 512, 2>(p, blocks, stream)
                        : backward<T, 512, 4>(p, blocks, stream);
}
// Rows that a block of the backward holds at a time, and blocks an SM, for D columns.
int backward_rows(int D) { return D <= 64 ? kBackBlock<8> / 8 : D <= 1024 ? kBackBlock<32> / 32 : 1; }
int backward_blocks(int D) { return D <= 256 ? 2 : D <= 1024 ? 1 : D <= 2048 ? 4 : D <= 4096 ? 2 : 1; }

anchor_attn_status_t add_norm(const anchor_attn_add_norm_t *a, bool bwd, void *stream_v) {
    if (!a) return ANCHOR_ATTN_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_v;
    auto flag = [](int v) { return v == 0 || v == 1; };
    if (!flag(a->dtype) || !flag(a->weight_f32) || !flag(a->bits8) || a->B < 0 || a->n < 0) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (a->D < 16 || a->D > 16384 || a->D % 16) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (!(isfinite(a->eps) && a->eps >= 0.f) || (bwd && a->bits8) || (!bwd && a->dweight)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    const int es = a->dtype ? 4 : 2;
    const size_t wbytes = (size_t)a->D * (a->weight_f32 ? 4 : es);
    if (((uintptr_t)a->weight & 15u) || ((uintptr_t)a->dweight & 3u) || ((uintptr_t)a->scales & 3u)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (a->B == 0 || a->n == 0) {
        if (a->dweight && cudaMemsetAsync(a->dweight, 0, wbytes, stream) != cudaSuccess) {
            cudaGetLastError();
            return ANCHOR_ATTN_ERR_CUDA;
        }
        return ANCHOR_ATTN_OK;
    }
    if ((long long)a->B * a->n > 0x7fffffffLL - 1024) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (!bwd && a->bits8 && !a->scales) return ANCHOR_ATTN_ERR_INVALID_ARG;
    NormParams p = {};
    p.rows = a->B * a->n, p.n = a->n, p.D = a->D, p.groups = a->group ? (a->D + a->group - 1) / a->group : 1;
    p.by_n = Divide((uint32_t)a->n), p.eps = a->eps, p.inv_d = 1.f / (float)a->D, p.w_f32 = a->weight_f32 || a->dtype;
    p.weight = a->weight, p.scales = a->scales;

    View in[3], out[2];
    int nin = 0, nout = 0;
    anchor_attn_status_t st = ANCHOR_ATTN_OK;
    auto add = [&](const anchor_attn_view_t &v, bool writes, int size, Rows &to) {
        if (st != ANCHOR_ATTN_OK) return;
        const View w = make_view(v, a->B, 1, a->n, a->D, size);
        st = check_view(w, writes);
        if (writes) out[nout++] = w;
        else in[nin++] = w;
        to = Rows{w.sb, w.sn, (void *)w.ptr};
    };
    if (!bwd) {
        add(a->X, false, es, p.x);
        if (a->R.ptr) {
            add(a->R, false, es, p.r);
            add(a->S, true, es, p.s);
        }
        add(a->Y, true, a->bits8 ? 1 : es, p.y);
    } else {
        add(a->S, false, es, p.s);
        add(a->dY, false, es, p.dy);
        if (a->dS.ptr) add(a->dS, false, es, p.ds);
        add(a->dX, true, es, p.dx);
    }
    if (st != ANCHOR_ATTN_OK) return st;
    // The sum may be written over X or R, and a gradient over dY or dS: a thread reads an element before it
    // writes it.
    const size_t scale_bytes = !bwd && a->bits8 ? (size_t)p.rows * p.groups * 4 : 0;
    for (int o = 0; o < nout; ++o) {
        const View &v = out[o];
        const bool over = bwd || (a->R.ptr && o == 0);
        for (int i = 0; i < nin; ++i)
            if (!(over && !(bwd && i == 0) && v.same(in[i])) && views_overlap(v, in[i])) return ANCHOR_ATTN_ERR_ALIAS;
        if (o == 1 && views_overlap(out[0], out[1])) return ANCHOR_ATTN_ERR_ALIAS;
        if (a->weight && bytes_overlap(v.ptr, (size_t)v.extent(), a->weight, wbytes)) return ANCHOR_ATTN_ERR_ALIAS;
        if (a->dweight && bytes_overlap(v.ptr, (size_t)v.extent(), a->dweight, wbytes)) return ANCHOR_ATTN_ERR_ALIAS;
        if (scale_bytes && bytes_overlap(v.ptr, (size_t)v.extent(), a->scales, scale_bytes)) return ANCHOR_ATTN_ERR_ALIAS;
    }
    for (int i = 0; i < nin; ++i) {
        if (a->dweight && bytes_overlap(in[i].ptr, (size_t)in[i].extent(), a->dweight, wbytes)) return ANCHOR_ATTN_ERR_ALIAS;
        if (scale_bytes && bytes_overlap(in[i].ptr, (size_t)in[i].extent(), a->scales, scale_bytes)) return ANCHOR_ATTN_ERR_ALIAS;
    }
    if (a->weight && a->dweight && bytes_overlap(a->weight, wbytes, a->dweight, wbytes)) return ANCHOR_ATTN_ERR_ALIAS;
    if (a->weight && scale_bytes && bytes_overlap(a->weight, wbytes, a->scales, scale_bytes)) return ANCHOR_ATTN_ERR_ALIAS;

    cudaError_t e = cudaSuccess;
    if (!bwd) {
        e = a->dtype ? forward<float>(p, a->bits8, a->group, stream) : forward<__nv_bfloat16>(p, a->bits8, a->group, stream);
    } else {
        const int held = backward_rows(a->D), most = kPlanSMs * backward_blocks(a->D);
        const int blocks = (int)std::min<long long>(((long long)p.rows + held - 1) / held, most);
        if (a->dweight) {
            if (getenv("ANCHOR_ATTN_TEST_FAIL_ALLOC") != nullptr) return ANCHOR_ATTN_ERR_ALLOC;
            if (workspace_alloc((void **)&p.part, (size_t)blocks * a->D * 4, stream) != cudaSuccess) {
                cudaGetLastError();
                return ANCHOR_ATTN_ERR_ALLOC;
            }
        }
        e = a->dtype ? backward<float>(p, blocks, stream) : backward<__nv_bfloat16>(p, blocks, stream);
        if (a->dweight) {
            if (e == cudaSuccess)
                e = launch_pdl(add_norm_weight_kernel, dim3((a->D + 31) / 32), dim3(1024), 0, stream, (const float *)p.part, blocks,
                               a->dweight, a->D, p.w_f32);
            const cudaError_t ef = cudaFreeAsync(p.part, stream);
            if (e == cudaSuccess) e = ef;
        }
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

anchor_attn_status_t anchor_attn_add_norm(const anchor_attn_add_norm_t *p, void *stream) { return anchor::add_norm(p, false, stream); }

anchor_attn_status_t anchor_attn_add_norm_backward(const anchor_attn_add_norm_t *p, void *stream) {
    return anchor::add_norm(p, true, stream);
}

}  // extern "C"
