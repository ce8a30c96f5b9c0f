// Cross attention in fp32 on CUDA cores, forward and backward (formulas in
// include/anchor_attn.h).
//
// Tiles of BM = 64, 32 or 16 rows by 64 columns.  Threads stand as 16 to a group of rows: one has TM
// rows (next to one another) and columns tx, tx + 16, tx + 32, tx + 48 of the scores, and TM rows by
// d / 16 columns of the outputs.  All tiles lie row by row in shared memory with a pitch of d + 4
// floats: 16-byte reads along d (scores) and along the columns (outputs) are then free of conflicts,
// and one copy serves both products.  What bounds it is those reads: at TM = 8 twelve of them feed 128
// FMAs a thread, at TM = 4 eight feed 64 (2 x 8 heads, 2048 x 2048, d = 64: 480 against 548 us; paired
// FMAs, half the instructions, gave 4 % at the most).  Fewer rows per tile when there are not CTAs for
// all SMs.  Tiles that stream by are copied asynchronously, each as soon as its place is free.
//
// Forward: online softmax, one pass over the keys; with parts, a CTA has a run of key tiles of its
// entry's own length, and leaves sums that a second launch joins.
// Backward: P again from lse; one kernel for both products that differ in what stays:
//   dQ          rows = queries, columns = keys:    dQ += dS K
//   dK and dV   rows = keys, columns = queries:    dV += P^T dH, dK += dS^T Q
// so every gradient is summed by one CTA in a fixed order, without atomics.
#include "common.cuh"
#include "cross.cuh"
#include "ptx.cuh"

#include <math.h>

namespace anchor {
namespace {

constexpr int kBN = 64;
// threads of a CTA, 16 to a row group: 128, with up to 8 rows each; at d = 128 256, with up to 4 (its
// tiles leave room for one CTA an SM)
template <int D> constexpr int kThreads = D == 128 ? 256 : 128;
template <int D> constexpr int kTY = kThreads<D> / 16;
constexpr int kPitchS = kBN + 4;
constexpr float kLog2e = 1.4426950408889634f;

// `rows` rows of D elements into shared memory, zeros where at(r) is null: asynchronous copies, one
// group a call
template <int D, typename At>
__device__ __forceinline__ void load_rows(float *dst, int rows, At at) {
    constexpr int C = D / 4;
    for (int i = threadIdx.x; i < rows * C; i += kThreads<D>) {
        const int r = i / C, c = 4 * (i - r * C);
        const float *src = at(r);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst + r * (D + 4) + c)),
                     "l"(src ? src + c : nullptr), "r"(src ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// all but the `left` groups begun last have landed
template <int left> __device__ __forceinline__ void landed() { asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory"); }

// s[i][j] = a row (ty TM + i) . b row (tx + 16 j)
template <int D, int TM>
__device__ __forceinline__ void dots(const float *a, const float *b, float (&s)[TM][4]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 x[TM], y[4];
#pragma unroll
        for (int i = 0; i < TM; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (ty * TM + i) * (D + 4) + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * (D + 4) + k);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
    }
}

// this thread's output columns: D / 16 of them, in runs of up to four
template <int D> constexpr int kCols = D / 16;
template <int D> __device__ __forceinline__ int col_of(int j) {
    const int tx = threadIdx.x & 15;
    return D >= 64 ? 4 * tx + 64 * (j / 4) + j % 4 : tx * kCols<D> + j;
}

// o[i][j] += sum_key w[ty TM + i][key] v[key][col j]
template <int D, int TM>
__device__ __forceinline__ void accumulate(const float *w, const float *v, float (&o)[TM][kCols<D>]) {
    const int ty = threadIdx.x >> 4;
#pragma unroll 2
    for (int k = 0; k < kBN; k += 4) {
        float x[TM][4];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            *reinterpret_cast<float4 *>(x[i]) = *reinterpret_cast<const float4 *>(w + (ty * TM + i) * kPitchS + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[kCols<D>];
            if constexpr (kCols<D> >= 4) {
#pragma unroll
                for (int j = 0; j < kCols<D>; j += 4)
                    *reinterpret_cast<float4 *>(y + j) =
                        *reinterpret_cast<const float4 *>(v + (k + q) * (D + 4) + col_of<D>(j));
            } else {
#pragma unroll
                for (int j = 0; j < kCols<D>; ++j) y[j] = v[(k + q) * (D + 4) + col_of<D>(j)];
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < kCols<D>; ++j) o[i][j] = fmaf(x[i][q], y[j], o[i][j]);
        }
    }
}

template <int D, int TM>
__device__ __forceinline__ void store_scores(float *dst, const float (&s)[TM][4]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[(ty * TM + i) * kPitchS + tx + 16 * j] = s[i][j];
}

// over the 16 threads of a row
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int D, int TM> constexpr size_t forward_smem() {
    return 4 * ((size_t)(kTY<D> * TM + 2 * kBN) * (D + 4) + kTY<D> * TM * kPitchS);
}

template <int D, int TM>
__global__ void __launch_bounds__(kThreads<D>) cross_simt_forward_kernel(const CrossProblem p, const CrossParts w, int tiles) {
    constexpr int BM = kTY<D> * TM;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sK = sQ + BM * (D + 4), *sV = sK + kBN * (D + 4), *sP = sV + kBN * (D + 4);
    grid_dependency_wait();
    grid_dependents_launch();
    const int tile = (int)(blockIdx.x % tiles), bk = (int)(blockIdx.x / tiles);
    const int b = bk / p.kv, k = bk - b * p.kv, r0 = tile * BM;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int L = cross_length(p, b), key_tiles = (L + kBN - 1) / kBN;
    const int t0 = (int)((long long)key_tiles * blockIdx.y / w.parts), t1 = (int)((long long)key_tiles * (blockIdx.y + 1) / w.parts);
    const float c = p.scale * kLog2e;
    const float *Q = (const float *)p.Q.ptr;
    const float *K = (const float *)p.K.ptr + b * p.K.sb + k * p.K.sh, *V = (const float *)p.V.ptr + b * p.V.sb + k * p.V.sh;
    auto load_k = [&](int t) { load_rows<D>(sK, kBN, [&](int r) { return t * kBN + r < L ? K + (t * kBN + r) * p.K.sn : nullptr; }); };
    auto load_v = [&](int t) { load_rows<D>(sV, kBN, [&](int r) { return t * kBN + r < L ? V + (t * kBN + r) * p.V.sn : nullptr; }); };
    load_rows<D>(sQ, BM, [&](int r) { return r0 + r < p.rows ? Q + cross_row(p, p.Q, b, k, r0 + r) : nullptr; });
    if (t0 < t1) {
        load_k(t0);
        load_v(t0);
    }
    float m[TM], l[TM], o[TM][kCols<D>];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kCols<D>; ++j) o[i][j] = 0.f;
    }
    // each of K and V is fetched again as soon as its tile has been used, while the other is
    for (int t = t0; t < t1; ++t) {
        landed<1>();  // K (and Q)
        __syncthreads();
        float s[TM][4];
        dots<D, TM>(sQ, sK, s);
        __syncthreads();
        if (t + 1 < t1) load_k(t + 1);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = t * kBN + tx + 16 * j < L ? s[i][j] * c : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            top = row_max(top);
            const float shift = top == -INFINITY ? 0.f : top;  // a row whose scores are all -infinity
            const float keep = exp2f(m[i] - shift);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - shift);
                sum += s[i][j];
            }
            l[i] = l[i] * keep + row_sum(sum);
            m[i] = top;
#pragma unroll
            for (int j = 0; j < kCols<D>; ++j) o[i][j] *= keep;
        }
        store_scores<D, TM>(sP, s);  // a warp writes and reads its own rows of P
        if (t + 1 < t1) landed<1>();
        else landed<0>();
        __syncthreads();  // V
        accumulate<D, TM>(sP, sV, o);
        __syncthreads();
        if (t + 1 < t1) load_v(t + 1);
    }
    landed<0>();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = r0 + ty * TM + i;
        if (r >= p.rows) continue;
        if (w.parts > 1) {
            const long long f = (long long)blockIdx.y * p.B * p.kv * p.rows + cross_flat(p, b, k, r);
#pragma unroll
            for (int j = 0; j < kCols<D>; ++j) w.o[f * D + col_of<D>(j)] = o[i][j];
            if (tx == 0) w.ml[f] = make_float2(m[i], l[i]);
            continue;
        }
        float *H = (float *)p.H.ptr + cross_row(p, p.H, b, k, r);
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // no state at all
#pragma unroll
        for (int j = 0; j < kCols<D>; ++j) H[col_of<D>(j)] = o[i][j] * inv;
        if (p.lse && tx == 0) p.lse[cross_flat(p, b, k, r)] = l[i] == 0.f ? -INFINITY : m[i] * (1.f / kLog2e) + logf(l[i]);
    }
}

template <int D, int TM> constexpr size_t backward_smem() {
    return 4 * ((size_t)(2 * kTY<D> * TM + 3 * kBN) * (D + 4) + kTY<D> * TM * kPitchS + 2 * 2 * kBN);
}

// KEYS: rows are keys, columns the query rows of the key head; else rows are query rows.
template <int D, int TM, bool KEYS>
__global__ void __launch_bounds__(kThreads<D>) cross_simt_backward_kernel(const CrossProblem p, const float *delta, int tiles) {
    constexpr int BM = kTY<D> * TM;
    extern __shared__ __align__(16) float sm[];
    // rows: (Q, dH) or (K, V); columns: (K, V) or (Q, dH)
    float *sA = sm, *sA2 = sA + BM * (D + 4), *sB = sA2 + BM * (D + 4) /* [2] */, *sB2 = sB + 2 * kBN * (D + 4), *sW = sB2 + kBN * (D + 4);
    float *sLD = sW + BM * kPitchS;  // KEYS: the columns' lse and D, [2][2][kBN]
    grid_dependency_wait();
    grid_dependents_launch();
    const int tile = (int)(blockIdx.x % tiles), bk = (int)(blockIdx.x / tiles);
    const int b = bk / p.kv, k = bk - b * p.kv, r0 = tile * BM;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int L = cross_length(p, b);
    const float c = p.scale * kLog2e;
    const float *Q = (const float *)p.Q.ptr, *G = (const float *)p.dH.ptr;
    const float *K = (const float *)p.K.ptr + b * p.K.sb + k * p.K.sh, *V = (const float *)p.V.ptr + b * p.V.sb + k * p.V.sh;
    auto q_row = [&](int r) { return r < p.rows ? Q + cross_row(p, p.Q, b, k, r) : nullptr; };
    auto g_row = [&](int r) { return r < p.rows ? G + cross_row(p, p.dH, b, k, r) : nullptr; };
    auto k_row = [&](int r) { return r < L ? K + r * p.K.sn : nullptr; };
    auto v_row = [&](int r) { return r < L ? V + r * p.V.sn : nullptr; };
    load_rows<D>(sA, BM, [&](int r) { return KEYS ? k_row(r0 + r) : q_row(r0 + r); });
    load_rows<D>(sA2, BM, [&](int r) { return KEYS ? v_row(r0 + r) : g_row(r0 + r); });
    float o[TM][kCols<D>], o2[KEYS ? TM : 1][kCols<D>], lse2[TM], dl[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < kCols<D>; ++j) {
            o[i][j] = 0.f;
            if (KEYS) o2[i][j] = 0.f;
        }
        const int r = r0 + ty * TM + i;
        lse2[i] = dl[i] = 0.f;
        if (!KEYS && r < p.rows) {
            const long long f = cross_flat(p, b, k, r);
            lse2[i] = p.lse[f] * kLog2e;
            dl[i] = delta[f];
        }
    }
    const int cols = KEYS ? (r0 < L ? p.rows : 0) : L;  // a tile of masked keys has no gradient
    // The first of the streaming tiles (used last) is fetched a step ahead into its other place, the
    // second as soon as it has been used.
    auto load_b = [&](int c0) {
        const int at = (c0 / kBN) & 1;
        if (KEYS && threadIdx.x < kBN) {
            const bool in = c0 + (int)threadIdx.x < p.rows;
            const long long f = in ? cross_flat(p, b, k, c0 + threadIdx.x) : 0;
            sLD[at * 2 * kBN + threadIdx.x] = in ? p.lse[f] * kLog2e : 0.f;
            sLD[at * 2 * kBN + kBN + threadIdx.x] = in ? delta[f] : 0.f;
        }
        load_rows<D>(sB + at * kBN * (D + 4), kBN, [&](int r) { return KEYS ? q_row(c0 + r) : k_row(c0 + r); });
    };
    auto load_b2 = [&](int c0) { load_rows<D>(sB2, kBN, [&](int r) { return KEYS ? g_row(c0 + r) : v_row(c0 + r); }); };
    if (cols > 0) {
        load_b(0);
        load_b2(0);
    }
    for (int c0 = 0; c0 < cols; c0 += kBN) {
        const bool more = c0 + kBN < cols;
        const float *sB0 = sB + ((c0 / kBN) & 1) * kBN * (D + 4), *sL = sLD + ((c0 / kBN) & 1) * 2 * kBN, *sD = sL + kBN;
        landed<0>();
        __syncthreads();
        if (more) load_b(c0 + kBN);
        float s[TM][4], g[TM][4];
        dots<D, TM>(sA, sB0, s);
        dots<D, TM>(sA2, sB2, g);
        if (!KEYS) {
            __syncthreads();
            if (more) load_b2(c0 + kBN);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = tx + 16 * j;
                const bool on = KEYS ? (r0 + ty * TM + i < L && c0 + col < p.rows) : c0 + col < L;
                s[i][j] = on ? exp2f(fmaf(s[i][j], c, -(KEYS ? sL[col] : lse2[i]))) : 0.f;
                g[i][j] = on ? s[i][j] * (g[i][j] - (KEYS ? sD[col] : dl[i])) : 0.f;
            }
        if constexpr (KEYS) {
            store_scores<D, TM>(sW, s);
            __syncwarp();
            accumulate<D, TM>(sW, sB2, o2);
            __syncthreads();
            if (more) load_b2(c0 + kBN);
        }
        store_scores<D, TM>(sW, g);
        __syncwarp();
        accumulate<D, TM>(sW, sB0, o);
        __syncwarp();
    }
    landed<0>();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = r0 + ty * TM + i;
        if (r >= (KEYS ? p.s : p.rows)) continue;
        float *dst = KEYS ? (float *)p.dK.ptr + b * p.dK.sb + k * p.dK.sh + r * p.dK.sn : (float *)p.dQ.ptr + cross_row(p, p.dQ, b, k, r);
#pragma unroll
        for (int j = 0; j < kCols<D>; ++j) dst[col_of<D>(j)] = o[i][j] * p.scale;
        if constexpr (KEYS) {
            dst = (float *)p.dV.ptr + b * p.dV.sb + k * p.dV.sh + r * p.dV.sn;
#pragma unroll
            for (int j = 0; j < kCols<D>; ++j) dst[col_of<D>(j)] = o2[i][j];
        }
    }
}

// rows of a tile: the most of 64, 32 and 16 whose tiles still give every SM a CTA, else 16
int tile_rows(const CrossProblem &p, long long rows) {
    const long long heads = (long long)p.B * p.kv;
    int bm = 64;
    while (bm > 16 && (heads * ((rows + bm - 1) / bm) < kPlanSMs || rows <= bm / 2)) bm /= 2;
    return bm;
}

template <int D, int TM>
cudaError_t forward(const CrossProblem &p, const CrossParts &w, cudaStream_t stream) {
    const int tiles = (p.rows + kTY<D> * TM - 1) / (kTY<D> * TM);
    constexpr size_t smem = forward_smem<D, TM>();
    static SmemOnce allow;
    const cudaError_t e = allow(cross_simt_forward_kernel<D, TM>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_simt_forward_kernel<D, TM>, dim3(tiles * p.B * p.kv, w.parts), dim3(kThreads<D>), smem, stream, p, w, tiles);
}

template <int D, int TM, bool KEYS>
cudaError_t backward(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    const int tiles = ((KEYS ? p.s : p.rows) + kTY<D> * TM - 1) / (kTY<D> * TM);
    constexpr size_t smem = backward_smem<D, TM>();
    static SmemOnce allow;
    const cudaError_t e = allow(cross_simt_backward_kernel<D, TM, KEYS>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_simt_backward_kernel<D, TM, KEYS>, dim3(tiles * p.B * p.kv), dim3(kThreads<D>), smem, stream, p, delta, tiles);
}

template <int D, bool KEYS>
cudaError_t backward_rows(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    const int bm = tile_rows(p, KEYS ? p.s : p.rows);
    return bm == 64   ? backward<D, 64 / kTY<D>, KEYS>(p, delta, stream)
           : bm == 32 ? backward<D, 32 / kTY<D>, KEYS>(p, delta, stream)
                      : backward<D, 16 / kTY<D>, KEYS>(p, delta, stream);
}
template <int D>
cudaError_t backward_d(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    const cudaError_t e = p.rows > 0 ? backward_rows<D, false>(p, delta, stream) : cudaSuccess;
    return e != cudaSuccess || p.s == 0 ? e : backward_rows<D, true>(p, delta, stream);
}

}  // namespace

// Parts of the key axis: none while the row tiles alone fill the SMs; else so many that two CTAs
// of them do, with two key tiles a part at least.
int cross_simt_parts(const CrossProblem &p) {
    const int bm = tile_rows(p, p.rows);
    const long long ctas = (long long)p.B * p.kv * ((p.rows + bm - 1) / bm);
    const long long want = 2 * kPlanSMs / std::max(1LL, ctas), most = (p.s + 2 * kBN - 1) / (2 * kBN);
    return (int)std::max(1LL, std::min(want, most));
}

cudaError_t launch_cross_simt_forward(const CrossProblem &p, const CrossParts &w, cudaStream_t stream) {
    const int bm = tile_rows(p, p.rows);
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return bm == 64   ? forward<D, 64 / kTY<D>>(p, w, stream)
               : bm == 32 ? forward<D, 32 / kTY<D>>(p, w, stream)
                          : forward<D, 16 / kTY<D>>(p, w, stream);
    };
    switch (p.d) {
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    default: return go(std::integral_constant<int, 128>{});
    }
}

cudaError_t launch_cross_simt_backward(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    switch (p.d) {
    case 16: return backward_d<16>(p, delta, stream);
    case 32: return backward_d<32>(p, delta, stream);
    case 64: return backward_d<64>(p, delta, stream);
    default: return backward_d<128>(p, delta, stream);
    }
}

}  // namespace anchor
