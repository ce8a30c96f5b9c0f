// Cross attention in fp32 on CUDA cores, forward and backward (formulas in
// include/anchor_attn.h).
//
// Tiles of BM = 64, 32 or 16 rows by 48 columns; 256 threads, in two halves.  A thread has BM / 16 rows by
// 6 columns of the scores and BM / 16 rows by d / 8 columns of the outputs.  All tiles lie row by row in
// shared memory with a pitch of d + 4 floats: 16-byte reads along d (scores) and along the columns
// (outputs) are then free of conflicts, and one copy serves both products.
//
// What bounds it: the FMAs and those reads together.  A warp's 16-byte read takes two cycles of shared memory
// for two rows of eight different places, and four for sixteen places in each half of the warp: with
// 4 x 8 threads a warp, its lanes in pairs of the same place, every read takes two, ten of them for 48
// FMAs of two each (2 x 8 heads, 2048 x 2048, a training step: 2168 -> 2079 us at d = 64 against 2 x 16
// threads a warp, 4133 -> 4050 at d = 128).  Two FMAs an instruction leave issue slots to the reads: 2156 ->
// 2079 and 4307 -> 4050.  Now 1804 and 3535: 43 TFLOP/s, 0.54 of the FMAs' rate.
//
// Forward: online softmax, one pass over the keys, every other tile of them by each half, whose sums are
// joined at the end; K and V are each fetched again as soon as their tile has been used.  With parts, a CTA
// has a run of key tiles of its entry's own length, and leaves sums that a second launch joins.
// Backward: P again from lse; two kinds of CTAs that differ in what stays:
//   dQ          rows = queries, columns = keys:    dQ += dS K
//   dK and dV   rows = keys, columns = queries:    dV += P^T dH, dK += dS^T Q
// in one launch, the longer CTAs first (two launches: 2011 us at d = 64, 3915 at 128).
// The first half makes S and P and sums dV, the second dP and dS and sums dK; of dQ each sums half of the
// keys.  Every gradient is summed by one CTA in a fixed order, without atomics.  (One half that did both:
// 4 x 6 heads, 197 x 300, d = 64, a training step of 122 us against 98 in two launches.)
#include "common.cuh"
#include "cross.cuh"
#include "ptx.cuh"

#include <math.h>

namespace anchor {
namespace {

constexpr int kBN = 48;       // rows of a tile that streams by
constexpr int kGroup = 128;   // threads of a half
constexpr int kThreads = 2 * kGroup;
constexpr int kNJ = kBN / 8;
constexpr int kPitchS = kBN;  // of P and dS: rows next to one another are 16 banks apart
template <int BM> constexpr int kTM = BM / 16;
template <int D> constexpr int kPerSM = D == 128 ? 1 : 2;
constexpr float kLog2e = 1.4426950408889634f;

// A thread of its half: 16 groups of 8, four groups a warp.  Group ty has rows ty, ty + 16, ..., thread
// tx columns tx, tx + 8, ...  Lanes 2 tx and 2 tx + 1 of half a warp are thread tx of two groups.
__device__ __forceinline__ int half() { return threadIdx.x / kGroup; }
__device__ __forceinline__ int lane_x() { return (threadIdx.x >> 1) & 7; }
__device__ __forceinline__ int lane_y() { return 4 * ((threadIdx.x % kGroup) >> 5) + ((threadIdx.x >> 3) & 2) + (threadIdx.x & 1); }
// barriers of a half, and between the halves (0 is __syncthreads)
__device__ __forceinline__ void half_sync() { asm volatile("bar.sync %0, %1;" ::"r"(1 + half()), "n"(kGroup) : "memory"); }
__device__ __forceinline__ void first_arrives() { asm volatile("bar.arrive 3, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void second_waits() { asm volatile("bar.sync 3, %0;" ::"n"(kThreads) : "memory"); }

// `rows` rows of D elements into shared memory by T threads, zeros where at(r) is null: asynchronous
// copies, one group a call
template <int D, int T, typename At>
__device__ __forceinline__ void load_rows(float *dst, int rows, At at) {
    constexpr int C = D / 4;
    for (int i = threadIdx.x % T; i < rows * C; i += T) {
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

// two FMAs in one instruction, each rounded as fmaf is
__device__ __forceinline__ void fma2(unsigned long long &c, unsigned long long a, unsigned long long b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ unsigned long long pair(float a, float b) {
    unsigned long long v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void unpair(unsigned long long v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

// s[i][j] = a row (ty + 16 i) . b row (tx + 8 j): even and odd columns in one pair of sums
template <int D, int TM>
__device__ __forceinline__ void dots(const float *a, const float *b, float (&s)[TM][kNJ]) {
    const int tx = lane_x(), ty = lane_y();
    unsigned long long c[TM][kNJ];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < kNJ; ++j) c[i][j] = 0;
#pragma unroll 8
    for (int k = 0; k < D; k += 4) {
        ulonglong2 x[TM], y[kNJ];
#pragma unroll
        for (int i = 0; i < TM; ++i) x[i] = *reinterpret_cast<const ulonglong2 *>(a + (ty + 16 * i) * (D + 4) + k);
#pragma unroll
        for (int j = 0; j < kNJ; ++j) y[j] = *reinterpret_cast<const ulonglong2 *>(b + (tx + 8 * j) * (D + 4) + k);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < kNJ; ++j) {
                fma2(c[i][j], x[i].x, y[j].x);
                fma2(c[i][j], x[i].y, y[j].y);
            }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < kNJ; ++j) {
            float even, odd;
            unpair(c[i][j], even, odd);
            s[i][j] = even + odd;
        }
}

// this thread's output columns: D / 8 of them, in runs of up to four
template <int D> constexpr int kCols = D / 8;
template <int D> __device__ __forceinline__ int col_of(int j) {
    const int tx = lane_x();
    return D >= 32 ? 4 * tx + 32 * (j / 4) + j % 4 : tx * kCols<D> + j;
}

// o[i][j] += sum_key w[ty + 16 i][key] v[key][col j], over `keys` keys
template <int D, int TM, int keys>
__device__ __forceinline__ void accumulate(const float *w, const float *v, float (&o)[TM][kCols<D>]) {
    constexpr int C = kCols<D>, C2 = C > 1 ? C / 2 : 1;
    const int ty = lane_y();
    unsigned long long c[TM][C2];
    if constexpr (C > 1) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < C2; ++j) c[i][j] = pair(o[i][2 * j], o[i][2 * j + 1]);
    }
#pragma unroll 4
    for (int k = 0; k < keys; k += 4) {
        float x[TM][4];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            *reinterpret_cast<float4 *>(x[i]) = *reinterpret_cast<const float4 *>(w + (ty + 16 * i) * kPitchS + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float *vr = v + (k + q) * (D + 4);
            if constexpr (C == 1) {
                const float y = vr[col_of<D>(0)];
#pragma unroll
                for (int i = 0; i < TM; ++i) o[i][0] = fmaf(x[i][q], y, o[i][0]);
            } else {
                unsigned long long y[C2];
                if constexpr (C >= 4) {
#pragma unroll
                    for (int j = 0; j < C2; j += 2)
                        *reinterpret_cast<ulonglong2 *>(y + j) = *reinterpret_cast<const ulonglong2 *>(vr + col_of<D>(2 * j));
                } else {
                    y[0] = *reinterpret_cast<const unsigned long long *>(vr + col_of<D>(0));
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const unsigned long long xx = pair(x[i][q], x[i][q]);
#pragma unroll
                    for (int j = 0; j < C2; ++j) fma2(c[i][j], xx, y[j]);
                }
            }
        }
    }
    if constexpr (C > 1) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < C2; ++j) unpair(c[i][j], o[i][2 * j], o[i][2 * j + 1]);
    }
}

template <int TM>
__device__ __forceinline__ void store_scores(float *dst, const float (&s)[TM][kNJ]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < kNJ; ++j) dst[(lane_y() + 16 * i) * kPitchS + lane_x() + 8 * j] = s[i][j];
}

// a half's sums to shared memory and back, by its own threads' numbers
template <int TM, int C> __device__ __forceinline__ void put_sums(float *to, const float (&o)[TM][C]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j) to[(i * C + j) * kGroup + threadIdx.x % kGroup] = o[i][j];
}
template <int C> __device__ __forceinline__ float sum_at(const float *from, int i, int j) {
    return from[(i * C + j) * kGroup + threadIdx.x % kGroup];
}

// over the 8 threads of a row
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 8; o > 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 8; o > 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int D, int BM> constexpr size_t forward_smem() {
    return 4 * ((size_t)(BM + 4 * kBN) * (D + 4) + 2 * BM * kPitchS);
}

template <int D, int BM>
__global__ void __launch_bounds__(kThreads, kPerSM<D>) cross_simt_forward_kernel(const CrossProblem p, const CrossParts w, int tiles) {
    constexpr int TM = kTM<BM>, C = kCols<D>;
    static_assert(BM * D <= 2 * kBN * (D + 4) && 2 * BM <= BM * kPitchS, "the second half's sums fit its tiles");
    extern __shared__ __align__(16) float sm[];
    const int h = half();
    float *sQ = sm, *sX = sQ + BM * (D + 4) + 2 * kBN * (D + 4) /* of the second half */;
    float *sK = sQ + BM * (D + 4) + h * 2 * kBN * (D + 4), *sV = sK + kBN * (D + 4);
    float *sPs = sm + (BM + 4 * kBN) * (D + 4), *sP = sPs + h * BM * kPitchS;
    grid_dependency_wait();
    grid_dependents_launch();
    const int tile = (int)(blockIdx.x % tiles), bk = (int)(blockIdx.x / tiles);
    const int b = bk / p.kv, k = bk - b * p.kv, r0 = tile * BM;
    const int tx = lane_x(), ty = lane_y();
    const int L = cross_length(p, b), key_tiles = (L + kBN - 1) / kBN;
    const int t0 = (int)((long long)key_tiles * blockIdx.y / w.parts), t1 = (int)((long long)key_tiles * (blockIdx.y + 1) / w.parts);
    const float c = p.scale * kLog2e;
    const float *Q = (const float *)p.Q.ptr;
    const float *K = (const float *)p.K.ptr + b * p.K.sb + k * p.K.sh, *V = (const float *)p.V.ptr + b * p.V.sb + k * p.V.sh;
    auto load_k = [&](int t) {
        load_rows<D, kGroup>(sK, t < t1 ? kBN : 0, [&](int r) { return t * kBN + r < L ? K + (t * kBN + r) * p.K.sn : nullptr; });
    };
    auto load_v = [&](int t) {
        load_rows<D, kGroup>(sV, t < t1 ? kBN : 0, [&](int r) { return t * kBN + r < L ? V + (t * kBN + r) * p.V.sn : nullptr; });
    };
    load_rows<D, kThreads>(sQ, BM, [&](int r) { return r0 + r < p.rows ? Q + cross_row(p, p.Q, b, k, r0 + r) : nullptr; });
    load_k(t0 + h);
    load_v(t0 + h);
    float m[TM], l[TM], o[TM][C];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) o[i][j] = 0.f;
    }
    landed<2>();
    __syncthreads();  // Q
    // each of K and V is fetched again as soon as its tile has been used, while the other is
    for (int t = t0 + h; t < t1; t += 2) {
        landed<1>();
        half_sync();  // K
        float s[TM][kNJ];
        dots<D, TM>(sQ, sK, s);
        half_sync();
        load_k(t + 2);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < kNJ; ++j) {
                s[i][j] = t * kBN + tx + 8 * j < L ? s[i][j] * c : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            top = row_max(top);
            const float shift = top == -INFINITY ? 0.f : top;  // a row whose scores are all -infinity
            const float keep = exp2f(m[i] - shift);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < kNJ; ++j) {
                s[i][j] = exp2f(s[i][j] - shift);
                sum += s[i][j];
            }
            l[i] = l[i] * keep + sum;  // of this thread's columns
            m[i] = top;
#pragma unroll
            for (int j = 0; j < C; ++j) o[i][j] *= keep;
        }
        store_scores<TM>(sP, s);  // a warp writes and reads its own rows of P
        landed<1>();
        half_sync();  // V
        accumulate<D, TM, kBN>(sP, sV, o);
        half_sync();
        load_v(t + 2);
    }
    landed<0>();
#pragma unroll
    for (int i = 0; i < TM; ++i) l[i] = row_sum(l[i]);
    // the second half's sums, on the larger maximum of the two
    if (h == 1) {
        put_sums(sX, o);
#pragma unroll
        for (int i = 0; i < TM; ++i)
            if (tx == 0) sP[ty + 16 * i] = m[i], sP[BM + ty + 16 * i] = l[i];
    }
    __syncthreads();
    if (h == 1) return;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int row = ty + 16 * i, r = r0 + row;
        const float m1 = sPs[BM * kPitchS + row], top = fmaxf(m[i], m1), shift = top == -INFINITY ? 0.f : top;
        const float f0 = exp2f(m[i] - shift), f1 = exp2f(m1 - shift);
        m[i] = top;
        l[i] = l[i] * f0 + sPs[BM * kPitchS + BM + row] * f1;
#pragma unroll
        for (int j = 0; j < C; ++j) o[i][j] = o[i][j] * f0 + sum_at<C>(sX, i, j) * f1;
        if (r >= p.rows) continue;
        if (w.parts > 1) {
            const long long f = (long long)blockIdx.y * p.B * p.kv * p.rows + cross_flat(p, b, k, r);
#pragma unroll
            for (int j = 0; j < C; ++j) w.o[f * D + col_of<D>(j)] = o[i][j];
            if (tx == 0) w.ml[f] = make_float2(m[i], l[i]);
            continue;
        }
        float *H = (float *)p.H.ptr + cross_row(p, p.H, b, k, r);
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // no state at all
#pragma unroll
        for (int j = 0; j < C; ++j) H[col_of<D>(j)] = o[i][j] * inv;
        if (p.lse && tx == 0) p.lse[cross_flat(p, b, k, r)] = l[i] == 0.f ? -INFINITY : m[i] * (1.f / kLog2e) + logf(l[i]);
    }
}

template <int D, int BM> constexpr size_t backward_smem() {
    return 4 * ((size_t)(2 * BM + 4 * kBN) * (D + 4) + 2 * BM * kPitchS + 2 * 2 * kBN);
}

// KEYS: rows are keys, columns the query rows of the key head; else rows are query rows.  `index`: of the
// CTA among those of its kind, `tiles` of them a key head.
template <int D, int BM, bool KEYS>
__device__ __forceinline__ void cross_simt_backward(const CrossProblem &p, const float *delta, int index, int tiles) {
    constexpr int TM = kTM<BM>, C = kCols<D>, kTile = kBN * (D + 4);
    static_assert(BM * D <= 2 * kTile, "the second half's sums fit the tiles");
    extern __shared__ __align__(16) float sm[];
    // rows: (Q, dH) or (K, V); columns: (K, V) or (Q, dH), two places each
    float *sA = sm, *sA2 = sA + BM * (D + 4), *sB = sA2 + BM * (D + 4), *sB2 = sB + 2 * kTile;
    float *sP = sB2 + 2 * kTile, *sS = sP + BM * kPitchS;
    float *sLD = sS + BM * kPitchS;  // KEYS: the columns' lse and D, [2][2][kBN]
    const int h = half();
    const int tile = index % tiles, bk = index / tiles;
    const int b = bk / p.kv, k = bk - b * p.kv, r0 = tile * BM;
    const int tx = lane_x(), ty = lane_y();
    const int L = cross_length(p, b);
    const float c = p.scale * kLog2e;
    const float *Q = (const float *)p.Q.ptr, *G = (const float *)p.dH.ptr;
    const float *K = (const float *)p.K.ptr + b * p.K.sb + k * p.K.sh, *V = (const float *)p.V.ptr + b * p.V.sb + k * p.V.sh;
    auto q_row = [&](int r) { return r < p.rows ? Q + cross_row(p, p.Q, b, k, r) : nullptr; };
    auto g_row = [&](int r) { return r < p.rows ? G + cross_row(p, p.dH, b, k, r) : nullptr; };
    auto k_row = [&](int r) { return r < L ? K + r * p.K.sn : nullptr; };
    auto v_row = [&](int r) { return r < L ? V + r * p.V.sn : nullptr; };
    load_rows<D, kThreads>(sA, BM, [&](int r) { return KEYS ? k_row(r0 + r) : q_row(r0 + r); });
    load_rows<D, kThreads>(sA2, BM, [&](int r) { return KEYS ? v_row(r0 + r) : g_row(r0 + r); });
    float o[TM][C], stat[TM];  // !KEYS: a row's lse (first half) or D (second half)
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < C; ++j) o[i][j] = 0.f;
        const int r = r0 + ty + 16 * i;
        stat[i] = 0.f;
        if (!KEYS && r < p.rows) {
            const long long f = cross_flat(p, b, k, r);
            stat[i] = h == 0 ? far_lse(p.lse[f] * kLog2e) : delta[f];
        }
    }
    const int cols = KEYS ? (r0 < L ? p.rows : 0) : L;  // a tile of masked keys has no gradient
    auto load = [&](int c0) {  // a step ahead, into the other place
        const int at = (c0 / kBN) & 1;
        if (KEYS && threadIdx.x < kBN) {
            const bool in = c0 + (int)threadIdx.x < p.rows;
            const long long f = in ? cross_flat(p, b, k, c0 + threadIdx.x) : 0;
            sLD[at * 2 * kBN + threadIdx.x] = in ? far_lse(p.lse[f] * kLog2e) : 0.f;
            sLD[at * 2 * kBN + kBN + threadIdx.x] = in ? delta[f] : 0.f;
        }
        load_rows<D, kThreads>(sB + at * kTile, kBN, [&](int r) { return KEYS ? q_row(c0 + r) : k_row(c0 + r); });
        load_rows<D, kThreads>(sB2 + at * kTile, kBN, [&](int r) { return KEYS ? g_row(c0 + r) : v_row(c0 + r); });
    };
    if (cols > 0) load(0);
    for (int c0 = 0; c0 < cols; c0 += kBN) {
        const int at = (c0 / kBN) & 1;
        const float *sB0 = sB + at * kTile, *sB20 = sB2 + at * kTile, *sStat = sLD + (at * 2 + h) * kBN;
        landed<0>();
        __syncthreads();
        if (c0 + kBN < cols) load(c0 + kBN);
        auto on = [&](int i, int j) {
            const int row = r0 + ty + 16 * i, col = c0 + tx + 8 * j;
            return KEYS ? row < L && col < p.rows : col < L;
        };
        float s[TM][kNJ];
        dots<D, TM>(h == 0 ? sA : sA2, h == 0 ? sB0 : sB20, s);
        if (h == 0) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < kNJ; ++j)
                    s[i][j] = on(i, j) ? exp2f(fmaf(s[i][j], c, -(KEYS ? sStat[tx + 8 * j] : stat[i]))) : 0.f;
            store_scores<TM>(sP, s);
            first_arrives();
        } else {
            second_waits();
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < kNJ; ++j)
                    s[i][j] = on(i, j) ? sP[(ty + 16 * i) * kPitchS + tx + 8 * j] * (s[i][j] - (KEYS ? sStat[tx + 8 * j] : stat[i])) : 0.f;
            store_scores<TM>(sS, s);
        }
        if constexpr (KEYS) {
            __syncwarp();  // a warp's own rows
            accumulate<D, TM, kBN>(h == 0 ? sP : sS, h == 0 ? sB20 : sB0, o);
        } else {
            __syncthreads();
            accumulate<D, TM, kBN / 2>(sS + h * (kBN / 2), sB0 + h * (kBN / 2) * (D + 4), o);
        }
    }
    landed<0>();
    if constexpr (!KEYS) {
        __syncthreads();
        if (h == 1) put_sums(sB, o);
        __syncthreads();
        if (h == 1) return;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = r0 + ty + 16 * i;
        if (r >= (KEYS ? p.s : p.rows)) continue;
        if constexpr (KEYS) {
            float *dst = h == 0 ? (float *)p.dV.ptr + b * p.dV.sb + k * p.dV.sh + r * p.dV.sn
                                : (float *)p.dK.ptr + b * p.dK.sb + k * p.dK.sh + r * p.dK.sn;
            const float f = h == 0 ? 1.f : p.scale;
#pragma unroll
            for (int j = 0; j < C; ++j) dst[col_of<D>(j)] = o[i][j] * f;
        } else {
            float *dst = (float *)p.dQ.ptr + cross_row(p, p.dQ, b, k, r);
#pragma unroll
            for (int j = 0; j < C; ++j) dst[col_of<D>(j)] = (o[i][j] + sum_at<C>(sB, i, j)) * p.scale;
        }
    }
}

template <int D, int BM>
__global__ void __launch_bounds__(kThreads, kPerSM<D>)
cross_simt_backward_kernel(const CrossProblem p, const float *delta, int q_tiles, int k_tiles, int first, bool keys_first) {
    grid_dependency_wait();
    grid_dependents_launch();
    const bool head = (int)blockIdx.x < first;
    const int index = (int)blockIdx.x - (head ? 0 : first);
    if (head == keys_first) cross_simt_backward<D, BM, true>(p, delta, index, k_tiles);
    else cross_simt_backward<D, BM, false>(p, delta, index, q_tiles);
}

// Parts of a forward's keys that make many CTAs out of few: of twelve tiles and more each (d < 128).
long long long_parts(const CrossProblem &p) { return p.d < 128 ? (p.s + kBN - 1) / kBN / 12 : 0; }

// Rows of a forward's tile: the most of 64, 32 and 16 whose tiles, or long parts of them, still give every SM a CTA
// (parts: two), else 16.
int tile_rows(const CrossProblem &p) {
    int bm = 64;
    auto few = [&] {
        const long long ctas = (long long)p.B * p.kv * ((p.rows + bm - 1) / bm);
        return ctas < kPlanSMs && ctas * long_parts(p) < 2 * kPlanSMs;
    };
    while (bm > 16 && (few() || p.rows <= bm / 2)) bm /= 2;
    return bm;
}

// Rows of a backward's tiles: the least of the longest CTA's time and all CTAs' spread over the SMs' places,
// whichever is more, where a row costs a quarter more in tiles of 32 and twice as much in tiles of 16 (a training
// step of 4 x 6 heads, 197 x 300, d = 64: 79 us with 32, 87 with 64, 98 with 16; of 11 x 4 heads over 1, 119 x 8152: 1837
// with 64, 1500 with 32).
int backward_rows(const CrossProblem &p) {
    const double longest = std::max(3. * p.s, 4. * p.rows), all = 7. * p.B * p.kv * p.rows * (double)p.s / (kPlanSMs * (p.d < 128 ? 2 : 1));
    const double t64 = std::max(64 * longest, all), t32 = 1.25 * std::max(32 * longest, all), t16 = 2 * std::max(16 * longest, all);
    return t64 <= std::min(t32, t16) ? 64 : t32 <= t16 ? 32 : 16;
}

template <int D, int BM>
cudaError_t forward(const CrossProblem &p, const CrossParts &w, cudaStream_t stream) {
    const int tiles = (p.rows + BM - 1) / BM;
    constexpr size_t smem = forward_smem<D, BM>();
    static SmemOnce allow;
    const cudaError_t e = allow(cross_simt_forward_kernel<D, BM>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_simt_forward_kernel<D, BM>, dim3(tiles * p.B * p.kv, w.parts), dim3(kThreads), smem, stream, p, w, tiles);
}

template <int D, int BM>
cudaError_t backward(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    const int q_tiles = (p.rows + BM - 1) / BM, k_tiles = (p.s + BM - 1) / BM;
    // first those that take longer: four products over the queries against three over the keys
    const bool keys_first = 4LL * p.rows >= 3LL * p.s;
    const int first = (keys_first ? k_tiles : q_tiles) * p.B * p.kv;
    constexpr size_t smem = backward_smem<D, BM>();
    static SmemOnce allow;
    const cudaError_t e = allow(cross_simt_backward_kernel<D, BM>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_simt_backward_kernel<D, BM>, dim3((q_tiles + k_tiles) * p.B * p.kv), dim3(kThreads), smem, stream, p, delta,
                      q_tiles, k_tiles, first, keys_first);
}

}  // namespace

// Parts of the key axis: none while the row tiles alone fill the SMs; else so many that two CTAs of them do, with
// two key tiles a part at least.  Below d = 128, with few CTAs or very long keys, four times the places in long
// parts, which even out (11 x 4 heads over 1, 119 x 8152, d = 64: 516 -> 295 us; 16 heads, 128 x 8000: 197 -> 117; 64 x 8 heads, 1 x 8000: 735 -> 650; but 32
// heads, 500 x 2000: 226 -> 251, and at d = 128 3 x 8 heads, 300 x 3000: 360 -> 380).
int cross_simt_parts(const CrossProblem &p) {
    const int bm = tile_rows(p);
    const long long ctas = std::max(1LL, (long long)p.B * p.kv * ((p.rows + bm - 1) / bm)), tiles = (p.s + kBN - 1) / kBN;
    const long long some = std::min(2 * kPlanSMs / ctas, (tiles + 1) / 2);
    const long long many = ctas < kPlanSMs || tiles >= 96 ? std::min(8 * kPlanSMs / ctas, long_parts(p)) : 0;
    return (int)std::max({1LL, some, many});
}

cudaError_t launch_cross_simt_forward(const CrossProblem &p, const CrossParts &w, cudaStream_t stream) {
    const int bm = tile_rows(p);
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return bm == 64   ? forward<D, 64>(p, w, stream)
               : bm == 32 ? forward<D, 32>(p, w, stream)
                          : forward<D, 16>(p, w, stream);
    };
    switch (p.d) {
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    default: return go(std::integral_constant<int, 128>{});
    }
}

cudaError_t launch_cross_simt_backward(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    const int bm = backward_rows(p);
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return bm == 64 ? backward<D, 64>(p, delta, stream) : bm == 32 ? backward<D, 32>(p, delta, stream) : backward<D, 16>(p, delta, stream);
    };
    switch (p.d) {
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    default: return go(std::integral_constant<int, 128>{});
    }
}

}  // namespace anchor
