// Cross attention: argument checks, plan and launch; the join of a forward's parts; D = dH . H
// (formulas and layout in include/anchor_attn.h).
#include "cross.cuh"

#include <math.h>
#include <stdlib.h>

namespace anchor {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// One CTA per row: H = sum_parts o 2^(m - M) / sum_parts l 2^(m - M).  A warp takes every eighth part,
// lanes over the columns, and the warps' sums are added in order (with one warp for all parts its loads
// followed one another: 84 us for 152 parts).  Bound by the latency of a few loads.
template <typename T>
__global__ void __launch_bounds__(256) cross_join_kernel(const CrossProblem p, const CrossParts w, long long total) {
    __shared__ float s_o[8][128];
    __shared__ float s_l[8];
    grid_dependency_wait();
    grid_dependents_launch();
    const long long f = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float M = -INFINITY;
    for (int q = lane; q < w.parts; q += 32) M = fmaxf(M, w.ml[q * total + f].x);  // every warp for itself
    M = warp_max(M);
    const float shift = M == -INFINITY ? 0.f : M;
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int q = warp; q < w.parts; q += 8) {
        const float2 ml = w.ml[q * total + f];
        const float k = exp2f(ml.x - shift);
        l += ml.y * k;
        const float *src = w.o + (q * total + f) * p.d;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (32 * j + lane < p.d) o[j] = fmaf(src[32 * j + lane], k, o[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s_o[warp][32 * j + lane] = o[j];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= p.d) return;
    float sum = 0.f;
    l = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) sum += s_o[q][c], l += s_l[q];
    const int r = (int)(f % p.rows);
    const long long bk = f / p.rows;
    const int b = (int)(bk / p.kv), k = (int)(bk - (long long)b * p.kv);
    const float inv = l == 0.f ? 0.f : 1.f / l;  // no state at all
    ((T *)p.H.ptr)[cross_row(p, p.H, b, k, r) + c] = from_f32<T>(sum * inv);
    if (p.lse && c == 0) p.lse[f] = l == 0.f ? -INFINITY : M * (1.f / kLog2e) + logf(l);
}

// 16 bytes of a row per thread, the row's threads (2^log2 of them) next to one another in a warp.  Bound by
// memory.
template <typename T>
__global__ void __launch_bounds__(256) cross_delta_kernel(const CrossProblem p, float *delta, int total, int log2, Divide by_rows) {
    constexpr int V = 16 / sizeof(T);
    grid_dependency_wait();
    grid_dependents_launch();
    const int f = (int)(blockIdx.x * (256u >> log2) + (threadIdx.x >> log2));
    const int c = (int)(threadIdx.x & ((1u << log2) - 1)) * V;
    float s = 0.f;
    if (f < total) {
        const int bk = by_rows.of(f), r = f - bk * p.rows, b = p.by_kv.of(bk), k = bk - b * p.kv;
        T h[V], g[V];
        *reinterpret_cast<uint4 *>(h) = *reinterpret_cast<const uint4 *>((const T *)p.H.ptr + cross_row(p, p.H, b, k, r) + c);
        *reinterpret_cast<uint4 *>(g) = *reinterpret_cast<const uint4 *>((const T *)p.dH.ptr + cross_row(p, p.dH, b, k, r) + c);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(to_f32(h[i]), to_f32(g[i]), s);
    }
    for (int o = 1 << log2 >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (f < total && c == 0) delta[f] = s;
}

}  // namespace

cudaError_t launch_cross_join(const CrossProblem &p, const CrossParts &w, cudaStream_t stream) {
    const long long total = (long long)p.B * p.kv * p.rows;
    const dim3 grid((unsigned)total);
    return p.f32 ? launch_pdl(cross_join_kernel<float>, grid, dim3(256), 0, stream, p, w, total)
                 : launch_pdl(cross_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, p, w, total);
}

cudaError_t launch_cross_delta(const CrossProblem &p, float *delta, cudaStream_t stream) {
    const int total = p.B * p.kv * p.rows;
    int log2 = 0;
    while ((16 << log2) < p.d * (p.f32 ? 4 : 2)) ++log2;
    const dim3 grid((unsigned)(((long long)total + (256 >> log2) - 1) / (256 >> log2)));
    const Divide by_rows((uint32_t)p.rows);
    return p.f32 ? launch_pdl(cross_delta_kernel<float>, grid, dim3(256), 0, stream, p, delta, total, log2, by_rows)
                 : launch_pdl(cross_delta_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, p, delta, total, log2, by_rows);
}

namespace {

CrossView lower(const View &v) { return CrossView{v.ptr, v.sb, v.sh, v.sn}; }

anchor_attn_status_t cross(const anchor_attn_cross_t *a, bool bwd, void *stream_v) {
    if (!a) return ANCHOR_ATTN_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_v;
    if ((a->dtype != 0 && a->dtype != 1) || a->B < 0 || a->heads < 0 || a->kv_heads < 0 || a->n < 0 || a->s < 0)
        return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (a->d != 16 && a->d != 32 && a->d != 64 && a->d != 128) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (!isfinite(a->scale)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (a->B == 0 || a->heads == 0) {
        return a->heads == 0 && a->kv_heads > 0 && a->B > 0 && a->s > 0 ? ANCHOR_ATTN_ERR_INVALID_ARG : ANCHOR_ATTN_OK;
    }
    if (a->kv_heads == 0 || a->heads % a->kv_heads) return ANCHOR_ATTN_ERR_INVALID_ARG;
    // (room for the tiles that counts and walks add to a size, in 32 bits)
    if ((long long)a->n + a->s > (0x80000000LL - 1024) / ((long long)a->B * a->heads)) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    // (a backward has a tile and more of each kind for each of them, in one grid)
    if ((long long)a->B * a->kv_heads > 1LL << 29) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (((uintptr_t)a->lse & 3u) || ((uintptr_t)a->lengths & 3u)) return ANCHOR_ATTN_ERR_INVALID_ARG;

    CrossProblem p = {};
    p.B = a->B, p.heads = a->heads, p.kv = a->kv_heads, p.group = a->heads / a->kv_heads;
    p.n = a->n, p.s = a->s, p.d = a->d, p.rows = p.group * a->n;
    p.by_n = Divide((uint32_t)std::max(1, a->n)), p.by_kv = Divide((uint32_t)a->kv_heads);
    p.scale = a->scale, p.f32 = a->dtype == 1;
    p.lse = a->lse, p.lengths = a->lengths;
    const int es = p.f32 ? 4 : 2;
    const bool queries = a->n > 0, states = a->s > 0;
    View in[6], out[3];
    const void *in_dense[2] = {a->lengths, bwd ? a->lse : nullptr};
    const size_t rows_bytes = (size_t)a->B * a->heads * a->n * 4;
    const size_t in_dense_bytes[2] = {(size_t)a->B * 4, rows_bytes};
    int nin = 0, nout = 0;
    anchor_attn_status_t st = ANCHOR_ATTN_OK;
    auto add = [&](const anchor_attn_view_t &v, bool q, bool writes, CrossView &to) {
        if (st != ANCHOR_ATTN_OK || !(q ? queries : states)) return;
        const View w = make_view(v, a->B, q ? a->heads : a->kv_heads, q ? a->n : a->s, a->d, es);
        st = check_view(w, writes);
        if (writes) out[nout++] = w;
        else in[nin++] = w;
        to = lower(w);
    };
    add(a->Q, true, false, p.Q);
    add(a->K, false, false, p.K);
    add(a->V, false, false, p.V);
    add(a->H, true, !bwd, p.H);
    if (bwd) {
        add(a->dH, true, false, p.dH);
        add(a->dQ, true, true, p.dQ);
        add(a->dK, false, true, p.dK);
        add(a->dV, false, true, p.dV);
        if (queries && !a->lse) return ANCHOR_ATTN_ERR_INVALID_ARG;
    }
    if (st != ANCHOR_ATTN_OK) return st;
    for (int o = 0; o < nout; ++o) {
        for (int i = 0; i < nin; ++i)
            if (views_overlap(out[o], in[i])) return ANCHOR_ATTN_ERR_ALIAS;
        for (int i = 0; i < o; ++i)
            if (views_overlap(out[o], out[i])) return ANCHOR_ATTN_ERR_ALIAS;
        for (int i = 0; i < 2; ++i)
            if (in_dense[i] && bytes_overlap(out[o].ptr, (size_t)out[o].extent(), in_dense[i], in_dense_bytes[i]))
                return ANCHOR_ATTN_ERR_ALIAS;
        if (!bwd && a->lse && bytes_overlap(out[o].ptr, (size_t)out[o].extent(), a->lse, rows_bytes))
            return ANCHOR_ATTN_ERR_ALIAS;
    }
    if (!bwd && a->lse) {
        for (int i = 0; i < nin; ++i)
            if (bytes_overlap(a->lse, rows_bytes, in[i].ptr, (size_t)in[i].extent())) return ANCHOR_ATTN_ERR_ALIAS;
        if (a->lengths && bytes_overlap(a->lse, rows_bytes, a->lengths, (size_t)a->B * 4)) return ANCHOR_ATTN_ERR_ALIAS;
    }
    if (!queries && !(bwd && states)) return ANCHOR_ATTN_OK;

    cudaError_t e = cudaSuccess;
    void *ws = nullptr;
    auto take = [&](size_t bytes) -> bool {
        if (getenv("ANCHOR_ATTN_TEST_FAIL_ALLOC") != nullptr) return false;
        if (workspace_alloc(&ws, bytes, stream) == cudaSuccess) return true;
        cudaGetLastError();
        return false;
    };
    if (!bwd) {
        CrossPlan plan = p.f32 ? CrossPlan{cross_simt_parts(p), true} : cross_tc_plan(p);
        CrossParts w = {nullptr, nullptr, plan.parts};
        const bool join = plan.parts > 1 && plan.workspace;
        if (join) {
            const size_t total = (size_t)p.B * p.kv * p.rows * w.parts;
            if (!take(total * (p.d * 4 + 8))) return ANCHOR_ATTN_ERR_ALLOC;
            w.o = (float *)ws;
            w.ml = (float2 *)(w.o + total * p.d);
        }
        e = p.f32 ? launch_cross_simt_forward(p, w, stream) : launch_cross_tc_forward(p, w, stream);
        if (e == cudaSuccess && join) e = launch_cross_join(p, w, stream);
    } else {
        // D, and the sums of a backward whose steps are cut into parts
        const size_t d_bytes = (rows_bytes + 255) / 256 * 256, sums_bytes = p.f32 || !queries ? 0 : cross_tc_backward_sums(p);
        if (queries && !take(d_bytes + sums_bytes)) return ANCHOR_ATTN_ERR_ALLOC;
        float *delta = (float *)ws, *sums = queries ? delta + d_bytes / 4 : nullptr;
        if (p.f32) {
            if (queries) e = launch_cross_delta(p, delta, stream);
            if (e == cudaSuccess) e = launch_cross_simt_backward(p, delta, stream);
        } else {
            e = launch_cross_tc_backward(p, delta, sums, stream);
        }
    }
    if (ws) {
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

anchor_attn_status_t anchor_attn_cross_forward(const anchor_attn_cross_t *p, void *stream) {
    return anchor::cross(p, false, stream);
}

anchor_attn_status_t anchor_attn_cross_backward(const anchor_attn_cross_t *p, void *stream) {
    return anchor::cross(p, true, stream);
}

}  // extern "C"
