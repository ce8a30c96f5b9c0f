// Attention with decaying states, token by token (formulas in include/anchor_attn.h): few tokens, whose states
// are read, moved on and written.
//
// A CTA takes CB columns of one head's state (columns are independent of one another), held in registers by 256
// threads, four columns a thread and every (256 / (CB / 4))-th row; a token's h is summed over a warp's rows by
// shuffles and over the warps through shared memory, in a fixed order.  Bound by reading and writing the states: 64 requests, 32
// heads, d = 128, bf16: 46 us, 5.8 TB/s with six CTAs an SM (48.5 with as many as the registers gave; 16 columns a CTA 67, 64: 49).
// Several tokens are bound by latency, one after the other, each fetched and summed between barriers: 2 tokens 58, 4: 81, 8: 136.  Shared
// slots: each CTA reads all B slots, which counts from about a thousand requests on (with slots and without: 1024 x 4 heads, d = 128: 98, 84; 4096 x 2: 235,
// 164; 16384 x 1, d = 64: 374, 112).
// One size for all, so that a request's bits do not depend on the batch.
#include "decay.cuh"

namespace anchor {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kColumns = 32;

template <typename T, int D, int CB>
__global__ void __launch_bounds__(kThreads, 6) decay_step_kernel(const __grid_constant__ DecayStep p) {
    constexpr int W = CB / 4, R = kThreads / W, N = (D + R - 1) / R, kBlocks = D / CB;  // threads a row, rows at a time, rows a thread
    __shared__ __align__(16) float sq[2][D], sk[2][D], sv[2][CB];
    __shared__ float4 part[2][kWarps][W];
    __shared__ int s_next, s_before;
    grid_dependency_wait();
    grid_dependents_launch();
    const int cb = blockIdx.x % kBlocks, at = blockIdx.x / kBlocks, h = at % p.heads;
    int b = at / p.heads;
    const int slot = p.slots ? __ldg(p.slots + b) : b;
    const bool held = slot >= 0 && slot < p.count;
    const int w = threadIdx.x % W, r = threadIdx.x / W, c0 = cb * CB;
    const long long offset = ((long long)slot * p.heads + h) * D * D + c0 + 4 * w;
    float4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (held && p.from && (D % R == 0 || r < D)) x[i] = *reinterpret_cast<const float4 *>(p.from + offset + (long long)(r + i * R) * D);
    }
    const float rate = decay_rate(p.log_decay, h), g = expf(rate), rest = decay_rest(rate, 1.f, g);
    // Entries that share a slot are taken in order by the CTA of the first.
    bool more = false;
    if (p.slots && held) {
        if (threadIdx.x == 0) s_next = p.B, s_before = 0;
        __syncthreads();
        for (int e = threadIdx.x; e < p.B; e += kThreads)
            if (e != b && __ldg(p.slots + e) == slot) {
                if (e < b) s_before = 1;
                else atomicMin(&s_next, e);
            }
        __syncthreads();
        if (s_before) return;
        more = s_next < p.B;
    }
    int buf = 0;
    for (;;) {
        const int L = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.n) : p.n;
        const T *Q = (const T *)p.Q.ptr + b * p.Q.sb + h * p.Q.sh, *K = (const T *)p.K.ptr + b * p.K.sb + h * p.K.sh,
                *V = (const T *)p.V.ptr + b * p.V.sb + h * p.V.sh;
        T *H = (T *)p.H.ptr + b * p.H.sb + h * p.H.sh;
        for (int t = 0; t < p.n; ++t, buf ^= 1) {
            const bool on = held && t < L;
            if (!on) {  // the same for all threads
                if (threadIdx.x < CB) H[t * p.H.sn + c0 + threadIdx.x] = from_f32<T>(0.f);
                continue;
            }
            for (int e = threadIdx.x; e < 2 * D + CB; e += kThreads) {
                if (e < D) sq[buf][e] = to_f32(Q[t * p.Q.sn + e]);
                else if (e < 2 * D) sk[buf][e - D] = to_f32(K[t * p.K.sn + e - D]);
                else sv[buf][e - 2 * D] = to_f32(V[t * p.V.sn + c0 + e - 2 * D]);
            }
            __syncthreads();
            const float4 v = *reinterpret_cast<const float4 *>(&sv[buf][4 * w]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (D % R != 0 && r >= D) continue;
                const float k = sk[buf][r + i * R], q = sq[buf][r + i * R];
                x[i].x = fmaf(x[i].x, g, fmaf(x[i].x, rest, k * v.x)), x[i].y = fmaf(x[i].y, g, fmaf(x[i].y, rest, k * v.y));
                x[i].z = fmaf(x[i].z, g, fmaf(x[i].z, rest, k * v.z)), x[i].w = fmaf(x[i].w, g, fmaf(x[i].w, rest, k * v.w));
                o.x = fmaf(q, x[i].x, o.x), o.y = fmaf(q, x[i].y, o.y), o.z = fmaf(q, x[i].z, o.z), o.w = fmaf(q, x[i].w, o.w);
            }
#pragma unroll
            for (int s = W; s < 32; s <<= 1) {
                o.x += __shfl_xor_sync(0xffffffffu, o.x, s), o.y += __shfl_xor_sync(0xffffffffu, o.y, s);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, s), o.w += __shfl_xor_sync(0xffffffffu, o.w, s);
            }
            if ((threadIdx.x & 31) < W) part[buf][threadIdx.x >> 5][w] = o;
            __syncthreads();
            if (threadIdx.x < CB) {
                float sum = 0.f;
#pragma unroll
                for (int y = 0; y < kWarps; ++y) sum += reinterpret_cast<const float *>(part[buf][y])[threadIdx.x];
                H[t * p.H.sn + c0 + threadIdx.x] = from_f32<T>(sum * p.scale);
            }
        }
        if (!more) break;
        b = s_next;
        __syncthreads();
        if (threadIdx.x == 0) s_next = p.B;
        __syncthreads();
        for (int e = b + 1 + threadIdx.x; e < p.B; e += kThreads)
            if (__ldg(p.slots + e) == slot) atomicMin(&s_next, e);
        __syncthreads();
        more = s_next < p.B;
    }
    if (held && p.to) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (D % R == 0 || r < D) *reinterpret_cast<float4 *>(p.to + offset + (long long)(r + i * R) * D) = x[i];
    }
}

template <typename T, int D>
cudaError_t launch(const DecayStep &p, cudaStream_t stream) {
    constexpr int CB = D < kColumns ? D : kColumns;
    const long long ctas = (long long)p.B * p.heads * (D / CB);
    return launch_pdl(decay_step_kernel<T, D, CB>, dim3((unsigned)ctas), dim3(kThreads), 0, stream, p);
}

template <typename T>
cudaError_t launch(const DecayStep &p, cudaStream_t stream) {
    switch (p.d) {
    case 16: return launch<T, 16>(p, stream);
    case 32: return launch<T, 32>(p, stream);
    case 64: return launch<T, 64>(p, stream);
    default: return launch<T, 128>(p, stream);
    }
}

}  // namespace

cudaError_t launch_decay_step(const DecayStep &p, bool f32, cudaStream_t stream) {
    return f32 ? launch<float>(p, stream) : launch<__nv_bfloat16>(p, stream);
}

}  // namespace anchor
