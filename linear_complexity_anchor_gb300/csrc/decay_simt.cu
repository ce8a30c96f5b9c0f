// Attention with decaying states on CUDA cores, fp32 throughout (formulas in decay.cuh).
//
// A CTA walks the rows of one batch entry's head (or of a segment of it) in chunks of 64, for CB columns of c
// and of the state:
//   S = a b^T (64 x 64), P = p g^(i-j) S below the diagonal, o = w g^(i+1) a X + P c,
//   X = g^64 X + s sum_j g^(63-j) b_j^T c_j.
// 16 x 16 threads; X is kept in registers, with a copy in shared memory for a X.  In blocks of 64 columns every number is read from
// shared memory for four uses at least, in blocks of 32 those of a and P for two, of 16 for one.  (64 + CB) (64 + d) FMAs per row at CB columns, of
// which 64 d are done again for each block of columns.  4 x 16 heads, 4096, d = 128: 1168 us forward, of which the FMAs would take 320: with
// eight warps an SM (137 KB of shared memory each CTA, whose tiles are fetched between two barriers, one chunk at a time, and nothing runs
// meanwhile) an instruction is issued every other cycle, and a warp waits 0.9 cycles of each 3.9 for tiles and 0.75 for shared memory.  8 x 12 heads,
// 4200, d = 64: 611 us forward (three segments; one: 958), 1293 backward.
#include "decay.cuh"

namespace anchor {
namespace {

constexpr int kC = 64, kThreads = 256;

template <int D, int CB> struct Geo {
    static constexpr int kPitch = D + 4, kPitchC = CB + 4, kPitchP = kC + 4;
    static constexpr int kA = 0, kB = kA + kC * kPitch, kCc = kB + kC * kPitch, kX = kCc + kC * kPitchC, kP = kX + D * kPitchC,
                         kPow = kP + kC * kPitchP, kFloats = kPow + kC + 4;
    static constexpr int kNC = CB / 16, kNB = D / 16;  // columns of c and rows of X of a thread
};

// rows [first, first + 64) of a view's columns [col, col + W), those from `rows` on zero
template <int W>
__device__ __forceinline__ void load(float *to, int pitch, const float *from, long long step, int rows, int col) {
    constexpr int kPer = W / 4;
    for (int x = threadIdx.x; x < kC * kPer; x += kThreads) {
        const int r = x / kPer, e = x % kPer * 4;
        *reinterpret_cast<float4 *>(to + r * pitch + e) =
            r < rows ? *reinterpret_cast<const float4 *>(from + r * step + col + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// N neighbouring floats, as wide as they are aligned
template <int N> __device__ __forceinline__ void take(const float *p, float *v) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(v + i) = *reinterpret_cast<const float4 *>(p + i);
    } else if constexpr (N == 2) {
        *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(p);
    } else {
        v[0] = p[0];
    }
}
template <int N> __device__ __forceinline__ void give(float *p, const float *v) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v[i];
}

// acc[4][NC] += x[4 rows][k] y[k][NC columns], k < K: x rows of pitch px, y rows of pitch py
template <int K, int NC>
__device__ __forceinline__ void product(const float *x, int px, const float *y, int py, float (&acc)[4][NC]) {
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float a[4][4], b[4][NC];
#pragma unroll
        for (int i = 0; i < 4; ++i) take<4>(x + i * px + k, a[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) take<NC>(y + (k + j) * py, b[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(a[i][j], b[j][c], acc[i][c]);
    }
}

// STATES: the sums of a segment alone (of `kind` blockIdx.y), else a pass (blockIdx.y).
template <int D, int CB, bool STATES>
__global__ void __launch_bounds__(kThreads) decay_simt_kernel(const __grid_constant__ DecayProblem p) {
    using G = Geo<D, CB>;
    constexpr int NC = G::kNC, NB = G::kNB, kBlocks = D / CB;
    extern __shared__ __align__(16) float sm[];
    float *sA = sm + G::kA, *sB = sm + G::kB, *sC = sm + G::kCc, *sX = sm + G::kX, *sP = sm + G::kP, *pw = sm + G::kPow;
    grid_dependency_wait();
    grid_dependents_launch();
    const int cb = blockIdx.x % kBlocks, at = blockIdx.x / kBlocks;
    const int segs = STATES ? p.segs - 1 : p.segs;
    const long long slice = at / segs;
    const int b = (int)(slice / p.heads), h = (int)(slice - (long long)b * p.heads);
    int which = blockIdx.y;
    if (STATES)
        while (p.pass[which].kind != (int)blockIdx.y) ++which;  // a pass of that kind
    const DecayPass &q = p.pass[which];
    const bool back = q.back;
    const int seg = at % segs + (STATES && back ? 1 : 0);  // the last one (in time) has no state behind it
    const int L = decay_length(p, b), rows = decay_rows(p, seg, L), r0 = seg * p.seg;
    const float rate = decay_rate(p.log_decay, h);
    // STATES: b and c in the order of the kind, not turned
    const bool turned = STATES ? false : q.turned;
    const CrossView &vb = STATES && q.turned ? q.c : q.b, &vc = STATES && q.turned ? q.b : q.c;
    const float *A = (const float *)q.a.ptr + b * q.a.sb + h * q.a.sh, *Bm = (const float *)vb.ptr + b * vb.sb + h * vb.sh,
            *Cm = (const float *)vc.ptr + b * vc.sb + h * vc.sh;
    float *O = (float *)q.o.ptr + b * q.o.sb + h * q.o.sh;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, c0 = cb * CB + tx * NC;
    if (threadIdx.x <= kC) pw[threadIdx.x] = expf(rate * (float)threadIdx.x);

    float x[NB][NC];
    const long long slot = (long long)slice * D * D;
    const float *from = STATES ? nullptr : p.segs > 1 ? p.states + (((long long)q.kind * p.slices() + slice) * p.segs + seg) * D * D
                                                      : q.state ? q.state + slot : nullptr;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int r = ty * NB + i;
            x[i][c] = !from ? 0.f : turned ? from[(c0 + c) * D + r] : from[r * D + c0 + c];
        }
    const int chunks = (rows + kC - 1) / kC;
    // what fp32 leaves of a whole chunk's factor of X (one that is not whole adds a rounding), and has left of those before
    const float rest = decay_rest(rate, (float)kC, expf(rate * (float)kC));
    float owed = 0.f;
    for (int k = 0; k < chunks; ++k) {
        const int first = (back ? chunks - 1 - k : k) * kC, count = min(kC, rows - first);
        const long long r = r0 + first;
        __syncthreads();
        if (!STATES) {
            load<D>(sA, G::kPitch, A + r * q.a.sn, q.a.sn, count, 0);
#pragma unroll
            for (int i = 0; i < NB; ++i) give<NC>(sX + (ty * NB + i) * G::kPitchC + tx * NC, x[i]);
        }
        load<D>(sB, G::kPitch, Bm + r * vb.sn, vb.sn, count, 0);
        load<CB>(sC, G::kPitchC, Cm + r * vc.sn, vc.sn, count, cb * CB);
        __syncthreads();
        if (!STATES) {
            float s[4][4] = {};
#pragma unroll 4
            for (int e = 0; e < D; e += 4) {
                float a4[4][4], b4[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) take<4>(sA + (ty * 4 + i) * G::kPitch + e, a4[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) take<4>(sB + (tx + 16 * j) * G::kPitch + e, b4[j]);
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a4[i][y], b4[j][y], s[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int y = ty * 4 + i, z = tx + 16 * j, far = back ? z - y : y - z;
                    sP[y * G::kPitchP + z] = far >= 0 ? s[i][j] * (q.p * pw[far]) : 0.f;
                }
            float o[4][NC] = {};
            product<D, NC>(sA + ty * 4 * G::kPitch, G::kPitch, sX + tx * NC, G::kPitchC, o);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int y = ty * 4 + i;
                const float f = y < count ? q.w * pw[back ? count - 1 - y : y + 1] : 0.f;
#pragma unroll
                for (int c = 0; c < NC; ++c) o[i][c] *= f;
            }
            product<kC, NC>(sP + ty * 4 * G::kPitchP, G::kPitchP, sC + tx * NC, G::kPitchC, o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int y = ty * 4 + i;
                if (y >= count) continue;
                float *to = O + (r + y) * q.o.sn + c0;
#pragma unroll
                for (int c = 0; c < NC; ++c) to[c] = o[i][c];
            }
        }
        float keep = pw[count];
        if (count == kC) keep = decay_next(keep, rest, owed);
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) x[i][c] *= keep;
#pragma unroll 4
        for (int j = 0; j < count; ++j) {
            const float f = q.s * pw[back ? j + 1 : count - 1 - j];
            float y[NB], z[NC];
            take<NB>(sB + j * G::kPitch + ty * NB, y);
            take<NC>(sC + j * G::kPitchC + tx * NC, z);
#pragma unroll
            for (int c = 0; c < NC; ++c) z[c] *= f;
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) x[i][c] = fmaf(y[i], z[c], x[i][c]);
        }
    }
    if (!STATES) {
        // rows of the segment from the length on
        const int end = min(p.seg, p.n - r0);
        const long long left = max(end - rows, 0) * (long long)CB;
        for (long long e = threadIdx.x; e < left; e += kThreads)
            O[(long long)(r0 + rows + e / CB) * q.o.sn + cb * CB + e % CB] = 0.f;
    }
    float *to = STATES ? p.states + (((long long)blockIdx.y * p.slices() + slice) * p.segs + seg) * D * D
                       : q.last && seg == (back ? 0 : p.segs - 1) ? q.last + slot : nullptr;
    if (to) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int r = ty * NB + i;
                if (turned) to[(c0 + c) * D + r] = x[i][c];
                else to[r * D + c0 + c] = x[i][c];
            }
    }
}

template <int D, int CB, bool STATES>
cudaError_t launch(const DecayProblem &p, cudaStream_t stream) {
    static SmemOnce once;
    constexpr size_t smem = Geo<D, CB>::kFloats * 4;
    cudaError_t e = once(decay_simt_kernel<D, CB, STATES>, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(p.slices() * (STATES ? p.segs - 1 : p.segs) * (D / CB)), STATES ? p.kinds : p.passes);
    return launch_pdl(decay_simt_kernel<D, CB, STATES>, grid, dim3(kThreads), smem, stream, p);
}

// Heads of 64 and 128 columns go in blocks of 64, or of 32 where blocks of 64 leave half of the SMs without one (us in blocks of
// 64 and 32: 4 x 6 heads x 197, d = 64, 24 CTAs of 64 columns 48, 40, backward, 72: 50, 42; 4 heads x 1000, d = 128, backward, 96:
// 106, 124; 8 x 12 x 4200, d = 64, 96: 974, 994; 4 x 16 x 4096, d = 128, 128: 1184, 1344).
template <bool STATES>
cudaError_t launch(const DecayProblem &p, cudaStream_t stream) {
    const long long ctas = p.slices() * p.segs * p.passes * (p.d / 64);
    const bool narrow = 2 * ctas <= kPlanSMs;
    switch (p.d) {
    case 16: return launch<16, 16, STATES>(p, stream);
    case 32: return launch<32, 32, STATES>(p, stream);
    case 64: return narrow ? launch<64, 32, STATES>(p, stream) : launch<64, 64, STATES>(p, stream);
    default: return narrow ? launch<128, 32, STATES>(p, stream) : launch<128, 64, STATES>(p, stream);
    }
}

}  // namespace

cudaError_t launch_decay_simt_states(const DecayProblem &p, cudaStream_t stream) {
    return launch<true>(p, stream);
}
cudaError_t launch_decay_simt(const DecayProblem &p, cudaStream_t stream) {
    return launch<false>(p, stream);
}

}  // namespace anchor
