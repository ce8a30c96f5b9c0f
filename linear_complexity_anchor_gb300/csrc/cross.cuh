// Cross attention: the problem as the launches see it (formulas and layout in
// include/anchor_attn.h).  Query rows are taken per key head: row r of key head k is query
// r % n of head k * group + r / n, so that the heads that share keys fill one tile.
#pragma once

#include "common.cuh"
#include "views.cuh"

namespace anchor {

struct CrossView {
    const void *ptr;
    long long sb, sh, sn;  // strides in elements
};

// Division by a number that the launch knows, as a product: for d > 0 and x < 2^31,
// x / d = (x + hi(x m)) >> l with l = ceil(log2 d), m = floor(2^32 (2^l - d) / d) + 1 (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994).
struct Divide {
    uint32_t d = 1, m = 1, l = 0;
    Divide() = default;
    explicit Divide(uint32_t by) : d(by) {
        while ((1ull << l) < by) ++l;
        m = (uint32_t)(((1ull << 32) * ((1ull << l) - by)) / by + 1);
    }
    __device__ __forceinline__ int of(int x) const { return (int)((__umulhi(m, (uint32_t)x) + (uint32_t)x) >> l); }
};

struct CrossProblem {
    CrossView Q, K, V, H, dH, dQ, dK, dV;
    float *lse;           // [B][heads][n] or null
    const int *lengths;   // [B] or null
    int B, heads, kv, group, n, s, d;
    int rows;             // group * n
    Divide by_n, by_kv;
    float scale;
    bool f32;
};

__device__ __forceinline__ int cross_length(const CrossProblem &p, int b) {
    return p.lengths ? min(max(__ldg(p.lengths + b), 0), p.s) : p.s;
}
// row r of key head k: its offset in a [B][heads][n][d] view
__device__ __forceinline__ long long cross_row(const CrossProblem &p, const CrossView &v, int b, int k, int r) {
    const int g = p.by_n.of(r), i = r - g * p.n;
    return b * v.sb + (long long)(k * p.group + g) * v.sh + (long long)i * v.sn;
}
// ... and in a dense [B][heads][n] array
__device__ __forceinline__ long long cross_flat(const CrossProblem &p, int b, int k, int r) {
    return ((long long)b * p.kv + k) * p.rows + r;  // the group's heads follow one another
}

// From here on scores (and lse, in log2) are rounded too coarsely for c s - m in one rounding.
constexpr float kFar = 0x1p20f;
// lse in log2 as the backward takes it, P = 2^(c s - lse).  It has been rounded six times (m, two factors, a product and a
// sum in the forward, its product with log2 e here; half a step each), which would take P past any range where lse is far.
// There it is raised by three and a half steps, so that P is at most 1.
__device__ __forceinline__ float far_lse(float x) { return fabsf(x) > kFar ? fmaf(fabsf(x), 0x1.cp-22f, x) : x; }

// The parts of a forward whose keys are cut over several CTAs: unnormalised sums and (maximum in
// units of log2, sum) per part, [parts][B * kv * rows][d] and [parts][B * kv * rows].
struct CrossParts {
    float *o;
    float2 *ml;
    int parts;
};
cudaError_t launch_cross_join(const CrossProblem &p, const CrossParts &w, cudaStream_t stream);
// D_r = dH_r . H_r, [B][heads][n] (fp32)
cudaError_t launch_cross_delta(const CrossProblem &p, float *delta, cudaStream_t stream);

// CUDA cores, fp32 arithmetic
int cross_simt_parts(const CrossProblem &p);
cudaError_t launch_cross_simt_forward(const CrossProblem &p, const CrossParts &w, cudaStream_t stream);
cudaError_t launch_cross_simt_backward(const CrossProblem &p, const float *delta, cudaStream_t stream);

// tensor cores, bf16
struct CrossPlan {
    int parts;       // of the key axis
    bool workspace;  // their sums go through a workspace and a second launch
};
CrossPlan cross_tc_plan(const CrossProblem &p);
cudaError_t launch_cross_tc_forward(const CrossProblem &p, const CrossParts &w, cudaStream_t stream);
// workspaces: D [B][heads][n], and sums of this many bytes
size_t cross_tc_backward_sums(const CrossProblem &p);
cudaError_t launch_cross_tc_backward(const CrossProblem &p, float *delta, float *sums, cudaStream_t stream);
cudaError_t cross_bwd_read_and_clear_error(unsigned *out);
cudaError_t cross_fwd_read_and_clear_error(unsigned *out);

}  // namespace anchor
