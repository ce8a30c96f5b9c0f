// Attention with decaying states: the problem as the launches see it (formulas and layout in
// include/anchor_attn.h).
//
// Forward and gradients have one form.  With g = exp(log_decay), a pass takes rows a, b, c and a state X,
//   o_i = sum_{j <= i} p g^(i-j) (a_i . b_j) c_j + w g^(i+1) a_i X,   X' = g^L X + s sum_j g^(L-1-j) b_j^T c_j
// and a pass backward in time the same with the rows of an entry in the other order, where the state that a row
// sees is one step nearer (its own row's step is not taken: w g^i):
//   H   (q, k, v)   X = state                        p = w = scale, s = 1
//   dQ  (dh, v, k)  X = state transposed             p = w = scale, s = 1
//   dK  (v, dh, q)  X = dlast transposed, backward   p = s = scale, w = 1
//   dV  (k, q, dh)  X = dlast, backward              p = s = scale, w = 1;  its X' is dstate
#pragma once

#include "cross.cuh"

#include <math.h>

namespace anchor {

struct DecayPass {
    CrossView a, b, c, o;
    float p, w, s;
    int back;             // backward in time
    int turned;           // the state is held transposed, [c][b]
    const float *state;   // [B][heads][d][d] or null for zeros
    float *last;          // the same, or null
    int kind;             // of the state: which of the workspace's
};

struct DecayProblem {
    DecayPass pass[3];
    int passes;
    const float *log_decay;  // [heads]
    const int *lengths;      // [B] or null
    int B, heads, n, d;
    bool f32;
    // A long sequence is cut into segments of `seg` rows.  states: [kind][B * heads][segs][d][d], first the sums of
    // each segment alone, then the states that they begin with.
    int segs, seg, kinds;
    float *states;
    __host__ __device__ long long slices() const { return (long long)B * heads; }
};

__device__ __forceinline__ int decay_length(const DecayProblem &p, int b) {
    return p.lengths ? min(max(__ldg(p.lengths + b), 0), p.n) : p.n;
}
// log_decay as it is used: at most 0, and finite, so that its product with 0 is 0 (exp(-1e4) is 0).
__device__ __forceinline__ float decay_rate(const float *log_decay, int h) {
    const float g = __ldg(log_decay + h);
    return g > 0.f ? 0.f : g < -1e4f ? -1e4f : g;
}
// What fp32 leaves of a factor keep = exp(x), x = rate count.  Rounded the same way each time, the factors of a sequence's chunks would add
// up (2^-24 of a state for each), so what they leave is made good.  For x above -1/2 from the series of exp(x) - 1, with what
// the square and the product x leave too: off by 2^-26 at most (half a step of x^3 / 6 and what follows), by 2^-31 above -1/8.
// Below, none: by the time that n factors' 2^-24 have added up no more than e^(-n / 2) is left.
__device__ __forceinline__ float decay_rest(float rate, float count, float keep) {
    const float x = rate * count, s = x * x;
    float u = 1.f / 362880.f;
    u = fmaf(x, u, 1.f / 40320.f), u = fmaf(x, u, 1.f / 5040.f), u = fmaf(x, u, 1.f / 720.f), u = fmaf(x, u, 1.f / 120.f);
    u = fmaf(x, u, 1.f / 24.f), u = fmaf(x, u, 1.f / 6.f), u = fmaf(s * x, u, 0.5f * fmaf(x, x, -s));
    // 1 + x + s / 2 + u, the larger ones first, each sum with what it leaves
    const float a = fmaf(0.5f, s, x), one = 1.f + a, left = ((1.f - one) + a) + (fmaf(0.5f, s, x - a) + u) + fmaf(rate, count, -x);
    return x > -0.5f ? (one - keep) + left : 0.f;
}
// The factor of the next chunk, with what those before have left (`owed`), and what it leaves itself: the product of a
// sequence's factors is never off by more than a rounding.
__device__ __forceinline__ float decay_next(float keep, float rest, float &owed) {
    owed += rest;
    const float by = keep + owed;
    owed = (keep - by) + owed;
    return by;
}
// the rows of segment `s` that count, of an entry with L
__device__ __forceinline__ int decay_rows(const DecayProblem &p, int s, int L) { return min(max(L - s * p.seg, 0), p.seg); }

// The sums of each segment but the last (in time) of each kind, and the passes: fp32, CUDA cores
cudaError_t launch_decay_simt_states(const DecayProblem &p, cudaStream_t stream);
cudaError_t launch_decay_simt(const DecayProblem &p, cudaStream_t stream);
// bf16, tensor cores
cudaError_t launch_decay_tc_states(const DecayProblem &p, cudaStream_t stream);
cudaError_t launch_decay_tc(const DecayProblem &p, cudaStream_t stream);
cudaError_t decay_read_and_clear_error(unsigned *out);

// Token by token, the state in registers.
struct DecayStep {
    CrossView Q, K, V, H;
    const float *log_decay;
    const int *lengths;      // [B] or null
    const int *slots;        // [B] or null: where an entry's state lies
    const float *from;       // states before, or null for zeros
    float *to;               // states behind, or null
    int B, heads, n, d, count;  // count: of slots
    float scale;
};
cudaError_t launch_decay_step(const DecayStep &p, bool f32, cudaStream_t stream);

}  // namespace anchor
