// Attention with decaying states: argument checks, plan and launch; the states that segments begin with
// (formulas and layout in include/anchor_attn.h and decay.cuh).
#include "decay.cuh"

#include <stdlib.h>

namespace anchor {
namespace {

// Four elements of one slice's states a thread: along the segments in time, the sums of a segment alone
// are replaced by the state before it.  Bound by the latency of loads from L2, of which kAhead are in flight (2 heads, d = 128, 16384
// rows: 9.4 us; in one number and with one load at a time it took 13.2, with eight 8.1).  The walk is carried as two numbers, and its factors with what fp32 leaves of them, so that a state is
// rounded once, however many segments there are.
constexpr int kAhead = 8;
struct Walk {
    float x, left = 0.f;
    // x <- x keep (1 + what fp32 leaves of keep) + t
    __device__ __forceinline__ void step(float keep, float rest, float t) {
        const float p = x * keep, s = p + t, b = s - p;
        left = fmaf(left, keep, fmaf(x, rest, fmaf(x, keep, -p))) + ((p - (s - b)) + (t - b));
        x = s + left;
        left = (s - x) + left;
    }
};
__global__ void __launch_bounds__(256) decay_prefix_kernel(const __grid_constant__ DecayProblem p) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int dd = p.d * p.d, per = dd / 4;
    const long long f = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int kind = blockIdx.y;
    if (f >= p.slices() * per) return;
    const long long slice = f / per;
    const int e = (int)(f - slice * per) * 4, b = (int)(slice / p.heads), h = (int)(slice - (long long)b * p.heads);
    int which = 0;
    while (p.pass[which].kind != kind) ++which;
    const bool back = p.pass[which].back;
    const float *first = p.pass[which].state;
    const float rate = decay_rate(p.log_decay, h);
    const int L = decay_length(p, b);
    const float4 from = first ? *reinterpret_cast<const float4 *>(first + slice * dd + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    Walk x{from.x}, y{from.y}, z{from.z}, w{from.w};
    // factors of whole segments, and of the one that the length ends in
    auto factor = [&](int rows) {
        const float keep = expf(rate * (float)rows);
        return make_float2(keep, decay_rest(rate, (float)rows, keep));
    };
    float2 whole, part;
    const float2 none = make_float2(1.f, 0.f);
    float *at = p.states + ((long long)kind * p.slices() + slice) * p.segs * dd + e;
    for (int k0 = 0; k0 < p.segs; k0 += kAhead) {
        float4 t[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + i, s = back ? p.segs - 1 - k : k;
            // (nothing is behind the last one)
            t[i] = k + 1 < p.segs ? __ldcg(reinterpret_cast<const float4 *>(at + (long long)s * dd)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (k0 == 0) whole = factor(p.seg), part = factor(L % p.seg);  // (while the first loads are under way)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + i, s = back ? p.segs - 1 - k : k, rows = decay_rows(p, s, L);
            if (k < p.segs) *reinterpret_cast<float4 *>(at + (long long)s * dd) = make_float4(x.x, y.x, z.x, w.x);
            const float2 f = rows == p.seg ? whole : rows > 0 ? part : none;
            if (k + 1 < p.segs) x.step(f.x, f.y, t[i].x), y.step(f.x, f.y, t[i].y), z.step(f.x, f.y, t[i].z), w.step(f.x, f.y, t[i].w);
        }
    }
}

CrossView lower(const View &v) { return CrossView{v.ptr, v.sb, v.sh, v.sn}; }

// What a call reads and writes, to find overlaps.
struct Regions {
    struct Dense { const void *ptr; size_t bytes; };
    View in[5], out[3];
    Dense din[5], dout[1];
    int nin = 0, nout = 0, ndin = 0, ndout = 0;
    void reads(const void *ptr, size_t bytes) {
        if (ptr && bytes) din[ndin++] = Dense{ptr, bytes};
    }
    void writes(const void *ptr, size_t bytes) {
        if (ptr && bytes) dout[ndout++] = Dense{ptr, bytes};
    }
    bool overlap() const {
        auto meets = [](const View &v, const Dense &x) { return bytes_overlap(v.ptr, (size_t)v.extent(), x.ptr, x.bytes); };
        for (int o = 0; o < nout; ++o) {
            for (int i = 0; i < nin; ++i)
                if (views_overlap(out[o], in[i])) return true;
            for (int i = 0; i < o; ++i)
                if (views_overlap(out[o], out[i])) return true;
            for (int i = 0; i < ndin; ++i)
                if (meets(out[o], din[i])) return true;
            for (int i = 0; i < ndout; ++i)
                if (meets(out[o], dout[i])) return true;
        }
        for (int o = 0; o < ndout; ++o) {
            for (int i = 0; i < nin; ++i)
                if (meets(in[i], dout[o])) return true;
            for (int i = 0; i < ndin; ++i)
                if (bytes_overlap(dout[o].ptr, dout[o].bytes, din[i].ptr, din[i].bytes)) return true;
        }
        return false;
    }
};

// The sizes that every call has.
anchor_attn_status_t check_sizes(int dtype, int B, int heads, int n, int d, float scale) {
    if ((dtype != 0 && dtype != 1) || B < 0 || heads < 0 || n < 0) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (d != 16 && d != 32 && d != 64 && d != 128) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (!isfinite(scale)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (B == 0 || heads == 0) return ANCHOR_ATTN_OK;
    if ((long long)B * heads > 1LL << 24 || (long long)n > (0x80000000LL - 1024) / ((long long)B * heads)) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    return ANCHOR_ATTN_OK;
}

bool misaligned(const void *p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

// Segments of a sequence: as many as take the least time, by what 128 rows of an item (64 columns of one pass of one head) take,
// in a pass and for a segment's sums, in us, what an item takes to begin and to end, rounds of items over the SMs, two launches
// more, and the segments' states, one after the other and through L2.  None where the items fill the SMs: segments read b and c
// twice.  Measured (us): bf16, d = 128, 4 x 16 heads x 16384: one segment 250, two 314; 2 x 16 x 8192: 121, 101, three 121;
// 16 x 16384: one 231, two 170, four 104, eight 110; 16 x 2049: one 36, four 30; d = 64, 8 x 12 x 4200: one 51, two 77; 12 x
// 16384: one 164, ten 44; one head of 32768: one 319, ten 61, 32: 32; fp32, d = 64, 8 x 12 x 4200: one 957, three 611; 4 x 12 x
// 2000: one 363, six 180; d = 128, 4 x 16 x 4096: one 1168, two 1451; d = 32, 16 x 12 x 2000: one 337, four 309.
void plan(DecayProblem &p) {
    const long long slices = p.slices(), halves = p.d == 128 ? 2 : 1;
    const float item = 2.2f, launches = 8.f;
    // fp32: CTAs an SM (by their shared memory), each of which takes 0.3 more for each beside it; narrow ones take three quarters
    const int beside = !p.f32 || p.d == 128 ? 1 : p.d == 64 ? 2 : 4;
    const float each128 = p.f32 ? p.d == 128 ? 37.f : p.d == 64 ? 29.f : 16.f : p.d == 128 ? 1.88f : 1.38f;
    const int tiles = (p.n + 127) / 128, most = (int)std::max<long long>(1, std::min<long long>(4 * kPlanSMs / (slices * halves), tiles / 2));
    auto time = [&](long long items, float rows128) {
        const long long a_sm = (items + kPlanSMs - 1) / kPlanSMs;
        const float pass = p.f32 && p.d >= 64 && 2 * items <= kPlanSMs ? 0.75f * each128 : each128;
        return (float)((a_sm + beside - 1) / beside) * (rows128 * pass * (0.7f + 0.3f * (float)std::min<long long>(beside, a_sm)) + item);
    };
    float best = 0.f;
    int want = 1;
    for (int s = 1; s <= most; ++s) {
        const float each = (float)((tiles + s - 1) / s);
        float t = time(slices * halves * p.passes * s, each);
        if (s > 1)
            t += time(slices * halves * p.kinds * (s - 1), 0.48f * each) + launches + 0.1f * (float)s + (float)(slices * p.kinds * s) * (float)(p.d * p.d) * 3e-6f;
        if (s == 1) best = t - 2.f;  // (the host's part of a call grows too: 12 x 1500, d = 64: 20 us, in segments 25)
        else if (t < best) best = t, want = s;
    }
    p.seg = (tiles + want - 1) / want * 128;
    p.segs = std::max(1, (int)(((long long)p.n + p.seg - 1) / p.seg));
}

// A call of few tokens goes token by token, which costs more with each, where a chunk costs the same for all.  Measured (us, by tokens and in a
// chunk, states in and out / neither): bf16, 64 x 32 heads, d = 128, 8 tokens: 137, 197 / 109, 109; 12: 194, 196 / 159, 108; d = 64, 8: 49, 82 / 45, 51;
// 12: 70, 82 / 63, 51; d = 16, 8: 25, 72 / 25, 51; 24: 66, 72 / 65, 52; 256 x 12, d = 64, 8: 76, 122 / 65, 74; 12: 107, 121 / 93, 74.  fp32,
// 64 x 32, d = 128, 16 tokens: 263, 415 / 215, 342; 32: 503, 455 / 489, 411; d = 64, 16: 99, 107 / 81, 96; 24: 146, 122 / 120, 103; d = 16, 12: 35, 37 / 34, 36; 16:
// 45, 38 / 44, 37.  Few heads take 13 to 20 both ways.  With states bf16 could go on to 12 to 24 tokens by d; the bits of H would
// then depend on whether there are any.
bool by_steps(const anchor_attn_decay_t *a) { return a->n <= (a->dtype ? 16 : 8); }

cudaError_t run(DecayProblem &p, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (p.segs > 1) {
        e = p.f32 ? launch_decay_simt_states(p, stream) : launch_decay_tc_states(p, stream);
        const long long threads = p.slices() * (p.d * p.d / 4);
        // few threads are spread over the SMs (2 heads, d = 128, 16384 rows: 9.4 us, in CTAs of 256 10.4; one head of 64: 13.0, 15.2; but 16
        // heads, d = 128, 2049 rows: a call takes 32.2 us with CTAs of 64, 31.5 with 256)
        const int each = threads <= kPlanSMs * 256 ? 64 : 256;
        if (e == cudaSuccess) e = launch_pdl(decay_prefix_kernel, dim3((unsigned)((threads + each - 1) / each), p.kinds), dim3(each), 0, stream, p);
    }
    if (e != cudaSuccess) return e;
    return p.f32 ? launch_decay_simt(p, stream) : launch_decay_tc(p, stream);
}

anchor_attn_status_t finish(cudaError_t e) {
    if (e == cudaSuccess) return ANCHOR_ATTN_OK;
    cudaGetLastError();
    return ANCHOR_ATTN_ERR_CUDA;
}

anchor_attn_status_t decay(const anchor_attn_decay_t *a, bool bwd, void *stream_v) {
    if (!a) return ANCHOR_ATTN_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_v;
    anchor_attn_status_t st = check_sizes(a->dtype, a->B, a->heads, a->n, a->d, a->scale);
    if (st != ANCHOR_ATTN_OK || a->B == 0 || a->heads == 0) return st;
    if (!a->log_decay || misaligned(a->log_decay, 4) || misaligned(a->lengths, 4)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (misaligned(a->state, 16) || misaligned(a->last, 16) || misaligned(a->dlast, 16) || misaligned(a->dstate, 16)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    const int es = a->dtype ? 4 : 2;
    const size_t state_bytes = (size_t)a->B * a->heads * a->d * a->d * 4;
    Regions g;
    CrossView Q{}, K{}, V{}, H{}, dH{}, dQ{}, dK{}, dV{};
    auto add = [&](const anchor_attn_view_t &v, bool writes, CrossView &to) {
        if (st != ANCHOR_ATTN_OK || a->n == 0) return;
        const View w = make_view(v, a->B, a->heads, a->n, a->d, es);
        st = check_view(w, writes);
        if (writes) g.out[g.nout++] = w;
        else g.in[g.nin++] = w;
        to = lower(w);
    };
    add(a->Q, false, Q);
    add(a->K, false, K);
    add(a->V, false, V);
    g.reads(a->log_decay, (size_t)a->heads * 4);
    g.reads(a->lengths, (size_t)a->B * 4);
    g.reads(a->state, state_bytes);
    if (!bwd) {
        add(a->H, true, H);
        g.writes(a->last, state_bytes);
    } else {
        add(a->dH, false, dH);
        add(a->dQ, true, dQ);
        add(a->dK, true, dK);
        add(a->dV, true, dV);
        g.reads(a->dlast, state_bytes);
        g.writes(a->dstate, state_bytes);
    }
    if (st != ANCHOR_ATTN_OK) return st;
    if (g.overlap()) return ANCHOR_ATTN_ERR_ALIAS;
    if (a->n == 0) {
        float *to = bwd ? a->dstate : a->last;
        const float *from = bwd ? a->dlast : a->state;
        if (!to) return ANCHOR_ATTN_OK;
        return finish(from ? cudaMemcpyAsync(to, from, state_bytes, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(to, 0, state_bytes, stream));
    }
    if (!bwd && by_steps(a)) {
        DecayStep s = {};
        s.Q = Q, s.K = K, s.V = V, s.H = H, s.log_decay = a->log_decay, s.lengths = a->lengths, s.from = a->state, s.to = a->last;
        s.B = a->B, s.heads = a->heads, s.n = a->n, s.d = a->d, s.count = a->B, s.scale = a->scale;
        return finish(launch_decay_step(s, a->dtype == 1, stream));
    }
    DecayProblem p = {};
    p.log_decay = a->log_decay, p.lengths = a->lengths, p.B = a->B, p.heads = a->heads, p.n = a->n, p.d = a->d, p.f32 = a->dtype == 1;
    const float c = a->scale;
    if (!bwd) {
        p.passes = p.kinds = 1;
        p.pass[0] = DecayPass{Q, K, V, H, c, c, 1.f, 0, 0, a->state, a->last, 0};
    } else {
        p.passes = 3, p.kinds = 2;
        p.pass[0] = DecayPass{dH, V, K, dQ, c, c, 1.f, 0, 1, a->state, nullptr, 0};
        p.pass[1] = DecayPass{V, dH, Q, dK, c, 1.f, c, 1, 1, a->dlast, nullptr, 1};
        p.pass[2] = DecayPass{K, Q, dH, dV, c, 1.f, c, 1, 0, a->dlast, a->dstate, 1};
    }
    plan(p);
    if (p.segs > 1) {
        if (getenv("ANCHOR_ATTN_TEST_FAIL_ALLOC") != nullptr) return ANCHOR_ATTN_ERR_ALLOC;
        if (workspace_alloc((void **)&p.states, state_bytes * p.segs * p.kinds, stream) != cudaSuccess) {
            cudaGetLastError();
            return ANCHOR_ATTN_ERR_ALLOC;
        }
    }
    cudaError_t e = run(p, stream);
    if (p.states) {
        const cudaError_t ef = cudaFreeAsync(p.states, stream);
        if (e == cudaSuccess) e = ef;
    }
    return finish(e);
}

anchor_attn_status_t decay_step(const anchor_attn_decay_step_t *a, void *stream_v) {
    if (!a) return ANCHOR_ATTN_ERR_INVALID_ARG;
    anchor_attn_status_t st = check_sizes(a->dtype, a->B, a->heads, a->n, a->d, a->scale);
    if (st != ANCHOR_ATTN_OK) return st;
    if (a->slot_count < 0 || (!a->slots && a->slot_count < a->B)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (a->heads > 0 && (long long)a->slot_count > (1LL << 40) / a->heads) return ANCHOR_ATTN_ERR_UNSUPPORTED;
    if (a->B == 0 || a->heads == 0 || a->n == 0) return ANCHOR_ATTN_OK;
    if (!a->log_decay || misaligned(a->log_decay, 4) || misaligned(a->slots, 4) || misaligned(a->states, 16)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (!a->states && a->slot_count > 0) return ANCHOR_ATTN_ERR_INVALID_ARG;
    const int es = a->dtype ? 4 : 2;
    Regions g;
    DecayStep s = {};
    const anchor_attn_view_t *in[3] = {&a->Q, &a->K, &a->V};
    CrossView *to[3] = {&s.Q, &s.K, &s.V};
    for (int i = 0; i < 3; ++i) {
        const View w = make_view(*in[i], a->B, a->heads, a->n, a->d, es);
        if ((st = check_view(w, false)) != ANCHOR_ATTN_OK) return st;
        g.in[g.nin++] = w;
        *to[i] = lower(w);
    }
    const View w = make_view(a->H, a->B, a->heads, a->n, a->d, es);
    if ((st = check_view(w, true)) != ANCHOR_ATTN_OK) return st;
    g.out[g.nout++] = w;
    s.H = lower(w);
    g.reads(a->log_decay, (size_t)a->heads * 4);
    g.reads(a->slots, (size_t)a->B * 4);
    g.writes(a->states, (size_t)a->slot_count * a->heads * a->d * a->d * 4);
    if (g.overlap()) return ANCHOR_ATTN_ERR_ALIAS;
    s.log_decay = a->log_decay, s.slots = a->slots, s.from = a->states, s.to = a->states;
    s.B = a->B, s.heads = a->heads, s.n = a->n, s.d = a->d, s.count = a->slot_count, s.scale = a->scale;
    return finish(launch_decay_step(s, a->dtype == 1, (cudaStream_t)stream_v));
}

}  // namespace
}  // namespace anchor

extern "C" {

anchor_attn_status_t anchor_attn_decay_forward(const anchor_attn_decay_t *p, void *stream) { return anchor::decay(p, false, stream); }

anchor_attn_status_t anchor_attn_decay_backward(const anchor_attn_decay_t *p, void *stream) { return anchor::decay(p, true, stream); }

anchor_attn_status_t anchor_attn_decay_step(const anchor_attn_decay_step_t *p, void *stream) { return anchor::decay_step(p, stream); }

}  // extern "C"
