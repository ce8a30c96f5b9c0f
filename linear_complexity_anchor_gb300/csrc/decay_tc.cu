// Attention with decaying states in bf16 on the tensor cores (formulas in decay.cuh).
//
// A CTA walks the rows of one batch entry's head (or of a segment of it) in chunks of 128.  With i, j rows of a
// chunk of `count`, X the state before it (d x d, fp32, in tensor memory) and X~ its bf16 image in shared memory:
//   S = a b^T,  P = g^(i-j) S below the diagonal (bf16, over S),  o = p P c + w g^(i+1) (a X~)
//   X <- g^count X + (s g^(count-1-j) b_j)^T c
// (a pass backward in time: the other triangle, g^(j-i), g^(count-1-i), g^(j+1), chunks from the last to the first).
//
// Roundings: P and X~ to bf16, each once, where they meet c and a; the rows g^(count-1-j) b_j are two bf16
// numbers (what the first leaves of them is the second), so that X is exact to 2^-17 or better: it is an fp32
// result, and its own rounding in X~ stays the only one of the part of o that goes by it.  With one number o
// would carry three roundings there, 1.7 times a lone one, against 1.4.
//
// Warps 0 to 3 (rows): P from S, and o from the two products; a thread a row.  Warps 4 to 7 (state): X~ and the decay of X, a
// thread a row of X; the rows of b times their weights, in place, a thread a row, with their second numbers in a
// tile of their own.  Warp 8 loads tiles by TMA into a ring (a, b, c of each chunk in turn), warp 9 issues
// the products, in the order S, a X~, P c, X.  Tensor memory: S (P over it), the two products of o and X; at 64 columns a X~
// lies over the half of S that P leaves, and two CTAs share an SM.
//
// STATES: the sums of a segment alone, s sum_j g^(rows-1-j) b_j^T c_j: the last product alone, with weights that count from the
// segment's end, so that X needs no decay on the way; all eight warps weight rows.
#include "cross_tc.cuh"
#include "decay.cuh"

namespace anchor {

__device__ unsigned int g_decay_error;  // bit 0: a wait gave up

namespace {

using namespace cross_tc;

// D columns (heads of 16 and 32 are 64)
template <int D, bool STATES>
struct Geo {
    static constexpr int kPerSM = D == 64 ? 2 : 1;
    static constexpr int kSlots = STATES && D == 128 ? 6 : 5, kPer = STATES ? 2 : 3;  // tiles of the ring and of a chunk
    static constexpr int kImgBytes = D * D * 2;
    // With 64 columns X's product has 128 rows all the same, of which the upper 64 are not read: their operand
    // starts kHalf behind the tile's start, which has to be within the buffer.
    static constexpr int kHalf = D == 64 ? kImgBytes : kBlock;
    static constexpr int kLo = 0, kRing = kTile<D>, kImg = kRing + kSlots * kTile<D>;
    static constexpr int kPow = kImg + (STATES && D == 128 ? 0 : kImgBytes);
    static constexpr int kBars = kPow + 132 * 4, kNBars = 2 * kSlots + 8, kSmem = kBars + kNBars * 8 + 16 + 1024;
    static constexpr int kLoad = 8, kIssue = 9, kThreads = 320;
    static constexpr uint32_t kColS = 0, kColIn = 128, kColBy = D == 64 ? 64 : 256, kColX = STATES ? 0 : D == 64 ? 192 : 384;
    static constexpr uint32_t kCols = STATES ? D : D == 64 ? 256 : 512;
    static_assert((kSmem + 1024) * kPerSM <= 228 * 1024, "shared memory");
};

struct TcParams {
    DecayProblem p;
    TileMap a[3], b[3], c[3];
};

// The 16-byte chunks [from, to) of a row of b, times its weight w, as two bf16 numbers: the first in place, the second in `lo`.
// `on`: the row counts (else zeros, whatever it holds).
__device__ __forceinline__ void weight_row(uint8_t *tile, uint8_t *lo, int row, int from, int to, float w, bool on) {
    const uint64_t w2 = f32x2(w, w);
#pragma unroll 4
    for (int c = from; c < to; ++c) {
        const uint32_t at = chunk_at(row, c);
        const uint4 raw = *reinterpret_cast<const uint4 *>(tile + at);
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t x = mul_f32x2(f32x2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u)), w2);
            float x0, x1, r0, r1;
            f32x2_split(x, x0, x1);
            h[i] = pack2(x0, x1);
            // (what is left is exact)
            f32x2_split(add_f32x2(x, f32x2(-__uint_as_float(h[i] << 16), -__uint_as_float(h[i] & 0xffff0000u))), r0, r1);
            l[i] = pack2(r0, r1);
            if (!on) h[i] = l[i] = 0u;
        }
        *reinterpret_cast<uint4 *>(tile + at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// X += (hi + lo)^T c: both d x 128 operands contracted over the rows
template <int D, int kHalf>
__device__ __forceinline__ void product_x(uint32_t x, uint32_t hi, uint32_t lo, uint32_t c, bool add) {
    constexpr uint32_t id = idesc_bf16_f32(kRows, D, true, true);
    const uint64_t h = smem_desc_sw128(hi, kHalf, 1024), l = smem_desc_sw128(lo, kHalf, 1024), cd = desc_mn(c);
#pragma unroll
    for (int k = 0; k < kRows / 16; ++k) umma_bf16(x, h + step_mn(k), cd + step_mn(k), id, k > 0 || add ? 1u : 0u);
#pragma unroll
    for (int k = 0; k < kRows / 16; ++k) umma_bf16(x, l + step_mn(k), cd + step_mn(k), id, 1u);
}

template <int D, bool STATES>
__global__ void __launch_bounds__(Geo<D, STATES>::kThreads, Geo<D, STATES>::kPerSM) decay_kernel(const __grid_constant__ TcParams a) {
    using G = Geo<D, STATES>;
    constexpr int NS = G::kSlots, PER = G::kPer;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *pw = reinterpret_cast<float *>(sm + G::kPow);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G::kBars);
    uint64_t *full = bars, *empty = full + NS, *s_full = empty + NS, *p_full = s_full + 1, *o_full = p_full + 1, *o_free = o_full + 1,
             *img_full = o_free + 1, *b_full = img_full + 1, *x_full = b_full + 1, *done = x_full + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + G::kNBars);
    const DecayProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 4);
        mbar_init(o_full, 1);
        mbar_init(o_free, 4);
        mbar_init(img_full, D / 32);
        mbar_init(b_full, STATES ? 8 : 4);
        mbar_init(x_full, 1);
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == G::kIssue) tmem_alloc(s_tmem, G::kCols);
    grid_dependency_wait();
    grid_dependents_launch();

    // the passes of a segment are neighbours, so that what they share is read once
    const int kinds = STATES ? p.kinds : p.passes, index = blockIdx.x / kinds, of = blockIdx.x - index * kinds;
    const int segs = STATES ? p.segs - 1 : p.segs;
    const int slice = index / segs, b = slice / p.heads, h = slice - b * p.heads;
    int which = of;
    if (STATES)
        while (p.pass[which].kind != of) ++which;  // a pass of that kind
    const DecayPass &q = p.pass[which];
    const bool back = q.back;
    const int seg = index - slice * segs + (STATES && back ? 1 : 0);  // the last one (in time) has no state behind it
    const int L = decay_length(p, b), rows = decay_rows(p, seg, L), r0 = seg * p.seg;
    const float rate = decay_rate(p.log_decay, h);
    if (threadIdx.x <= kRows) pw[threadIdx.x] = expf(rate * (float)threadIdx.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    const bool turned = STATES ? false : q.turned;
    // STATES: b and c in the order of the kind, not turned
    const TileMap &map_a = a.a[which], &map_b = STATES && q.turned ? a.c[which] : a.b[which], &map_c = STATES && q.turned ? a.b[which] : a.c[which];
    const int K = (rows + kRows - 1) / kRows;
    const int dd = p.d * p.d;
    const float *from = STATES ? nullptr : p.segs > 1 ? p.states + (((long long)q.kind * p.slices() + slice) * p.segs + seg) * dd
                                                      : q.state ? q.state + (long long)slice * dd : nullptr;
    float *to = STATES ? p.states + (((long long)of * p.slices() + slice) * p.segs + seg) * dd
                       : q.last && seg == (back ? 0 : p.segs - 1) ? q.last + (long long)slice * dd : nullptr;
    const bool begun = from != nullptr;
    // chunk k's first row in the segment, its rows; whether X takes it
    auto first_of = [&](int k) { return (back ? K - 1 - k : k) * kRows; };
    auto count_of = [&](int k) { return min(kRows, rows - first_of(k)); };
    auto takes = [&](int k) { return STATES || k + 1 < K || to != nullptr; };
    unsigned int *error = &g_decay_error;
    auto slot = [&](int t) { return sm + G::kRing + t % NS * kTile<D>; };
    auto parity = [](int t) { return (uint32_t)((t / NS) & 1); };

    if (warp == G::kLoad) {
        if (lane == 0) {
            int t = 0;
            bool ok = true;
            for (int k = 0; k < K && ok; ++k) {
                const int row = r0 + first_of(k);
#pragma unroll
                for (int x = 0; x < PER; ++x, ++t) {
                    if (t >= NS && !(ok = bwait(empty + t % NS, parity(t - NS), error))) break;
                    const TileMap &m = PER == 2 ? (x == 0 ? map_b : map_c) : x == 0 ? map_a : x == 1 ? map_b : map_c;
                    mbar_arrive_expect_tx(full + t % NS, kTile<D>);
                    load_tile<D, kRows, kRows>(slot(t), m, full + t % NS, row, h, b);
                }
            }
            // the CTA leaves only once its copies have landed
            for (int x = max(0, t - NS); x < t; ++x) bwait(full + x % NS, parity(x), error);
        }
        __syncwarp();
    } else if (warp == G::kIssue) {
        if (lane == 0) {
            const uint32_t base = smem_u32(sm), lo = base + G::kLo;
            auto at = [&](int t) { return base + G::kRing + t % NS * kTile<D>; };
            constexpr uint32_t idS = idesc_bf16_f32(kRows, kRows, false, false), idO = idesc_bf16_f32(kRows, D, false, true);
            const int steps = (p.d + 15) / 16;
            bool ok = true;
            int images = 0;
            for (int k = 0; k < K && ok; ++k) {
                const int t = k * PER;
                const uint32_t par = (uint32_t)(k & 1), before = par ^ 1u;
                if constexpr (STATES) {
                    if (!(ok = bwait(full + (t + 1) % NS, parity(t + 1), error) && bwait(b_full, par, error))) break;
                    tc_fence_after();
                    product_x<D, G::kHalf>(tmem + G::kColX, at(t), lo, at(t + 1), k > 0);
                    umma_commit(x_full);
                    umma_commit(empty + t % NS);
                    umma_commit(empty + (t + 1) % NS);
                    continue;
                }
                const bool has = begun || k > 0, partial = count_of(k) < kRows;
                if (!(ok = bwait(full + t % NS, parity(t), error) && bwait(full + (t + 1) % NS, parity(t + 1), error))) break;
                if (D == 64 && k > 0 && !(ok = bwait(o_free, before, error))) break;
                tc_fence_after();
                product_k<D>(tmem + G::kColS, desc_k(at(t)), desc_k(at(t + 1)), idS, steps, [] {});
                umma_commit(s_full);
                if (D == 128 && k > 0 && !(ok = bwait(o_free, before, error))) break;
                if (D == 64 && !(ok = bwait(p_full, par, error))) break;
                if (has) {
                    if (!(ok = bwait(img_full, (uint32_t)(images & 1), error))) break;
                    ++images;
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        umma_bf16(tmem + G::kColBy, desc_k(at(t)) + step_k(s), desc_mn(base + G::kImg) + step_mn(s), idO, s > 0 ? 1u : 0u);
                }
                umma_commit(empty + t % NS);
                if (D == 128 && !(ok = bwait(p_full, par, error))) break;
                if (!(ok = bwait(full + (t + 2) % NS, parity(t + 2), error))) break;
                // (rows of c behind the length are zeros by then)
                if (partial && !(ok = bwait(b_full, par, error))) break;
                tc_fence_after();
                product_mn<64, kRows>(tmem + G::kColIn, tmem + G::kColS, desc_mn(at(t + 2)), idO, kRows / 16, false);
                umma_commit(o_full);
                if (takes(k)) {
                    if (!partial && !(ok = bwait(b_full, par, error))) break;
                    tc_fence_after();
                    product_x<D, G::kHalf>(tmem + G::kColX, at(t + 1), lo, at(t + 2), has);
                    umma_commit(x_full);
                }
                umma_commit(empty + (t + 1) % NS);
                umma_commit(empty + (t + 2) % NS);
            }
            umma_commit(done);
            bwait(done, 0u, error);
        }
        __syncwarp();
    } else {
        const int w4 = warp & 3, row = w4 * 32 + lane;
        const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
        if constexpr (STATES) {
            // both groups: half of the columns each
            const int half = warp >> 2;
            bool ok = true;
            for (int k = 0; k < K && ok; ++k) {
                const int t = k * PER, first = first_of(k), count = count_of(k);
                if (!(ok = bwait(full + t % NS, parity(t), error))) break;
                if (count < kRows && !(ok = bwait(full + (t + 1) % NS, parity(t + 1), error))) break;
                if (k > 0 && !(ok = bwait(x_full, (uint32_t)((k - 1) & 1), error))) break;
                const float w = q.s * expf(rate * (float)(back ? first + row + 1 : rows - 1 - first - row));
                weight_row(slot(t), sm + G::kLo, row, half * D / 16, (half + 1) * D / 16, w, row < count);
                if (half == 0 && count < kRows) zero_rows<D>(slot(t + 1), row, count, kRows);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_full);
            }
            if (ok && K > 0) ok = bwait(x_full, (uint32_t)((K - 1) & 1), error);
            tc_fence_after();
            if (ok && w4 * 32 < D) {
                const int c0 = half * D / 2;
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    float x[32];
                    if (K > 0) {
                        tmem_ld32(tmem + lanes + G::kColX + c0 + c, x);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = 0.f;
                    }
                    if (row < p.d) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (c0 + c + i < p.d) *reinterpret_cast<float4 *>(to + row * p.d + c0 + c + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                    }
                }
            }
        } else if (warp < 4) {
            // ------------------------------------------------------------------ rows
            __nv_bfloat16 *O = (__nv_bfloat16 *)q.o.ptr + b * q.o.sb + h * q.o.sh;
            bool ok = true;
            for (int k = 0; k < K && ok; ++k) {
                const uint32_t par = (uint32_t)(k & 1);
                const int count = count_of(k);
                const bool has = begun || k > 0;
                if (!(ok = bwait(s_full, par, error))) break;
                tc_fence_after();
#pragma unroll 1
                for (int j0 = 0; j0 < kRows; j0 += 32) {
                    uint32_t packed[16];
                    // blocks on the other side of the diagonal are not read
                    if (back ? j0 + 31 < w4 * 32 || j0 >= count : j0 > w4 * 32 + 31) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) packed[x] = 0u;
                    } else {
                        float s[32];
                        tmem_ld32(tmem + lanes + G::kColS + j0, s);
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const int j = j0 + x, far = back ? j - row : row - j;
                            s[x] = far >= 0 && (!back || j < count) ? s[x] * pw[max(far, 0)] : 0.f;
                        }
#pragma unroll
                        for (int x = 0; x < 16; ++x) packed[x] = pack2(s[2 * x], s[2 * x + 1]);
                    }
                    tmem_st16(tmem + lanes + G::kColS + j0 / 2, packed);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
                if (!(ok = bwait(o_full, par, error))) break;
                tc_fence_after();
                const float f = q.w * pw[back ? max(count - 1 - row, 0) : row + 1];
                __nv_bfloat16 *to_row = O + (long long)(r0 + first_of(k) + row) * q.o.sn;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float in[32];
                    tmem_ld32(tmem + lanes + G::kColIn + c, in);
                    if (has) {
                        float by[32];
                        tmem_ld32(tmem + lanes + G::kColBy + c, by);
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 32; ++x) in[x] = fmaf(f, by[x], q.p * in[x]);
                    } else {
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 32; ++x) in[x] *= q.p;
                    }
                    if (c + 32 == D) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_free);
                    }
                    if (row < count) {
#pragma unroll
                        for (int x = 0; x < 32; x += 8)
                            if (c + x < p.d)
                                *reinterpret_cast<uint4 *>(to_row + c + x) =
                                    make_uint4(pack2(in[x], in[x + 1]), pack2(in[x + 2], in[x + 3]), pack2(in[x + 4], in[x + 5]), pack2(in[x + 6], in[x + 7]));
                    }
                }
            }
            // rows of the segment from the length on
            const int end = min(p.seg, p.n - r0), per = p.d / 8;
            for (int e = threadIdx.x; e < max(end - rows, 0) * per; e += 128)
                *reinterpret_cast<uint4 *>(O + (long long)(r0 + rows + e / per) * q.o.sn + e % per * 8) = make_uint4(0, 0, 0, 0);
        } else {
            // ------------------------------------------------------------------ state
            const bool mine = w4 * 32 < D;  // the warp has rows of X
            bool ok = true;
            for (int k = 0; k < K && ok; ++k) {
                const int t = k * PER, count = count_of(k);
                if (k > 0 && !(ok = bwait(x_full, (uint32_t)((k - 1) & 1), error))) break;
                tc_fence_after();
                if ((begun || k > 0) && mine) {
                    const float keep = pw[count];
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float x[32];
                        if (k > 0) {
                            tmem_ld32(tmem + lanes + G::kColX + c, x);
                            tmem_ld_wait();
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[i] = row < p.d && c + i < p.d ? (turned ? from[(c + i) * p.d + row] : from[row * p.d + c + i]) : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4 *>(sm + G::kImg + chunk_at(row, (c + i) / 8)) =
                                make_uint4(pack2(x[i], x[i + 1]), pack2(x[i + 2], x[i + 3]), pack2(x[i + 4], x[i + 5]), pack2(x[i + 6], x[i + 7]));
                        if (takes(k)) {
                            uint32_t y[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(x[i] * keep);
                            tmem_st32(tmem + lanes + G::kColX + c, y);
                        }
                    }
                    tmem_st_wait();
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(img_full);
                }
                if (takes(k)) {
                    // the tile has landed, and S has read it
                    if (!(ok = bwait(full + (t + 1) % NS, parity(t + 1), error) && bwait(s_full, (uint32_t)(k & 1), error))) break;
                    weight_row(slot(t + 1), sm + G::kLo, row, 0, D / 8, q.s * pw[back ? row + 1 : max(count - 1 - row, 0)], row < count);
                }
                if (count < kRows) {
                    if (!(ok = bwait(full + (t + 2) % NS, parity(t + 2), error))) break;
                    zero_rows<D>(slot(t + 2), row, count, kRows);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_full);
            }
            if (to && mine && ok && (K == 0 || (ok = bwait(x_full, (uint32_t)((K - 1) & 1), error)))) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float x[32];
                    if (K > 0) {
                        tmem_ld32(tmem + lanes + G::kColX + c, x);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = from && row < p.d && c + i < p.d ? (turned ? from[(c + i) * p.d + row] : from[row * p.d + c + i]) : 0.f;
                    }
                    if (row < p.d) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < p.d) {
                                if (turned) to[(c + i) * p.d + row] = x[i];
                                else to[row * p.d + c + i] = x[i];
                            }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == G::kIssue) tmem_dealloc(tmem, G::kCols);
}

template <int D, bool STATES>
cudaError_t launch(const DecayProblem &p, cudaStream_t stream) {
    TcParams a;
    a.p = p;
    for (int i = 0; i < p.passes; ++i) {
        const DecayPass &q = p.pass[i];
        if (!make_tile_map(&a.a[i], q.a, p.B, p.heads, p.n, p.d, kRows) || !make_tile_map(&a.b[i], q.b, p.B, p.heads, p.n, p.d, kRows) ||
            !make_tile_map(&a.c[i], q.c, p.B, p.heads, p.n, p.d, kRows))
            return cudaErrorInvalidValue;
    }
    static SmemOnce once;
    const cudaError_t e = once(decay_kernel<D, STATES>, Geo<D, STATES>::kSmem);
    if (e != cudaSuccess) return e;
    const long long ctas = p.slices() * (STATES ? p.segs - 1 : p.segs) * (STATES ? p.kinds : p.passes);
    return launch_pdl(decay_kernel<D, STATES>, dim3((unsigned)ctas), dim3(Geo<D, STATES>::kThreads), Geo<D, STATES>::kSmem, stream, a);
}

}  // namespace

cudaError_t launch_decay_tc_states(const DecayProblem &p, cudaStream_t stream) {
    return p.d == 128 ? launch<128, true>(p, stream) : launch<64, true>(p, stream);
}
cudaError_t launch_decay_tc(const DecayProblem &p, cudaStream_t stream) {
    return p.d == 128 ? launch<128, false>(p, stream) : launch<64, false>(p, stream);
}
cudaError_t decay_read_and_clear_error(unsigned *out) {
    const unsigned zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(out, g_decay_error, sizeof(unsigned));
    return e == cudaSuccess ? cudaMemcpyToSymbol(g_decay_error, &zero, sizeof(unsigned)) : e;
}

}  // namespace anchor
