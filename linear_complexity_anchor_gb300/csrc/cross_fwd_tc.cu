// Cross attention forward in bf16 on the tensor cores (formulas in include/anchor_attn.h).
//
// A CTA has one or two tiles of 128 query rows of one key head, and walks that head's keys in tiles of KT:
// S = Q K^T into tensor memory, a thread takes 64 columns of a row (two threads a row for KT = 128), the
// running maximum and sum, and leaves P = 2^(c s - m) as bf16 over S's columns, O += P V from there.
// (One thread for 128 columns was bound by its own latency: the tensor pipe 36 % active against 62 in 8 heads,
// 9728 x 2048, d = 128.)  Q is loaded with plain 16-byte loads (rows of several heads, any strides), K
// and V by TMA into a ring, K and V in turn, by a warp of their own; one thread of another warp issues
// the products.
//
// Two tiles: while the rows of one take their exponentials the tensor cores run the other's
//   P0 V -> O0, Q0 K' -> S0   |   P1 V -> O1, Q1 K' -> S1
// and each K and V tile is read from L2 once for 256 rows.  S and O of both fill the 512 columns
// at d = 128, so P lies over S: the products of one CTA run in the order they are issued, and the
// next S is issued after the P V that reads it.  Bound by that round of a tile, S, its rows, P V; 8 heads,
// 9728 x 2048, d = 128: 62 us, 1.3 PFLOP/s; 8 times that 1.36, with the power cap at 3 % of the clock.  At d = 64 keys go in tiles
// of 64, a thread a row, and two CTAs share an SM: 4 x 12 heads, 4200 x 1000: 75 us against 91 for tiles of 128.
// One tile (up to 128 rows, a token of serving above all): bound by reading K and V (64 entries of 5000 states,
// 8 heads of 128: 197 us, 6.6 TB/s).  At d = 128 S has two buffers, the next S is issued before the softmax
// of this one, and three stages of 64 KB are in flight; at d = 64 two CTAs share an SM.
// Few rows and long keys: the key tiles of an entry (of its own length) are cut over gridDim.y
// CTAs.  Up to eight are a cluster, which joins their sums over distributed shared memory; more leave them
// for a second launch (rule and reason at cross_tc_plan).
//
// The maximum a row is scaled by moves only when it grows by more than 2^8 over the one in use:
// P stays below 2^8, its relative rounding is the same, and O (in tensor memory) is rescaled
// rarely.  P is rounded to bf16 (the operand type of the product; its relative error of 2^-9 is that
// of rounding V); the row sum is taken over the fp32 values.
// Keys from the entry's length on: S masked by select, so that nothing they hold matters, and
// their rows of V are zeroed in shared memory (0 times an infinity is not 0).
#include "cluster.cuh"
#include "cross_tc.cuh"

#include <math.h>

namespace anchor {

__device__ unsigned int g_cross_fwd_error;  // bit 0: a wait gave up

namespace {

using namespace cross_tc;

constexpr float kSlack = 8.f;  // log2 of how far a maximum may be passed before O is rescaled

// What scores are scaled by, in log2 (the sign is Q's).  Not 0, so that a masked score stays -infinity: with a
// scale of 0 the scores are 0, by Q.
__device__ __forceinline__ float score_scale(const CrossProblem &p) { return p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e; }

// With a scale of 0: eight elements of Q times 0 (infinities and NaN are NaN then).
__device__ __forceinline__ void times_zero(uint4 *q) {
    __nv_bfloat162 *x = reinterpret_cast<__nv_bfloat162 *>(q);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __hmul2(x[i], __float2bfloat162_rn(0.f));
}

// D columns (heads of 16 and 32 are 64), NQ row tiles, key tiles of KT.
template <int D, int NQ, int KT>
struct Geo {
    static constexpr int kNH = KT / 64;                      // threads of a row, 64 columns of S each
    static constexpr int kNS = NQ == 1 && D == 128 ? 2 : 1;  // S buffers of a tile
    static constexpr int kStages = D == 128 ? (NQ == 1 ? 3 : 2) : (NQ == 1 ? 2 : 3);  // of a K and a V tile
    static constexpr int kPerSM = D == 64 ? 2 : 1;
    static constexpr int kRowWarps = 4 * kNH * NQ, kThreads = 32 * kRowWarps + 64;
    static constexpr int kStage = 2 * kTile<D, KT>;
    static constexpr int kQ = 0, kRing = NQ * kTile<D>, kEx = kRing + kStages * kStage;
    static constexpr int kBars = kEx + NQ * 2 * kRows * 4;
    static constexpr int kNBars = NQ + 2 * kStages + 2 * NQ * kNS + NQ + 4 * NQ + 1;
    static constexpr int kSmem = kBars + kNBars * 8 + 16 + 1024;
    // the join's sums and (m, l), over the ring
    static constexpr int kJoinPitch = D + 4, kJoinMl = kRing + kRows * kJoinPitch * 4;
    static_assert(NQ == 2 || kRows * (kJoinPitch * 4 + 8) <= kStages * kStage, "the join fits the ring");
    static constexpr uint32_t kColO = KT * NQ * kNS, kCols = kColO + NQ * D <= 256 ? 256 : 512;
    static_assert((kSmem + 1024) * kPerSM <= 228 * 1024, "shared memory");
    static_assert(kColO + NQ * D <= 512 && kCols * kPerSM <= 512, "tensor memory");
};

struct FwdParams {
    CrossProblem p;
    CrossParts w;
    TileMap k, v;
    int tiles;
    Divide by_tiles;
    bool cluster;  // the parts are a cluster's CTAs, which join them
};

template <int D, int NQ, int KT>
__global__ void __launch_bounds__(Geo<D, NQ, KT>::kThreads, Geo<D, NQ, KT>::kPerSM)
cross_fwd_kernel(const __grid_constant__ FwdParams a) {
    using G = Geo<D, NQ, KT>;
    constexpr int NS = G::kNS, ST = G::kStages, NH = G::kNH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G::kBars);
    uint64_t *q_full = bars, *full = q_full + NQ, *empty = full + ST, *s_full = empty + ST, *p_full = s_full + NQ * NS,
             *o_full = p_full + NQ * NS, *pair = o_full + NQ, *done = pair + 4 * NQ;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + G::kNBars);
    const CrossProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kLoad = G::kRowWarps, kIssue = kLoad + 1;
    const int bk = a.by_tiles.of((int)blockIdx.x), tile = (int)blockIdx.x - bk * a.tiles;
    const int b = p.by_kv.of(bk), kh = bk - b * p.kv, r0 = tile * NQ * kRows;
    const int left = p.rows - r0;                        // rows of this CTA that exist
    const int nq = NQ == 2 && left > kRows ? 2 : 1;

    if (threadIdx.x == 0) {
        for (int q = 0; q < NQ; ++q) {
            const int warps = min(max((left - q * kRows + 31) / 32, 1), 4);  // with a row that exists
            mbar_init(q_full + q, 4 * NH);
            mbar_init(o_full + q, 1);
            for (int w = 0; w < 4; ++w) mbar_init(pair + 4 * q + w, 2);
            for (int s = 0; s < NS; ++s) {
                mbar_init(s_full + q * NS + s, 1);
                mbar_init(p_full + q * NS + s, NH * warps);
            }
        }
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == kIssue) tmem_alloc(s_tmem, G::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dependency_wait();
    grid_dependents_launch();

    const int L = cross_length(p, b), key_tiles = (L + KT - 1) / KT;
    const int t0 = (int)((long long)key_tiles * blockIdx.y / a.w.parts);
    const int nt = (int)((long long)key_tiles * (blockIdx.y + 1) / a.w.parts) - t0;
    unsigned int *error = &g_cross_fwd_error;

    if (warp == kLoad) {
        if (lane == 0 && nt > 0) {
            tma_prefetch_desc(&a.k.map);
            tma_prefetch_desc(&a.v.map);
            // stage i: K of tile i, and V of tile i - NS, which are used at one time
            int i = 0;
            for (; i < nt + NS; ++i) {
                const int st = i % ST;
                if (i >= ST && !bwait(empty + st, (uint32_t)((i / ST - 1) & 1), error)) break;
                uint8_t *dst = sm + G::kRing + st * G::kStage;
                mbar_arrive_expect_tx(full + st, (i < nt ? kTile<D, KT> : 0) + (i >= NS ? kTile<D, KT> : 0));
                if (i >= NS) load_tile<D, KT, KT>(dst + kTile<D, KT>, a.v, full + st, (t0 + i - NS) * KT, kh, b);
                if (i < nt) load_tile<D, KT, KT>(dst, a.k, full + st, (t0 + i) * KT, kh, b);
            }
            // the CTA leaves only once its copies have landed
            for (int j = max(0, i - ST); j < i; ++j) bwait(full + j % ST, (uint32_t)((j / ST) & 1), error);
        }
        __syncwarp();
        // the rows and the first stages of the CTA that will follow on this SM, into L2
        const long long then = (long long)blockIdx.x + G::kPerSM * kPlanSMs;
        if (a.w.parts == 1 && then < (long long)gridDim.x) {
            const int bk2 = a.by_tiles.of((int)then), tile2 = (int)then - bk2 * a.tiles, b2 = p.by_kv.of(bk2), kh2 = bk2 - b2 * p.kv;
            if (lane < 2 && tile2 == 0) {
                const TileMap &m = lane ? a.v : a.k;
                for (int t = 0; t < ST && t * KT < p.s; ++t)
#pragma unroll
                    for (int q = 0; q < D / 64; ++q) prefetch_tile(&m.map, 64 * q, t * KT, kh2 * m.by_head, b2 * m.by_batch);
            }
            for (int x = tile2 * NQ * kRows + lane; x < min(p.rows, (tile2 + 1) * NQ * kRows); x += 32) {
                const char *q = (const char *)((const __nv_bfloat16 *)p.Q.ptr + cross_row(p, p.Q, b2, kh2, x));
                for (int y = 0; y < 2 * p.d; y += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + y));
            }
        }
    } else if (warp == kIssue) {
        if (lane == 0 && nt > 0) {
            // A tile's rows wait for S, this thread for their P, the rows for the next S: that round is
            // what a step takes, so between a P and its products there is nothing to do here but the wait
            // for it.  (A commit takes 70 cycles, a wait on a complete barrier 130.)  That the step's K
            // and V, in one stage, have landed is seen behind products.
            const int ksteps = (p.d + 15) / 16;
            const uint32_t base = smem_u32(sm), ring = base + G::kRing;
            const uint32_t idO = idesc_bf16_f32(kRows, p.d < D ? p.d : D, false, true);
            const uint32_t idS = idesc_bf16_f32(kRows, KT, false, false);
            const int last16 = (min(KT, L - (t0 + nt - 1) * KT) + 15) / 16 * 16;  // keys of the last tile, in 16s
            const uint32_t idL = idesc_bf16_f32(kRows, last16, false, false);
            const uint64_t qd0 = desc_k(base + G::kQ), kd0 = desc_k(ring), vd0 = desc_mn(ring + kTile<D, KT>);
            constexpr uint64_t kStep = G::kStage / 16, kNextQ = kTile<D> / 16;  // of descriptors
            auto nothing = [] {};
            bool ok = true;
            for (int i = 0; i < NS && ok; ++i) {
                if (i < nt) {
                    ok = bwait(full + i % ST, 0u, error);
                    for (int q = 0; q < nq && ok; ++q) {
                        if (i == 0) ok = bwait(q_full + q, 0u, error);
                        tc_fence_after();
                        if (!ok) break;
                        product_k<D>(tmem + KT * (q * NS + i), qd0 + q * kNextQ, kd0 + (i % ST) * kStep, i == nt - 1 ? idL : idS, ksteps, nothing);
                        umma_commit(s_full + q * NS + i);
                    }
                }
                umma_commit(empty + i % ST);
            }
            bool landed = false;  // this step's stage, as seen during the step before
            for (int j = 0; j < nt && ok; ++j) {
                const int i = j + NS, st = i % ST, steps = j == nt - 1 ? last16 / 16 : KT / 16;
                const uint64_t vd = vd0 + st * kStep, kd = kd0 + st * kStep;
                const uint32_t par = (uint32_t)((j / NS) & 1), id = i == nt - 1 ? idL : idS;
                if (!landed && !(ok = bwait(full + st, (uint32_t)((i / ST) & 1), error))) break;
                landed = false;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    if (q >= nq) break;
                    const uint32_t S = tmem + KT * (q * NS + j % NS);
                    if (!(ok = bwait(p_full + q * NS + j % NS, par, error))) break;
                    tc_fence_after();
                    product_mn<32, KT>(tmem + G::kColO + q * D, S, vd, idO, steps, j > 0);
                    if (NS == 2 || j == nt - 1) umma_commit(o_full + q);
                    if (i >= nt) continue;
                    product_k<D>(S, qd0 + q * kNextQ, kd, id, ksteps, [&] {
                        if (q == nq - 1) landed = mbar_test(full + (i + 1) % ST, (uint32_t)(((i + 1) / ST) & 1));
                    });
                    umma_commit(s_full + q * NS + j % NS);
                }
                umma_commit(empty + st);
            }
            umma_commit(done);
            bwait(done, 0u, error);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ rows
        // warp: tile q, columns 64 half .. + 63 of S, lanes 32 w4 .. + 31
        const int q = warp / (4 * NH), half = NH == 2 ? (warp >> 2) & 1 : 0, w4 = warp & 3;
        const int row = w4 * 32 + lane;                      // of the tile
        const int r = r0 + q * kRows + row;                  // of the key head
        const bool mine = r < p.rows;
        const bool active = r0 + q * kRows + w4 * 32 < p.rows;  // the warp has a row
        uint8_t *sQ = sm + G::kQ + q * kTile<D>;
        const float c = score_scale(p);
        // this warp's 32 rows by its part of the columns, 16 bytes a lane
        constexpr int kLanes = D / (8 * NH), kPart = D / NH;
        const int my_row = lane / kLanes, my_chunk = half * kLanes + lane % kLanes;
        if (nt > 0) {
            // Q, negated for a negative scale
            const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
            uint4 x[kLanes];
            each_row<kLanes>(mine ? cross_row(p, p.Q, b, kh, r) : -1, p.Q.sn, [&](int i, int, long long o) {
                x[i] = make_uint4(0, 0, 0, 0);
                if (o >= 0 && my_chunk * 8 < p.d) x[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)p.Q.ptr + o + my_chunk * 8);
            });
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                x[i].x ^= flip, x[i].y ^= flip, x[i].z ^= flip, x[i].w ^= flip;
                *reinterpret_cast<uint4 *>(sQ + chunk_at(w4 * 32 + i * (32 / kLanes) + my_row, my_chunk)) = x[i];
            }
            if (p.scale == 0.f)
                for (int i = 0; i < kLanes; ++i) times_zero(reinterpret_cast<uint4 *>(sQ + chunk_at(w4 * 32 + i * (32 / kLanes) + my_row, my_chunk)));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + q);
        }
        const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
        const uint32_t tO = tmem + lanes + G::kColO + q * D;
        // the two halves of a row meet over its slots [half], and over a barrier of their two warps
        float *ex = reinterpret_cast<float *>(sm + G::kEx + q * 2 * kRows * 4) + row;
        uint64_t *meet = pair + q * 4 + w4;
        // The maximum in use (of s), what it takes to move it, and this half's sum.  A score's exponent is c s - m in one
        // rounding, m = c u rounded before: P and its sum share 2^(what that left), up to 2^(2^-24 |m|), which H
        // does not see until it overflows.  A row whose m is far moves at every tile, where u is taken from s
        // instead, and shift, otherwise m, is 0.
        float u_max = -INFINITY, shift = 0.f, limit = -INFINITY, l = 0.f;
        bool ok = true;
        if (active && q < nq) {
            for (int j = 0; j < nt && ok; ++j) {
                const int buf = q * NS + j % NS;
                const uint32_t tS = tmem + lanes + KT * buf + 64 * half;
                if (!bwait(s_full + buf, (uint32_t)((j / NS) & 1), error)) { ok = false; break; }
                tc_fence_after();
                const int keys = min(KT, L - (t0 + j) * KT) - 64 * half;  // of this half that count (may be none)
                float s[64];
                tmem_ld32(tS, s);
                if (keys > 32) tmem_ld32(tS + 32, s + 32);
                tmem_ld_wait();
                if (keys < 64) {
#pragma unroll
                    for (int x = 0; x < 64; ++x)
                        if (x >= keys) s[x] = -INFINITY;
                }
                float t8[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) t8[x] = max3_f32(s[x], s[8 + x], s[16 + x]);
#pragma unroll
                for (int y = 24; y < 56; y += 16)
#pragma unroll
                    for (int x = 0; x < 8; ++x) t8[x] = max3_f32(t8[x], s[y + x], s[y + 8 + x]);
#pragma unroll
                for (int x = 0; x < 8; ++x) t8[x] = fmaxf(t8[x], s[56 + x]);
                float top = fmaxf(max3_f32(t8[0], t8[1], t8[2]), max3_f32(t8[3], t8[4], max3_f32(t8[5], t8[6], t8[7])));
                // Two S buffers: O up to the tile before, waited for at every step: S runs ahead of it, and a
                // warp two phases behind a barrier would take the older phase for the one it wants.
                // (One: this S was issued after the product that O waits for.)
                if (NS == 2 && j > 0 && !bwait(o_full + q, (uint32_t)((j - 1) & 1), error)) { ok = false; break; }
                if (NH == 2) {
                    // (that product has read P of both halves, so both have read the slots)
                    ex[half * kRows] = top;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(meet);
                    if (!bwait(meet, (uint32_t)(j & 1), error)) { ok = false; break; }
                    top = fmaxf(ex[0], ex[kRows]);
                }
                const bool moves = c * top > limit;
                if (__any_sync(0xffffffffu, moves)) {
                    float f = 1.f;
                    if (moves && !(limit == -INFINITY && top <= u_max)) {
                        const float m = __fmul_rn(c, top);
                        const bool far = fabsf(m) > kFar;
                        f = ex2(far ? c * (u_max - top) : __fmul_rn(c, u_max) - m);
                        u_max = top;
                        shift = far ? 0.f : m, limit = far ? -INFINITY : __fadd_rn(m, kSlack);
                    }
                    if (j > 0) {
                        // this half of O's columns (complete up to the tile before) to the new maximum
                        tc_fence_after();
                        l *= f;
#pragma unroll 1
                        for (int x = half * kPart; x < (half + 1) * kPart; x += 8) {
                            uint32_t o[8];
                            tmem_ld8(tO + x, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 8; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                            tmem_st8(tO + x, o);
                        }
                        tmem_st_wait();
                    }
                    if (moves && limit == -INFINITY) {
#pragma unroll
                        for (int x = 0; x < 64; ++x) s[x] -= u_max;
                    }
                    __syncwarp();
                }
                const uint64_t c2 = f32x2(c, c), m2 = f32x2(-shift, -shift);
                uint64_t z[2] = {0, 0};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t u[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        float e0, e1;
                        f32x2_split(fma_f32x2(f32x2(s[32 * x + 2 * y], s[32 * x + 2 * y + 1]), c2, m2), e0, e1);
                        e0 = ex2(e0), e1 = ex2(e1);
                        z[y & 1] = add_f32x2(z[y & 1], f32x2(e0, e1));
                        u[y] = pack2(e0, e1);
                    }
                    tmem_st16(tS + 16 * x, u);  // over columns that this warp has read
                }
                float za, zb;
                f32x2_split(add_f32x2(z[0], z[1]), za, zb);
                l += za + zb;
                tmem_st_wait();
                if (L < p.s && q == 0 && half == 0 && L - (t0 + j) * KT < KT) {
                    // the last tile's rows of V that do not count, once (the other tile's product comes later)
                    const int i = j + NS, st = i % ST, from = L - (t0 + j) * KT;
                    if (!bwait(full + st, (uint32_t)((i / ST) & 1), error)) { ok = false; break; }
                    const int warps = min((left + 31) / 32, 4);
                    for (int t = row; t < KT; t += 32 * warps) zero_rows<D>(sm + G::kRing + st * G::kStage + kTile<D, KT>, t, from, (from + 15) / 16 * 16);
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + buf);
            }
            if (ok && nt > 0) {
                // O, then the halves' sums (over the maxima, which all warps have read by then)
                ok = bwait(o_full + q, (uint32_t)((NS == 2 ? nt - 1 : 0) & 1), error);
                if (NH == 2) {
                    ex[half * kRows] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(meet);
                    ok = ok && bwait(meet, (uint32_t)(nt & 1), error);
                    l = ex[0] + ex[kRows];
                }
            }
            tc_fence_after();
        }
        const float m = __fmul_rn(c, u_max);
        if (active && q < nq && ok) {
            const long long f = cross_flat(p, b, kh, mine ? r : 0);
            const int to = min(p.d, (half + 1) * kPart);
            if (a.cluster) {
                // sums and (m, l) to this CTA's ring (the copies and products are done), for the cluster's join
                float *sO = reinterpret_cast<float *>(sm + G::kRing) + row * G::kJoinPitch;
                if (half == 0) reinterpret_cast<float2 *>(sm + G::kJoinMl)[row] = make_float2(nt > 0 ? m : -INFINITY, l);
                float o[32];
#pragma unroll 1
                for (int x = half * kPart; x < to; x += 32) {
                    if (nt > 0) {
                        tmem_ld32(tO + x, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] = 0.f;
                    }
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        *reinterpret_cast<float4 *>(sO + x + 4 * y) = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                }
            } else if (a.w.parts > 1) {
                const long long at = (long long)blockIdx.y * p.B * p.kv * p.rows + f;
                if (mine && half == 0) a.w.ml[at] = make_float2(nt > 0 ? m : -INFINITY, l);
                float o[32];
#pragma unroll 1
                for (int x = half * kPart; x < to; x += 32) {
                    if (nt > 0) {
                        tmem_ld32(tO + x, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] = 0.f;
                    }
                    if (!mine) continue;
                    float4 *dst = reinterpret_cast<float4 *>(a.w.o + at * p.d + x);
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        if (x + 4 * y < p.d) dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                }
            } else {
                // rows of H through this warp's rows and columns of the Q tile (all scores have been taken)
                const float inv = l == 0.f ? 0.f : 1.f / l;
                float o[32];
#pragma unroll 1
                for (int x = half * kPart; x < to; x += 32) {
                    if (nt > 0) {
                        tmem_ld32(tO + x, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] = 0.f;
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float *e = o + 8 * y;
                        *reinterpret_cast<uint4 *>(sQ + chunk_at(row, x / 8 + y)) =
                            make_uint4(pack2(e[0] * inv, e[1] * inv), pack2(e[2] * inv, e[3] * inv),
                                       pack2(e[4] * inv, e[5] * inv), pack2(e[6] * inv, e[7] * inv));
                    }
                }
                __syncwarp();
                each_row<kLanes>(mine ? cross_row(p, p.H, b, kh, r) : -1, p.H.sn, [&](int, int rr, long long to) {
                    if (to >= 0 && my_chunk * 8 < p.d)
                        *reinterpret_cast<uint4 *>((__nv_bfloat16 *)p.H.ptr + to + my_chunk * 8) =
                            *reinterpret_cast<const uint4 *>(sQ + chunk_at(w4 * 32 + rr, my_chunk));
                });
                if (p.lse && mine && half == 0) p.lse[f] = l == 0.f ? -INFINITY : m * (1.f / kLog2e) + logf(l);
            }
        }
        tc_fence_before();
        __syncwarp();
    }
    __syncthreads();
    if (warp == kIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kCols);
    }
    if constexpr (NQ == 1) {
        if (!a.cluster) return;
        // The parts of a cluster joined over distributed shared memory, in rank order: 8 columns of a row a
        // thread, the rows spread over the cluster's CTAs.  Every CTA gets here (its waits are bounded).
        cl::sync_all();
        const int parts = a.w.parts, per = p.d / 8, rows = min(left, kRows);
        const uint32_t sO = smem_u32(sm + G::kRing), sMl = smem_u32(sm + G::kJoinMl);
        for (int i = (int)blockIdx.y * G::kThreads + (int)threadIdx.x; i < rows * per; i += parts * G::kThreads) {
            const int row = i / per, c = i - row * per, r = r0 + row;
            float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < parts; ++q) m = fmaxf(m, cl::ld_f32(cl::map_shared(sMl + row * 8, q)));
            const float shift = m == -INFINITY ? 0.f : m;
            for (int q = 0; q < parts; ++q) {
                const uint32_t ml = cl::map_shared(sMl + row * 8, q), at = cl::map_shared(sO + (row * G::kJoinPitch + 8 * c) * 4, q);
                const float k = ex2(cl::ld_f32(ml) - shift);
                const float4 x = cl::ld_f4(at), y = cl::ld_f4(at + 16);
                l = fmaf(cl::ld_f32(ml + 4), k, l);
                o[0] = fmaf(x.x, k, o[0]), o[1] = fmaf(x.y, k, o[1]), o[2] = fmaf(x.z, k, o[2]), o[3] = fmaf(x.w, k, o[3]);
                o[4] = fmaf(y.x, k, o[4]), o[5] = fmaf(y.y, k, o[5]), o[6] = fmaf(y.z, k, o[6]), o[7] = fmaf(y.w, k, o[7]);
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            *reinterpret_cast<uint4 *>((__nv_bfloat16 *)p.H.ptr + cross_row(p, p.H, b, kh, r) + 8 * c) =
                make_uint4(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv), pack2(o[4] * inv, o[5] * inv), pack2(o[6] * inv, o[7] * inv));
            if (p.lse && c == 0) p.lse[cross_flat(p, b, kh, r)] = l == 0.f ? -INFINITY : m * (1.f / kLog2e) + logf(l);
        }
        cl::sync_all();  // no CTA leaves while another reads its sums
    }
}

// One key tile (s <= 128: a prompt's states): nothing to walk, so a CTA is short and what counts is
// that an SM has several of them, one loading while another computes.  128 threads, a row each, no
// warps of their own for loads and products; O lies over the half of S's columns that P leaves free
// (d <= 64), so that four CTAs share the 512 columns of an SM (d = 128: two).  S is read twice, for
// the maximum and for the exponentials, instead of being kept in 128 registers.  256 x 12 heads, 197
// queries over up to 77 states at d = 64: 57 us against 130 for the walk: bound by
// each CTA's own chain of loads, products and rows, four of which an SM overlaps (half of the issue slots).
template <int D>
struct Short {
    static constexpr int kQ = 0, kK = kTile<D>, kVv = 2 * kTile<D>, kBars = 3 * kTile<D>;
    static constexpr int kSmem = kBars + 4 * 8 + 16 + 1024;
    static constexpr int kPerSM = D == 64 ? 4 : 2;
    static constexpr uint32_t kColO = D == 64 ? 64 : 128, kCols = D == 64 ? 128 : 256;
    static_assert((kSmem + 1024) * kPerSM <= 228 * 1024 && kCols * kPerSM <= 512, "per SM");
};

template <int D>
__global__ void __launch_bounds__(kRows, Short<D>::kPerSM) cross_short_kernel(const __grid_constant__ FwdParams a) {
    using G = Short<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(sm + G::kBars), *v_full = k_full + 1, *s_full = v_full + 1, *o_full = s_full + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(o_full + 1);
    const CrossProblem &p = a.p;
    const int row = threadIdx.x, warp = row >> 5, lane = row & 31;
    const int bk = a.by_tiles.of((int)blockIdx.x), tile = (int)blockIdx.x - bk * a.tiles;
    const int b = p.by_kv.of(bk), kh = bk - b * p.kv, r = tile * kRows + row;
    const bool mine = r < p.rows, active = tile * kRows + 32 * warp < p.rows;
    unsigned int *error = &g_cross_fwd_error;
    if (row == 0) {
        mbar_init(k_full, 1);
        mbar_init(v_full, 1);
        mbar_init(s_full, 1);
        mbar_init(o_full, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(s_tmem, G::kCols);
    grid_dependency_wait();
    if (row == 0) {
        mbar_arrive_expect_tx(k_full, kTile<D>);
        load_tile<D, kRows, kRows>(sm + G::kK, a.k, k_full, 0, kh, b);
        mbar_arrive_expect_tx(v_full, kTile<D>);
        load_tile<D, kRows, kRows>(sm + G::kVv, a.v, v_full, 0, kh, b);
    }
    // Q, K and V of the CTA that will follow on this SM, into L2
    const long long then = (long long)blockIdx.x + G::kPerSM * kPlanSMs;
    if (then < (long long)gridDim.x) {
        const int bk2 = a.by_tiles.of((int)then), tile2 = (int)then - bk2 * a.tiles, b2 = p.by_kv.of(bk2), kh2 = bk2 - b2 * p.kv;
        if (tile2 * kRows + row < p.rows) {
            const char *q = (const char *)((const __nv_bfloat16 *)p.Q.ptr + cross_row(p, p.Q, b2, kh2, tile2 * kRows + row));
            for (int x = 0; x < 2 * p.d; x += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + x));
        }
        if (tile2 == 0 && row == 0) {
#pragma unroll
            for (int q = 0; q < D / 64; ++q) {
                prefetch_tile(&a.k.map, 64 * q, 0, kh2 * a.k.by_head, b2 * a.k.by_batch);
                prefetch_tile(&a.v.map, 64 * q, 0, kh2 * a.v.by_head, b2 * a.v.by_batch);
            }
        }
    }
    const int L = cross_length(p, b);
    uint8_t *sQ = sm + G::kQ;
    constexpr int kLanes = D / 8;
    {
        const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
        const int ch = lane % kLanes;
        uint4 x[kLanes];
        each_row<kLanes>(mine ? cross_row(p, p.Q, b, kh, r) : -1, p.Q.sn, [&](int i, int, long long o) {
            x[i] = make_uint4(0, 0, 0, 0);
            if (o >= 0 && ch * 8 < p.d) x[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)p.Q.ptr + o + ch * 8);
        });
#pragma unroll
        for (int i = 0; i < kLanes; ++i) {
            x[i].x ^= flip, x[i].y ^= flip, x[i].z ^= flip, x[i].w ^= flip;
            *reinterpret_cast<uint4 *>(sQ + chunk_at(warp * 32 + i * (32 / kLanes) + lane / kLanes, ch)) = x[i];
        }
        if (p.scale == 0.f)
            for (int i = 0; i < kLanes; ++i) times_zero(reinterpret_cast<uint4 *>(sQ + chunk_at(warp * 32 + i * (32 / kLanes) + lane / kLanes, ch)));
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (not before the tensor memory is held: the next kernel's would be taken first, and wait for this one)
    grid_dependents_launch();
    const uint32_t tmem = *s_tmem, mine_at = tmem + ((uint32_t)(warp * 32) << 16);
    const int l16 = (L + 15) / 16;
    bool ok = true;
    if (row == 0 && L > 0) {
        ok = bwait(k_full, 0u, error);
        tc_fence_after();
        if (ok)
            product_k<D>(tmem, desc_k(smem_u32(sQ)), desc_k(smem_u32(sm + G::kK)), idesc_bf16_f32(kRows, 16 * l16, false, false), (p.d + 15) / 16,
                         [] {});
        umma_commit(s_full);
    }
    __syncwarp();
    const float c = score_scale(p);
    float m = -INFINITY, l = 0.f;
    if (L > 0) {
        ok = bwait(s_full, 0u, error) && ok;
        tc_fence_after();
        if (ok && active) {
            float s[32];
#pragma unroll 1
            for (int x = 0; x < L; x += 32) {
                tmem_ld32(mine_at + x, s);
                tmem_ld_wait();
                float t4[4] = {m, -INFINITY, -INFINITY, -INFINITY};
                if (L - x < 32) {
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (x + y >= L) s[y] = -INFINITY;
                }
#pragma unroll
                for (int y = 0; y < 32; y += 8)
#pragma unroll
                    for (int z = 0; z < 4; ++z) t4[z] = max3_f32(t4[z], s[y + z], s[y + 4 + z]);
                m = fmaxf(max3_f32(t4[0], t4[1], t4[2]), t4[3]);
            }
            // (a row whose maximum is far: as above)
            const float u_max = m;
            m *= c;
            const bool far = fabsf(m) > kFar && m != -INFINITY;
            const float shift = far || m == -INFINITY ? 0.f : m;
            const int whole = __any_sync(0xffffffffu, far) ? 0 : L - 31;  // from here on scores need a look
            const uint64_t c2 = f32x2(c, c), m2 = f32x2(-shift, -shift);
            uint64_t z2[2] = {0, 0};
#pragma unroll 1
            for (int x = 0; x < L; x += 32) {
                tmem_ld32(mine_at + x, s);
                tmem_ld_wait();
                if (x >= whole) {
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (x + y >= L) s[y] = -INFINITY;
                    if (far) {
#pragma unroll
                        for (int y = 0; y < 32; ++y) s[y] -= u_max;
                    }
                    __syncwarp();
                }
                uint32_t u[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    float e0, e1;
                    f32x2_split(fma_f32x2(f32x2(s[2 * y], s[2 * y + 1]), c2, m2), e0, e1);
                    e0 = ex2(e0), e1 = ex2(e1);
                    z2[y & 1] = add_f32x2(z2[y & 1], f32x2(e0, e1));
                    u[y] = pack2(e0, e1);
                }
                tmem_st16(mine_at + x / 2, u);  // over columns that have been read
            }
            float za, zb;
            f32x2_split(add_f32x2(z2[0], z2[1]), za, zb);
            l = za + zb;
            tmem_st_wait();
        }
        if (L < p.s) {  // rows of V that do not count
            ok = bwait(v_full, 0u, error) && ok;
            zero_rows<D>(sm + G::kVv, row, L, 16 * l16);
            fence_proxy_async_smem();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (row == 0) {
        // (both copies have landed before the CTA leaves)
        const bool landed = bwait(v_full, 0u, error) && bwait(k_full, 0u, error);
        if (L > 0) {
            tc_fence_after();
            if (landed && ok)
                product_mn<64, kRows>(tmem + G::kColO, tmem, desc_mn(smem_u32(sm + G::kVv)), idesc_bf16_f32(kRows, p.d < D ? p.d : D, false, true), l16, false);
            umma_commit(o_full);
        }
    }
    __syncwarp();
    if (L > 0) {
        ok = bwait(o_full, 0u, error) && ok;
        tc_fence_after();
    }
    if (ok && active) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float o[32];
#pragma unroll 1
        for (int x = 0; x < p.d; x += 32) {
            if (L > 0) {
                tmem_ld32(mine_at + G::kColO + x, o);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = 0.f;
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float *e = o + 8 * y;
                *reinterpret_cast<uint4 *>(sQ + chunk_at(row, x / 8 + y)) =
                    make_uint4(pack2(e[0] * inv, e[1] * inv), pack2(e[2] * inv, e[3] * inv), pack2(e[4] * inv, e[5] * inv),
                               pack2(e[6] * inv, e[7] * inv));
            }
        }
        __syncwarp();
        const int ch = lane % kLanes;
        each_row<kLanes>(mine ? cross_row(p, p.H, b, kh, r) : -1, p.H.sn, [&](int, int rr, long long to) {
            if (to >= 0 && ch * 8 < p.d)
                *reinterpret_cast<uint4 *>((__nv_bfloat16 *)p.H.ptr + to + ch * 8) =
                    *reinterpret_cast<const uint4 *>(sQ + chunk_at(warp * 32 + rr, ch));
        });
        if (p.lse && mine) p.lse[cross_flat(p, b, kh, r)] = l == 0.f ? -INFINITY : m * (1.f / kLog2e) + logf(l);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kCols);
    }
}

bool is_short(const CrossProblem &p) { return p.s <= kRows; }

// Two tiles a CTA where rows fill them; one for up to 128 rows.
int tiles_per_cta(const CrossProblem &p) { return p.rows > kRows ? 2 : 1; }

template <int D, int NQ, int KT>
cudaError_t launch(const CrossProblem &p, const CrossParts &w, cudaStream_t stream) {
    using G = Geo<D, NQ, KT>;
    FwdParams a;
    a.p = p;
    a.w = w;
    a.tiles = (p.rows + NQ * kRows - 1) / (NQ * kRows);
    a.by_tiles = Divide((uint32_t)a.tiles);
    if (p.s > 0 && (!make_tile_map(&a.k, p.K, p.B, p.kv, p.s, p.d, KT) || !make_tile_map(&a.v, p.V, p.B, p.kv, p.s, p.d, KT)))
        return cudaErrorInvalidValue;
    static SmemOnce allow;
    const cudaError_t e = allow(cross_fwd_kernel<D, NQ, KT>, G::kSmem);
    if (e != cudaSuccess) return e;
    a.cluster = NQ == 1 && w.parts > 1 && !w.o;
    if (a.cluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(a.tiles * p.B * p.kv, w.parts);
        cfg.blockDim = dim3(G::kThreads);
        cfg.dynamicSmemBytes = G::kSmem;
        cfg.stream = stream;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = 1, at[1].val.clusterDim.y = (unsigned)w.parts, at[1].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, cross_fwd_kernel<D, NQ, KT>, a);
    }
    return launch_pdl(cross_fwd_kernel<D, NQ, KT>, dim3(a.tiles * p.B * p.kv, w.parts), dim3(G::kThreads), G::kSmem, stream, a);
}

template <int D>
cudaError_t launch_short(const CrossProblem &p, cudaStream_t stream) {
    FwdParams a;
    a.p = p;
    a.w = CrossParts{nullptr, nullptr, 1};
    a.tiles = (p.rows + kRows - 1) / kRows;
    a.by_tiles = Divide((uint32_t)a.tiles);
    if (!make_tile_map(&a.k, p.K, p.B, p.kv, p.s, p.d, kRows) || !make_tile_map(&a.v, p.V, p.B, p.kv, p.s, p.d, kRows))
        return cudaErrorInvalidValue;
    static SmemOnce allow;
    const cudaError_t e = allow(cross_short_kernel<D>, Short<D>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_short_kernel<D>, dim3(a.tiles * p.B * p.kv), dim3(kRows), Short<D>::kSmem, stream, a);
}

}  // namespace

namespace cross_tc {

bool make_tile_map(TileMap *m, const CrossView &v, int B, int heads, int rows, int d, int box_rows) {
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (Encode)f;
    }();
    if (!encode) return false;
    m->by_head = heads > 1 && v.sh > 0;
    m->by_batch = B > 1 && v.sb > 0;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)rows, m->by_head ? (cuuint64_t)heads : 1, m->by_batch ? (cuuint64_t)B : 1};
    // the stride of an axis of one entry is not used, but has to be one
    const cuuint64_t strides[3] = {(cuuint64_t)(rows > 1 ? v.sn : d) * 2, (cuuint64_t)(m->by_head ? v.sh : d) * 2,
                                   (cuuint64_t)(m->by_batch ? v.sb : d) * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, one[4] = {1, 1, 1, 1};
    return encode(&m->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(v.ptr), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace cross_tc

// Parts of the key axis: none while the row tiles alone fill the SMs; else so many that they do.  Up to
// kCluster of them are the CTAs of a cluster, which joins them itself: a token of 12 heads over 1500
// states takes one launch and no workspace.  More (a second launch joins them) where each of the
// cluster's would have more than kClusterTiles tiles.
// One tile of rows, CTAs enough for the SMs but long: parts of kLong tiles and more, a cluster's, where the last
// wave would be long and thin: entries of lengths of their own, for a few waves, or, longer still, hardly more CTAs
// than places (64 x 8 key heads, up to 8192 states, d = 128: 215 -> 204 us; 24 x 8, up to 16384: 193 -> 155; 20 x 8,
// 65536 each: 1089 -> 773; 20 x 8, 32768 each, d = 64: 348 -> 239; but 200 x 12, up to 8200, d = 64: 523 -> 544; 32 x
// 8, 8192 each, d = 128: 153 -> 169; 14 x 8: 69 -> 82).  The join takes about 5 us of each of a cluster's CTAs: 128 x 8, up
// to 2048: 110 -> 149.
constexpr int kCluster = 8, kClusterTiles = 8, kLong = 32;
CrossPlan cross_tc_plan(const CrossProblem &p) {
    if (is_short(p)) return CrossPlan{1, false};
    const int nq = tiles_per_cta(p), per_sm = p.d <= 64 ? 2 : 1;
    const long long ctas = (long long)p.B * p.kv * ((p.rows + nq * kRows - 1) / (nq * kRows)), places = (long long)per_sm * kPlanSMs;
    const long long want = places / std::max(1LL, ctas), tiles = (p.s + kRows - 1) / kRows;
    if (nq == 1 && want > 1 && (want <= kCluster || tiles <= kCluster * kClusterTiles))
        return CrossPlan{(int)std::min(std::min(want, (long long)kCluster), tiles), false};
    if (nq == 1 && want <= 1 && (p.lengths ? tiles >= 2 * kLong && ctas < 6 * places : tiles >= 4 * kLong && 3 * ctas < 4 * places))
        return CrossPlan{(int)std::min(tiles / kLong, (long long)kCluster), false};
    const int parts = (int)std::max(1LL, std::min(want, (tiles + 1) / 2));
    return CrossPlan{parts, parts > 1};
}

cudaError_t launch_cross_tc_forward(const CrossProblem &p, const CrossParts &w, cudaStream_t stream) {
    const int nq = tiles_per_cta(p);
    if (is_short(p) && p.s > 0) return p.d > 64 ? launch_short<128>(p, stream) : launch_short<64>(p, stream);
    if (p.d > 64) return nq == 2 ? launch<128, 2, 128>(p, w, stream) : launch<128, 1, 128>(p, w, stream);
    return nq == 2 ? launch<64, 2, 64>(p, w, stream) : launch<64, 1, 128>(p, w, stream);
}

cudaError_t cross_fwd_read_and_clear_error(unsigned *out) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_cross_fwd_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_cross_fwd_error, &zero, sizeof(unsigned));
}

}  // namespace anchor
