// Cross attention backward in bf16 on the tensor cores (formulas in include/anchor_attn.h):
//   P = 2^(c S - lse), S = Q K^T;  dS = P o (dH V^T - D), D = dH . H;
//   dQ = scale dS K;  dV = P^T dH;  dK = scale dS^T Q.
//
// Two kinds of CTAs, one that keeps queries and one that keeps keys, so that every gradient is summed in
// tensor memory by one CTA in a fixed order, without atomics.  S and dP are made twice for
// that: seven products where five would do.  Both are of one launch, those that take longer first, so that
// the others fill the SMs that they leave (D comes from a launch before, but see kFine; with the queries
// first and D made by them, in a launch of their own, 2 x 16 heads over 4, 2049 x 1500, d = 128: 188 us
// against 152).  CTAs that walk long are cut into parts (see Parts).
//
//   queries   a tile of 128 rows of Q and dH stays, the keys of the entry stream by:
//             S = Q K^T, dP = dH V^T, dQ += dS K
//   keys      a tile of 128 rows of K and V stays, the queries of all heads that share it
//             stream by: S^T = K Q^T, dP^T = V dH^T, dV += P^T dH, dK += dS^T Q
//
// Streaming tiles of W = 128 rows at d = 128, where S, dP, dV and dK fill tensor memory; of 64 below,
// which leaves room for two CTAs an SM (one fetches its rows while the other computes).  Row warps
// take 32 columns of S and dP each, a row a thread: warp w has lanes 32 (w % 4) .. + 31 of tensor memory
// and columns 32 (w / 4) .. + 31.  P^T and dS go back to tensor memory as bf16 operands, each warp's
// over columns that it has read itself.  The products are issued so that the tensor cores have
// work while the rows are between two of their steps:
//   keys      after P^T(j): dV += P^T(j) dH, S^T(j + 1)      while the rows make dS^T(j)
//             after dS^T(j): dK += dS^T(j) Q, dP^T(j + 1)    while the rows make P^T(j + 1)
//   queries   after S(j) is read: S(j + 1);  after dS(j): dQ += dS(j) K, dP(j + 1)
// (a product that overwrites an operand is issued after the one that reads it).  P and dS are rounded to
// bf16, the operands' type (dS to two of them at times, see kFine); S, dP, P in dS, and all sums are fp32.
// States from the length on: P and dS are zero there by select, and rows of K that meet a zero of dS
// are zeroed in shared memory.
#include "cross_tc.cuh"

#include <algorithm>

#include <math.h>

#include <type_traits>

namespace anchor {

__device__ unsigned int g_cross_bwd_error;  // bit 0: a wait gave up

namespace {

using namespace cross_tc;

constexpr int kSlice = 32;  // columns of S and dP that a row warp takes

// Up to kFine states dS meets K and Q as two bf16 numbers, the second what the rounding of the first left: an
// eighth product and a ninth.  dQ and dK carry the rounding of dS, their own, and that of H through D, which
// is 2^-9 of dP over the root of the number of states that weigh: with few of them the three together are
// up to 1.8 times a lone rounding of the result (8 states; 1.56 at 50, 1.50 at 256), and with two numbers 1.46,
// 1.19, 1.07.  It takes 6 % of time at 77 states, 10 at 300, 18 at 600, 25 at 1000 and more.
// One tile of states: the queries' CTAs make D from P and dP instead (1.00 at 8 and 50), and the keys' CTAs follow in
// a launch of their own (256 x 12 heads, 49 x 49: 130 us against 133 with D from H).
// More than kFine, d <= 64: for dQ in some of the key tiles, so that no gradient is much further off than a rounding of its
// own and one of dS, which is where dK (1.41 to 1.45) and d = 128 (1.45 to 1.48) are anyway.  dQ at d = 64 and 32, 390 to
// 8000 states: 1.47 to 1.52 with none, 1.37 to 1.42 with every fourth tile, 1.04 to 1.09 with all; at d = 16 1.66 with
// none, 1.58 with every fourth, 1.17 with all: there every second, 1.46.  The backward of 8 x 12 heads, 4200 x 1000, d = 64:
// 454 us with none, 470 with every fourth, 498 with all.  Which tiles is a matter of their place among the entry's states alone.
constexpr int kFine = 384;
__device__ __forceinline__ int fine_tiles(int d) { return d > 16 ? 4 : 2; }

// D columns (heads of 16 and 32 are 64), streaming tiles of W rows.
template <int D, int W>
struct Geo {
    static constexpr int kSlices = W / kSlice, kRowWarps = 4 * kSlices;
    static constexpr int kLoad = kRowWarps, kStat = kRowWarps + 1, kIssue = kRowWarps + 2, kThreads = 32 * (kRowWarps + 3);
    static constexpr int kPerSM = D == 64 ? 2 : 1;
    // Slots of the two tiles that stream by (Q or K, dH or V).  The first of step j is in use from the
    // middle of step j - 1 to the end of step j, the second from the end of step j - 1: with one slot
    // more for the first, both are loaded a step and more ahead.
    static constexpr int kNB = D == 128 ? 2 : 4, kNA = kNB + 1;
    static constexpr int kSlot = kTile<D, W>;
    static constexpr int kFix = 0, kA = 2 * kTile<D>, kB = kA + kNA * kSlot;
    static constexpr int kStatB = kB + kNB * kSlot;  // keys: lse, D of W columns
    static constexpr int kBars = kStatB + 2 * W * 4;
    static constexpr int kNBars = kNA + 2 * kNB + 15;
    static constexpr int kSmem = kBars + kNBars * 8 + 16 + 1024;
    static constexpr uint32_t kColS = 0, kColP = W, kColA = 2 * W;  // S, dP, then the sums
    static constexpr uint32_t kCols = 2 * W + 2 * D;                // of tensor memory
    static_assert((kSmem + 1024) * kPerSM <= 228 * 1024, "shared memory");
    static_assert(kCols * kPerSM <= 512 && (kCols == 256 || kCols == 512), "tensor memory");
};

struct BwdParams {
    CrossProblem p;
    float *delta;        // D
    TileMap q, g, k, v;  // g: dH
    int tiles[2];        // of the queries and of the keys of a key head
    Divide by_tiles[2];
    int parts[2];        // of the steps of a tile
    Divide by_parts[2];
    float *sums[2];      // with parts: [part][B * kv * rows of the kind][d] (queries), [2 d] (keys: dV, dK)
    int first;           // CTAs of the kind that comes first
    bool keys_first;
    bool exact;          // one tile of states: the queries' CTAs make D themselves
};

// The work of CTA `index` of its kind (KEYS: see above).  FINE: dS as two numbers.  CUT:
// steps in parts (a kernel of its own: 5 % more time for all where the numbers of parts are read).
template <int D, bool KEYS, int W, bool FINE, bool CUT>
__device__ __forceinline__ void cross_bwd(const BwdParams &a, int index) {
    using G = Geo<D, W>;
    constexpr int kRowWarps = G::kRowWarps, kLoad = G::kLoad, kStat = G::kStat, kIssue = G::kIssue;
    constexpr uint32_t kColS = G::kColS, kColP = G::kColP, kColA = G::kColA;
    constexpr int NA = G::kNA, NB = G::kNB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G::kBars);
    uint64_t *a_full = bars /* [NA] */, *b_full = a_full + NA /* [NB] */, *empty = b_full + NB /* [NB] */, *fix_full = empty + NB,
             *s_full = fix_full + 1, *dp_full = s_full + 1, *p_full = dp_full + 1, *ds_full = p_full + 1, *lse_full = ds_full + 1,
             *lse_empty = lse_full + 1, *d_full = lse_empty + 1, *d_empty = d_full + 1, *acc = d_empty + 1, *done = acc + 1,
             *meet = done + 1 /* [4] */;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + G::kNBars);
    float *stat = reinterpret_cast<float *>(sm + G::kStatB);
    const CrossProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = CUT ? a.parts[KEYS] : 1, item = CUT ? a.by_parts[KEYS].of(index) : index, part = CUT ? index - item * parts : 0;
    const int bk = a.by_tiles[KEYS].of(item), tile = item - bk * a.tiles[KEYS];
    const TileMap &map_a = KEYS ? a.q : a.k, &map_b = KEYS ? a.g : a.v;  // the tiles that stream by
    const int b = p.by_kv.of(bk), kh = bk - b * p.kv, r0 = tile * kRows;
    unsigned int *error = &g_cross_bwd_error;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NA; ++s) mbar_init(a_full + s, 1);
        for (int s = 0; s < NB; ++s) {
            mbar_init(b_full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(fix_full, KEYS ? 1 : kRowWarps);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, kRowWarps);
        mbar_init(ds_full, kRowWarps);
        mbar_init(lse_full, 1);
        mbar_init(lse_empty, kRowWarps);
        mbar_init(d_full, 1);
        mbar_init(d_empty, kRowWarps);
        mbar_init(acc, 1);
        mbar_init(done, 1);
        for (int s = 0; s < 4; ++s) mbar_init(meet + s, G::kSlices);
        fence_mbar_init();
    }
    if (warp == kIssue) tmem_alloc(s_tmem, G::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dependency_wait();
    grid_dependents_launch();

    const int L = cross_length(p, b);
    // steps over the tiles that stream by: keys of the entry, or the queries of each head in turn
    const int per_head = (p.n + W - 1) / W;
    const int steps = KEYS ? (r0 < L ? p.group * per_head : 0) : (L + W - 1) / W;
    const int j0 = CUT ? (int)((long long)steps * part / parts) : 0;
    const int nt = CUT ? (int)((long long)steps * (part + 1) / parts) - j0 : steps;
    // A walk over the steps: tile t of head g (without divisions, which the issuing thread would wait
    // for).
    struct Walk {
        int t, g, per_head, group;
        __device__ __forceinline__ void next() {
            if (++t == per_head) {
                t = 0;
                if (++g == group) g = 0;
            }
        }
    };
    const int around = KEYS ? per_head : steps, g0 = CUT && KEYS && part > 0 ? j0 / per_head : 0;
    const Walk start{j0 - g0 * per_head, g0, around, KEYS ? p.group : 1};
    const int some = fine_tiles(p.d) - 1;
    auto two = [=](int j) { return FINE || (D == 64 && !KEYS && ((j0 + j) & some) == 0); };  // dS of step j is two numbers
    // columns of a tile that exist
    auto width = [&](int t) { return min(W, (KEYS ? p.n : L) - t * W); };

    if (warp == kLoad) {
        if (lane == 0 && nt > 0) {
            if (KEYS) {
                mbar_arrive_expect_tx(fix_full, 2 * kTile<D>);
                load_tile<D, kRows, W>(sm + G::kFix, a.k, fix_full, r0, kh, b);
                load_tile<D, kRows, W>(sm + G::kFix + kTile<D>, a.v, fix_full, r0, kh, b);
            }
            int ja = 0, jb = 0;  // steps whose tiles have been asked for
            Walk wa = start, wb = start;
            auto load_a = [&]() {
                if (ja >= nt) return;
                mbar_arrive_expect_tx(a_full + ja % NA, G::kSlot);
                load_tile<D, W, W>(sm + G::kA + ja % NA * G::kSlot, map_a, a_full + ja % NA, wa.t * W, KEYS ? kh * p.group + wa.g : kh, b);
                ++ja;
                wa.next();
            };
            auto load_b = [&]() {
                if (jb >= nt) return;
                mbar_arrive_expect_tx(b_full + jb % NB, G::kSlot);
                load_tile<D, W, W>(sm + G::kB + jb % NB * G::kSlot, map_b, b_full + jb % NB, wb.t * W, KEYS ? kh * p.group + wb.g : kh, b);
                ++jb;
                wb.next();
            };
            for (int j = 0; j < NB; ++j) {
                load_a();
                load_b();
            }
            load_a();
            int i = 0;  // steps that are done
            for (; i < nt - NB; ++i) {
                if (!bwait(empty + i % NB, (uint32_t)((i / NB) & 1), error)) break;
                load_b();
                load_a();
            }
            // the CTA leaves only once its copies have landed
            for (int j = max(0, ja - NA); j < ja; ++j) bwait(a_full + j % NA, (uint32_t)((j / NA) & 1), error);
            for (int j = max(0, jb - NB); j < jb; ++j) bwait(b_full + j % NB, (uint32_t)((j / NB) & 1), error);
            if (KEYS) bwait(fix_full, 0u, error);
        }
        __syncwarp();
        // What the CTA that will follow on this SM begins with, into L2: where CTAs are short (few states; 64 x 8
        // heads, 197 x 300, d = 128: 182 -> 174 us; with many it takes 1 % more).
        if constexpr (FINE) {
            const int then = index + G::kPerSM * kPlanSMs;
            if (parts == 1 && then < a.tiles[KEYS] * p.B * p.kv) {
                const int bk2 = a.by_tiles[KEYS].of(then), tile2 = then - bk2 * a.tiles[KEYS], b2 = p.by_kv.of(bk2), kh2 = bk2 - b2 * p.kv;
                if (lane < 2) {
                    const TileMap &stay = lane ? a.v : a.k, &by = lane ? map_b : map_a;
                    const int head = KEYS ? kh2 * p.group : kh2;
#pragma unroll
                    for (int q = 0; q < D / 64; ++q) {
                        if (KEYS)
                            for (int t = 0; t < kRows; t += W) prefetch_tile(&stay.map, 64 * q, tile2 * kRows + t, kh2 * stay.by_head, b2 * stay.by_batch);
                        if (tile2 == 0)
                            for (int t = 0; t < min(NB * W, KEYS ? p.n : p.s); t += W) prefetch_tile(&by.map, 64 * q, t, head * by.by_head, b2 * by.by_batch);
                    }
                }
                if (!KEYS) {
                    for (int x = tile2 * kRows + lane; x < min(p.rows, (tile2 + 1) * kRows); x += 32) {
                        const char *q = (const char *)((const __nv_bfloat16 *)p.Q.ptr + cross_row(p, p.Q, b2, kh2, x));
                        const char *g = (const char *)((const __nv_bfloat16 *)p.dH.ptr + cross_row(p, p.dH, b2, kh2, x));
                        for (int y = 0; y < 2 * p.d; y += 128) {
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + y));
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(g + y));
                        }
                    }
                }
            }
        }
    } else if (warp == kStat) {
        if (KEYS) {
            // - lse (in log2) and - D of each step's columns, read a step ahead; columns that do not exist: P = 0
            constexpr int kX = W / 32;
            float next[2 * kX];
            Walk w = start;
            auto fetch = [&]() {
                const int i0 = w.t * W;
                const long long f = ((long long)b * p.heads + kh * p.group + w.g) * p.n + i0;
#pragma unroll
                for (int x = 0; x < kX; ++x) {
                    const bool in = i0 + 32 * x + lane < p.n;
                    next[x] = in ? -far_lse(p.lse[f + 32 * x + lane] * kLog2e) : -INFINITY;
                    next[kX + x] = in ? -a.delta[f + 32 * x + lane] : 0.f;
                }
                w.next();
            };
            bool ok = true;
            if (nt > 0) fetch();
            for (int j = 0; j < nt && ok; ++j) {
                if (j > 0 && !(ok = bwait(lse_empty, (uint32_t)((j - 1) & 1), error))) break;
#pragma unroll
                for (int x = 0; x < kX; ++x) stat[32 * x + lane] = next[x];
                __syncwarp();
                if (lane == 0) mbar_arrive(lse_full);
                if (j > 0 && !(ok = bwait(d_empty, (uint32_t)((j - 1) & 1), error))) break;
#pragma unroll
                for (int x = 0; x < kX; ++x) stat[W + 32 * x + lane] = next[kX + x];
                __syncwarp();
                if (lane == 0) mbar_arrive(d_full);
                if (j + 1 < nt) fetch();
            }
        }
        __syncwarp();
    } else if (warp == kIssue) {
        if (lane == 0 && nt > 0) {
            const int ksteps = (p.d + 15) / 16;
            const uint32_t base = smem_u32(sm);
            const uint32_t idA = idesc_bf16_f32(kRows, p.d < D ? p.d : D, false, true);
            const uint64_t f0 = desc_k(base + G::kFix), f1 = desc_k(base + G::kFix + kTile<D>);
            // (a commit takes this thread 70 cycles, a wait on a complete barrier 130: one barrier frees both
            // tiles of a step, and that the next products' tiles have landed is looked at while these run)
            auto slot_a = [&](int j) { return base + G::kA + j % NA * G::kSlot; };
            auto slot_b = [&](int j) { return base + G::kB + j % NB * G::kSlot; };
            uint64_t *const a_bar = a_full, *const b_bar = b_full;
            auto a_par = [](int j) { return (uint32_t)((j / NA) & 1); };
            auto b_par = [](int j) { return (uint32_t)((j / NB) & 1); };
            // columns of the walk's tiles in 16s: all but a head's (an entry's) last are full
            const int last16 = (width(around - 1) + 15) / 16;
            const uint32_t idF = idesc_bf16_f32(kRows, W, false, false), idL = idesc_bf16_f32(kRows, 16 * last16, false, false);
            // sum += (operand in tensor memory) x (a tile that streams by)
            auto along = [&](uint32_t sum, uint32_t op, uint32_t tile, bool last, bool add) {
                product_mn<kSlice / 2, W>(sum, op, desc_mn(tile), idA, last ? last16 : W / 16, add);
            };
            Walk w = start;
            bool last = w.t == around - 1;
            auto nothing = [] {};
            bool ok = bwait(fix_full, 0u, error) && bwait(a_bar, 0u, error) && bwait(b_bar, 0u, error);
            tc_fence_after();
            if (ok) {
                product_k<D>(tmem + kColS, f0, desc_k(slot_a(0)), last ? idL : idF, ksteps, nothing);
                umma_commit(s_full);
                product_k<D>(tmem + kColP, f1, desc_k(slot_b(0)), last ? idL : idF, ksteps, nothing);
                umma_commit(dp_full);
            }
            bool landed_a = false, landed_b = false;  // the next products' tiles, as seen during these
            for (int j = 0; j < nt && ok; ++j) {
                const bool more = j + 1 < nt;
                const uint32_t par = (uint32_t)(j & 1);
                w.next();
                const bool then = w.t == around - 1;  // the next step's
                // the rows have read S(j) (and left P^T(j) over it)
                if (more && !landed_a && !(ok = bwait(a_bar + (j + 1) % NA, a_par(j + 1), error))) break;
                if (!(ok = bwait(p_full, par, error))) break;
                tc_fence_after();
                if (KEYS) along(tmem + kColA, tmem + kColS, slot_b(j), last, j > 0);  // dV += P^T dH
                if (more) {
                    product_k<D>(tmem + kColS, f0, desc_k(slot_a(j + 1)), then ? idL : idF, ksteps,
                                 [&] { landed_b = mbar_test(b_bar + (j + 1) % NB, b_par(j + 1)); });
                    umma_commit(s_full);
                }
                // the rows have left dS(j) over dP(j)
                if (more && !landed_b && !(ok = bwait(b_bar + (j + 1) % NB, b_par(j + 1), error))) break;
                if (!(ok = bwait(ds_full, par, error))) break;
                tc_fence_after();
                const uint32_t sum = tmem + kColA + (KEYS ? D : 0);
                along(sum, tmem + kColP, slot_a(j), last, j > 0);  // dK += dS^T Q, dQ += dS K
                if (two(j)) along(sum, tmem + kColP + kSlice / 2, slot_a(j), last, true);
                if (more) {
                    product_k<D>(tmem + kColP, f1, desc_k(slot_b(j + 1)), then ? idL : idF, ksteps,
                                 [&] { landed_a = mbar_test(a_bar + (j + 2) % NA, a_par(j + 2)); });
                    umma_commit(dp_full);
                }
                umma_commit(empty + j % NB);
                last = then;
            }
            if (ok) umma_commit(acc);
            umma_commit(done);
            bwait(done, 0u, error);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ rows
        const int quarter = warp >> 2, w4 = warp & 3, row = w4 * 32 + lane, r = r0 + row;
        const bool mine = r < (KEYS ? L : p.rows);  // a row that counts
        const uint32_t trow = tmem + ((uint32_t)(w4 * 32) << 16);
        const uint64_t c = f32x2(p.scale * kLog2e, p.scale * kLog2e);
        uint64_t lse2 = f32x2(-INFINITY, -INFINITY), dl = 0;  // - lse (in log2) and - D of this row, twice
        if (!KEYS && nt > 0) {
            // the first half of the warps load the 128 rows of Q, each its part of the columns, the others those of dH
            constexpr int kParts = G::kSlices / 2, kLanes = D / (8 * kParts);
            const bool second = quarter >= kParts;
            const int ch = quarter % kParts * kLanes + lane % kLanes;
            const CrossView &v = second ? p.dH : p.Q;
            uint8_t *dst = sm + G::kFix + (second ? kTile<D> : 0);
            uint4 x[kLanes];
            each_row<kLanes>(mine ? cross_row(p, v, b, kh, r) : -1, v.sn, [&](int i, int, long long o) {
                x[i] = make_uint4(0, 0, 0, 0);
                if (o >= 0 && ch * 8 < p.d) x[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)v.ptr + o + ch * 8);
            });
#pragma unroll
            for (int i = 0; i < kLanes; ++i)
                *reinterpret_cast<uint4 *>(dst + chunk_at(w4 * 32 + i * (32 / kLanes) + lane / kLanes, ch)) = x[i];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(fix_full);
            if (mine) {
                const long long f = cross_flat(p, b, kh, r);
                const float x2 = -far_lse(p.lse[f] * kLog2e);
                lse2 = f32x2(x2, x2);
                if (!FINE || !a.exact) {
                    const float d2 = -a.delta[f];
                    dl = f32x2(d2, d2);
                }
            }
        }
        const uint32_t tS = trow + kColS + kSlice * quarter, tP = trow + kColP + kSlice * quarter;
        bool ok = true;
        Walk walk = start;
        for (int j = 0; j < nt && ok; ++j, walk.next()) {
            const int cols = width(walk.t) - kSlice * quarter;  // of this quarter that exist (may be none)
            const float *st = stat + kSlice * quarter;
            float e[32];
            if (!bwait(s_full, (uint32_t)(j & 1), error)) { ok = false; break; }
            if (KEYS && !bwait(lse_full, (uint32_t)(j & 1), error)) { ok = false; break; }
            tc_fence_after();
            tmem_ld32(tS, e);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
                ulonglong2 s4 = make_ulonglong2(lse2, lse2);
                if (KEYS) s4 = *reinterpret_cast<const ulonglong2 *>(st + x);
                f32x2_split(fma_f32x2(f32x2(e[x], e[x + 1]), c, s4.x), e[x], e[x + 1]);
                f32x2_split(fma_f32x2(f32x2(e[x + 2], e[x + 3]), c, s4.y), e[x + 2], e[x + 3]);
#pragma unroll
                for (int y = 0; y < 4; ++y) e[x + y] = ex2(e[x + y]);
            }
            const bool cut = !mine || (!KEYS && cols < kSlice);
            if (cut) {
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (!mine || x >= cols) e[x] = 0.f;
            }
            if (KEYS) {
                uint32_t u[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) u[x] = pack2(e[2 * x], e[2 * x + 1]);
                tmem_st16(tS, u);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (KEYS) mbar_arrive(lse_empty);
                mbar_arrive(p_full);
            }
            // dS
            if (KEYS && !bwait(d_full, (uint32_t)(j & 1), error)) { ok = false; break; }
            if (!bwait(dp_full, (uint32_t)(j & 1), error)) { ok = false; break; }
            tc_fence_after();
            {
                float g[32];
                uint32_t u[16];
                tmem_ld32(tP, g);
                tmem_ld_wait();
                if constexpr (FINE && !KEYS) {
                    if (a.exact) {  // D = sum_j P dP, over this warp's columns, then over the slices (a slot that one step leaves free)
                        float sum = 0.f;
#pragma unroll
                        for (int y = 0; y < 32; ++y) sum += cut && (!mine || y >= cols) ? 0.f : e[y] * g[y];
                        float *parts = reinterpret_cast<float *>(sm + G::kA + G::kSlot) + row;
                        parts[quarter * kRows] = sum;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(meet + w4);
                        if (!bwait(meet + w4, 0u, error)) { ok = false; break; }
                        sum = 0.f;
#pragma unroll
                        for (int x = 0; x < G::kSlices; ++x) sum += parts[x * kRows];
                        if (mine && quarter == 0) a.delta[cross_flat(p, b, kh, r)] = sum;
                        dl = f32x2(-sum, -sum);
                    }
                }
#pragma unroll
                for (int y = 0; y < 32; y += 4) {
                    ulonglong2 d4 = make_ulonglong2(dl, dl);
                    if (KEYS) d4 = *reinterpret_cast<const ulonglong2 *>(st + W + y);
                    f32x2_split(mul_f32x2(f32x2(e[y], e[y + 1]), add_f32x2(f32x2(g[y], g[y + 1]), d4.x)), g[y], g[y + 1]);
                    f32x2_split(mul_f32x2(f32x2(e[y + 2], e[y + 3]), add_f32x2(f32x2(g[y + 2], g[y + 3]), d4.y)), g[y + 2], g[y + 3]);
                }
                if (cut) {  // (a masked state's dP may be anything: zero by select, not by the product)
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (!mine || y >= cols) g[y] = 0.f;
                }
#pragma unroll
                for (int y = 0; y < 16; ++y) u[y] = pack2(g[2 * y], g[2 * y + 1]);
                tmem_st16(tP, u);
                if (two(j)) {  // what the rounding left, over the slice's other columns
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        u[y] = pack2(g[2 * y] - __uint_as_float(u[y] << 16), g[2 * y + 1] - __uint_as_float(u[y] & 0xffff0000u));
                    tmem_st16(tP + kSlice / 2, u);
                }
            }
            tmem_st_wait();
            if (!KEYS && walk.t == steps - 1 && quarter == 0 && L % W && L < p.s) {
                // the last tile's rows of K that do not count (S has read them)
                if (!bwait(a_full + j % NA, (uint32_t)((j / NA) & 1), error)) { ok = false; break; }
                zero_rows<D>(sm + G::kA + j % NA * G::kSlot, row, L % W, (L % W + 15) / 16 * 16);
                fence_proxy_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (KEYS) mbar_arrive(d_empty);
                mbar_arrive(ds_full);
            }
        }
        if (ok && nt > 0) ok = bwait(acc, 0u, error);
        tc_fence_after();
        // Rows out through shared memory (the tiles that stayed are not needed any more).  Keys: the first
        // half of the warps dV, the others dK, each its part of the columns; queries: all of them dQ.
        constexpr int kParts = KEYS ? G::kSlices / 2 : G::kSlices, kCols = D / kParts;  // of a warp
        const bool second = KEYS && quarter >= kParts;
        const float by = KEYS && !second ? 1.f : p.scale;
        uint8_t *stage = sm + G::kFix + (second ? kTile<D> : 0);
        const int from = quarter % kParts * kCols, to = min(p.d, from + kCols);
        if (ok && from < p.d) {
#pragma unroll 1
            for (int x = from; x < to; x += 32) {
                float o[32];
                if (nt > 0) {
                    tmem_ld32(trow + kColA + (second ? D : 0) + x, o);
                    tmem_ld_wait();
                }
                const bool some = nt > 0 && mine;
                if (CUT && parts > 1) {  // (cross_sums_kernel scales and rounds)
                    const int rows = KEYS ? p.s : p.rows, width = KEYS ? 2 * p.d : p.d;
                    float *dst = a.sums[KEYS] + (((long long)part * p.B * p.kv + bk) * rows + r) * width + (second ? p.d : 0) + x;
#pragma unroll
                    for (int y = 0; y < 32; y += 4)
                        if (r < rows && x + y < p.d)
                            *reinterpret_cast<float4 *>(dst + y) =
                                some ? make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                    continue;
                }
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = some ? o[y] * by : 0.f;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float *q = o + 8 * y;
                    *reinterpret_cast<uint4 *>(stage + chunk_at(row, x / 8 + y)) =
                        make_uint4(pack2(q[0], q[1]), pack2(q[2], q[3]), pack2(q[4], q[5]), pack2(q[6], q[7]));
                }
            }
            __syncwarp();
            const CrossView &v = KEYS ? (second ? p.dK : p.dV) : p.dQ;
            const bool exists = parts == 1 && r < (KEYS ? p.s : p.rows);
            const long long at = !exists ? -1 : KEYS ? b * v.sb + kh * v.sh + (long long)r * v.sn : cross_row(p, v, b, kh, r);
            // 16-byte chunks of this warp's rows and columns, a row's chunks by neighbouring lanes
            constexpr int kW = kCols / 8;
            const int ch = from / 8 + lane % kW;
            each_row<kW>(at, v.sn, [&](int, int rr, long long o) {
                if (o >= 0 && ch * 8 < p.d)
                    *reinterpret_cast<uint4 *>((__nv_bfloat16 *)v.ptr + o + ch * 8) =
                        *reinterpret_cast<const uint4 *>(stage + chunk_at(w4 * 32 + rr, ch));
            });
        }
        tc_fence_before();
        __syncwarp();
    }
    __syncthreads();
    if (warp == kIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kCols);
    }
}

template <int D, int W, bool FINE, bool CUT>
__global__ void __launch_bounds__(Geo<D, W>::kThreads, Geo<D, W>::kPerSM) cross_bwd_kernel(const __grid_constant__ BwdParams a) {
    const bool head = (int)blockIdx.x < a.first;
    const int index = (int)blockIdx.x - (head ? 0 : a.first);
    if (head == a.keys_first) cross_bwd<D, true, W, FINE, CUT>(a, index);
    else cross_bwd<D, false, W, FINE, CUT>(a, index);
}

// The sums of parts, in order, scaled and rounded: eight columns of a row a thread.  Bound by memory.
template <bool KEYS>
__global__ void __launch_bounds__(256) cross_sums_kernel(const CrossProblem p, const float *sums, int parts) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int rows = KEYS ? p.s : p.rows, width = KEYS ? 2 * p.d : p.d, per = width / 8;
    const long long total = (long long)p.B * p.kv * rows, i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long f = i / per;
    if (f >= total) return;
    int c = 8 * (int)(i - f * per);
    float o[8] = {};
    for (int q = 0; q < parts; ++q) {
        const float4 *src = reinterpret_cast<const float4 *>(sums + (q * total + f) * width + c);
        const float4 x = src[0], y = src[1];
        o[0] += x.x, o[1] += x.y, o[2] += x.z, o[3] += x.w, o[4] += y.x, o[5] += y.y, o[6] += y.z, o[7] += y.w;
    }
    const bool second = c >= p.d;
    if (second) c -= p.d;
    const float by = KEYS && !second ? 1.f : p.scale;
    const int bk = (int)(f / rows), r = (int)(f - (long long)bk * rows), b = bk / p.kv, k = bk - b * p.kv;
    const CrossView &v = KEYS ? (second ? p.dK : p.dV) : p.dQ;
    const long long at = KEYS ? b * v.sb + k * v.sh + (long long)r * v.sn : cross_row(p, v, b, k, r);
    *reinterpret_cast<uint4 *>((__nv_bfloat16 *)v.ptr + at + c) =
        make_uint4(pack2(o[0] * by, o[1] * by), pack2(o[2] * by, o[3] * by), pack2(o[4] * by, o[5] * by), pack2(o[6] * by, o[7] * by));
}

template <bool KEYS>
cudaError_t add_up(const CrossProblem &p, const float *sums, int parts, cudaStream_t stream) {
    const long long threads = (long long)p.B * p.kv * (KEYS ? 2LL * p.s : p.rows) * p.d / 8;
    return launch_pdl(cross_sums_kernel<KEYS>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, p, sums, parts);
}

// Parts of a kind's steps.  A CTA that walks longer than all CTAs spread over the SMs' places would take is cut, into
// parts of kSteps steps and more, whose sums a launch of its own adds in order.  With few states and many queries,
// above all, each key tile's CTA walks all queries (3 x 32 heads over 8, 1582 x 87, d = 16: the
// backward 125 us in one part, 60 in eight; 2 x 4 heads, 100 x 8192, d = 64: 131 against 34).
constexpr int kSteps = 8;
struct Parts {
    int of[2];
    size_t bytes[2];
};
Parts plan(const CrossProblem &p) {
    const int W = p.d > 64 ? 128 : 64, heads = p.B * p.kv;
    const long long places = (p.d > 64 ? 1 : 2) * (long long)kPlanSMs;
    const long long steps[2] = {(p.s + W - 1) / W, (long long)p.group * ((p.n + W - 1) / W)};
    const long long ctas[2] = {(long long)heads * ((p.rows + kRows - 1) / kRows), (long long)heads * ((p.s + kRows - 1) / kRows)};
    const long long cost[2] = {3 * steps[0], 4 * steps[1]};  // of a CTA, in products of a step
    const bool together = p.s > W;                           // (else the kinds' launches follow one another)
    Parts r = {{1, 1}, {0, 0}};
    if (p.rows == 0 || p.s == 0) return r;
    for (int i = 0; i < 2; ++i) {
        const long long all = ctas[i] * cost[i] + (together ? ctas[1 - i] * cost[1 - i] : 0), even = std::max(1LL, all / places);
        r.of[i] = (int)std::max(1LL, std::min((cost[i] + even - 1) / even, steps[i] / kSteps));
        r.bytes[i] = r.of[i] > 1 ? (size_t)r.of[i] * heads * (i ? 2ll * p.s : p.rows) * p.d * 4 : 0;
    }
    return r;
}

template <int D, int W, bool FINE, bool CUT>
cudaError_t backward(const CrossProblem &p, const Parts &parts, float *delta, float *sums, cudaStream_t stream) {
    using G = Geo<D, W>;
    BwdParams a;
    a.p = p;
    a.delta = delta;
    a.sums[0] = sums, a.sums[1] = sums + parts.bytes[0] / 4;
    int ctas[2] = {(p.rows + kRows - 1) / kRows, (p.s + kRows - 1) / kRows};
    for (int i = 0; i < 2; ++i) {
        a.tiles[i] = ctas[i], a.by_tiles[i] = Divide((uint32_t)std::max(1, ctas[i]));
        a.parts[i] = parts.of[i], a.by_parts[i] = Divide((uint32_t)parts.of[i]);
        ctas[i] *= p.B * p.kv * parts.of[i];
    }
    if (p.s > 0 && (!make_tile_map(&a.k, p.K, p.B, p.kv, p.s, p.d, W) || !make_tile_map(&a.v, p.V, p.B, p.kv, p.s, p.d, W)))
        return cudaErrorInvalidValue;
    if (p.s > 0 && p.n > 0 && (!make_tile_map(&a.q, p.Q, p.B, p.heads, p.n, p.d, W) || !make_tile_map(&a.g, p.dH, p.B, p.heads, p.n, p.d, W)))
        return cudaErrorInvalidValue;
    static SmemOnce allow;
    cudaError_t e = allow(cross_bwd_kernel<D, W, FINE, CUT>, G::kSmem);
    if (e != cudaSuccess) return e;
    auto run = [&](int grid) { return launch_pdl(cross_bwd_kernel<D, W, FINE, CUT>, dim3(grid), dim3(G::kThreads), G::kSmem, stream, a); };
    a.exact = p.s <= W;
    if (a.exact) {  // the keys' CTAs after the queries', who make D
        a.keys_first = false, a.first = ctas[0];
        if (ctas[0] > 0) e = run(ctas[0]);
        a.keys_first = true, a.first = ctas[1];
        if (e == cudaSuccess && ctas[1] > 0) e = run(ctas[1]);
    } else {
        if (ctas[0] > 0) e = launch_cross_delta(p, delta, stream);
        // first those that take longer: four products over the queries against three over the keys
        a.keys_first = 4LL * p.rows * parts.of[0] >= 3LL * p.s * parts.of[1];
        a.first = ctas[a.keys_first];
        if (e == cudaSuccess) e = run(ctas[0] + ctas[1]);
    }
    if (e == cudaSuccess && parts.of[0] > 1) e = add_up<false>(p, a.sums[0], parts.of[0], stream);
    if (e == cudaSuccess && parts.of[1] > 1) e = add_up<true>(p, a.sums[1], parts.of[1], stream);
    return e;
}

}  // namespace

size_t cross_tc_backward_sums(const CrossProblem &p) {
    const Parts parts = plan(p);
    return parts.bytes[0] + parts.bytes[1];
}

cudaError_t launch_cross_tc_backward(const CrossProblem &p, float *delta, float *sums, cudaStream_t stream) {
    const Parts parts = plan(p);
    auto fine = [&](auto f) {
        auto cut = [&](auto c) {
            constexpr bool F = decltype(f)::value, C = decltype(c)::value;
            return p.d > 64 ? backward<128, 128, F, C>(p, parts, delta, sums, stream) : backward<64, 64, F, C>(p, parts, delta, sums, stream);
        };
        return std::max(parts.of[0], parts.of[1]) > 1 ? cut(std::true_type{}) : cut(std::false_type{});
    };
    return p.s <= kFine ? fine(std::true_type{}) : fine(std::false_type{});
}

cudaError_t cross_bwd_read_and_clear_error(unsigned *out) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_cross_bwd_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_cross_bwd_error, &zero, sizeof(unsigned));
}

}  // namespace anchor
