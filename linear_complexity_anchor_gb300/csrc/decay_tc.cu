// Attention with decaying states in bf16 on the tensor cores (formulas in decay.cuh).
//
// The work comes in items: the rows of one batch entry's head (or of a segment of it), for 64 columns of c and of
// the state.  A CTA takes every gridDim.x-th item and walks its rows in chunks of 128; what loads, multiplies
// and stores runs on from item to item.  With i, j rows of a chunk of `count`, X the state before it (d x 64, fp32,
// in tensor memory) and X~ its bf16 image in shared memory:
//   S = a b^T,  P = g^(i-j) S below the diagonal (bf16),  o = p P c + w g^(i+1) (a X~)
//   X <- g^count X + b^T (s g^(count-1-j) c_j)
// (a pass backward in time: the other triangle, g^(j-i), g^(count-1-i), g^(j+1), chunks from the last to the first).
//
// Roundings: P and X~ to bf16, each once, where they meet c and a; the rows s g^(count-1-j) c_j are two bf16
// numbers (what the first leaves of them is the second), so that X's own rounding in X~ stays the only one of the part of o
// that goes by it (with one number o would carry three, 1.7 times a lone one, against 1.4).  A state that the caller is
// given is an fp32 result, which two numbers leave off by 3.9e-6 of itself.  So the chunks that count in it take a third
// product.  Heads that keep 0.73 of a state over a chunk: with m the weight of its middle row, b^T c itself and b^T times the
// rows of weight w / m - 1, whose roundings are less by as much; X takes m times their sum (such a chunk takes 0.2 us more).
// Others: the rows in three numbers, the third in the place of c once P c is complete (0.5 us).  A state is then off by 4 to 7e-7,
// as sums in fp32 are.  (4 x 16 heads x 16384, d = 128: 255 us without, 260, and 271 with three numbers throughout; made with the
// first two, before the products, 281.)
// What a chunk adds to X is a sum of its own, added by the rows, to nearest: the tensor cores' sums are cut off, which over many
// chunks would add up where X decays slowly (6e-6 of a state that reaches 3717 rows back, without a bound at a decay of 0; a
// loop that sums X there takes 3 % less at d = 64, nothing less at 128).  With X in registers a chunk took 5 % more at d = 64.  What fp32
// leaves of the factors g^count is carried from chunk to chunk (decay.cuh), for the same reason.
//
// Two groups of eight warps, a thread half of a row: the first makes P of the next chunk, and o from its two products; the
// second the weighted rows of c, X~ and X.  One warp loads tiles by TMA, one stores o's, one issues the products: P c, S of the
// next chunk, X, a X~, each as soon as its operands are there.  What a chunk takes is the second group's round (weights, X's
// product, X~, a X~) and the products' operands, which take three quarters of what the shared memory gives; all else is done
// beside it: 1.38 us at d = 64 and 1.88 at 128, from L2, without a state for the caller.  With one group for all, one step after the other, 1.6 and 1.9;
// with a group for each of the four steps 3.9, most of it spent on fetching instructions.
//
// STATES: the sums of a segment alone, s sum_j g^(rows-1-j) b_j^T c_j: the last product alone, with weights that count from the
// segment's end, so that no chunk's sum decays and those of kSums chunks are made in tensor memory.
// KEPT: a state is given to the caller.  (A call without one takes 3 % less in a kernel without that code.)
#include "cross_tc.cuh"
#include "decay.cuh"

#include <limits.h>

namespace anchor {

__device__ unsigned int g_decay_error;  // bit 0: a wait gave up

namespace {

using namespace cross_tc;

constexpr int kColumns = 64;                      // of c, of the state and of o, an item
constexpr int kTileC = kTile<kColumns>;
constexpr int kParts = 2;                         // threads of a row
constexpr int kGroup = 4 * kParts;                // warps of a group
constexpr int kWarpState = kGroup, kWarpLoad = 2 * kGroup, kWarpIssue = kWarpLoad + 1, kWarpStore = kWarpLoad + 2, kThreads = 32 * (kWarpLoad + 4);
constexpr int kSums = 4;                          // STATES: chunks whose sum is made in tensor memory
constexpr int kSlice = kColumns / kParts;         // columns of o, of the state and of c of a thread, kRows / kParts of P
// Registers of a thread: 640 threads have 96 at launch, 1920 for a lane of each warp; 8 * 136 + 8 * 80 + 4 * 40 = 1888.
constexpr int kRegsRows = 136, kRegsState = 80, kRegsOthers = 40;
constexpr uint32_t kColS = 0, kColP = 128, kColIn = 192, kColBy = 256, kColX = 320, kColAdd = 384, kCols = 512;  // of tensor memory

// D columns of a and b.  Heads of 16 and 32 are 64, whose other columns are zeros: a chunk takes what 64 take (8 x 12 heads x 4200, us: d = 64 51, 32:
// 49, 16: 47).
template <int D, bool STATES>
struct Geo {
    static constexpr int kStages = STATES ? 3 : D == 128 ? 2 : 3;
    static constexpr int kA = 0, kB = STATES ? 0 : kTile<D>, kC = kB + kTile<D>, kStage = kC + kTileC;  // of a stage
    static constexpr int kWeighted = STATES ? 2 : 1;  // buffers of the weighted rows of c
    static constexpr int kRing = 0, kW = kRing + kStages * kStage, kImg = kW + kWeighted * 2 * kTileC, kOut = kImg + (STATES ? 0 : D * kColumns * 2),
                         kPow = kOut + (STATES ? 0 : kTileC), kBars = kPow + (STATES ? 0 : kGroup * 64 * 4);
    static constexpr int kNBars = 2 * kStages + 12, kSmem = kBars + kNBars * 8 + 8;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kSlice == 32, "a row's part of a state fills two halves of its weighted rows");
};

struct TcParams {
    DecayProblem p;
    TileMap a[3], b[3], c[3], o[3];
    int items, halves;
    Divide by_segs, by_heads;
};

__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, const void *src, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"((uint64_t)map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// One item, as every warp sees it.
template <bool STATES>
struct Item {
    const DecayPass *q;
    int which, b, h, slice, seg, half, r0, rows, K, end, of, length;  // end: rows of the segment; length: of the entry
    bool back, turned;
    float rate;
    const float *from;  // states outside, or null
    float *to;
    int next_length;    // what is read for the next item is asked for while this one is walked
    float next_rate;

    __device__ __forceinline__ int place(const TcParams &a, int index, int &of) {
        const int kinds = STATES ? a.p.kinds : a.p.passes;
        // the halves and passes of a segment are neighbours, so that what they share is read once
        const int x = a.halves == 2 ? index >> 1 : index, y = kinds == 3 ? x / 3 : kinds == 2 ? x >> 1 : x;
        half = index - x * a.halves, of = x - y * kinds;
        return y;
    }
    __device__ __forceinline__ void ask(const TcParams &a, int index) {
        if (index >= a.items) return;
        int of, was = half;
        const int slice = a.by_segs.of(place(a, index, of)), b = a.by_heads.of(slice);
        half = was;
        next_length = decay_length(a.p, b), next_rate = decay_rate(a.p.log_decay, slice - b * a.p.heads);
    }
    __device__ __forceinline__ void set(const TcParams &a, int index) {
        const DecayProblem &p = a.p;
        const int segs = STATES ? p.segs - 1 : p.segs;
        const int y = place(a, index, of);
        slice = a.by_segs.of(y);
        b = a.by_heads.of(slice), h = slice - b * p.heads;
        length = next_length;
        rate = next_rate;
        ask(a, index + (int)gridDim.x);
        which = of;
        if (STATES)
            while (p.pass[which].kind != of) ++which;  // a pass of that kind
        q = &p.pass[which];
        back = q->back, turned = STATES ? false : q->turned;
        seg = y - slice * segs + (STATES && back ? 1 : 0);  // the last one (in time) has no state behind it
        r0 = seg * p.seg, end = min(p.seg, p.n - r0);
        rows = decay_rows(p, seg, length);
        K = (rows + kRows - 1) / kRows;
        const long long dd = p.d * p.d;
        float *in = p.states + (((long long)(STATES ? of : q->kind) * p.slices() + slice) * p.segs + seg) * dd;
        from = STATES ? nullptr : p.segs > 1 ? in : q->state ? q->state + slice * dd : nullptr;
        to = STATES ? in : q->last && seg == (back ? 0 : p.segs - 1) ? q->last + slice * dd : nullptr;
    }
    // chunk k: its first row in the segment, its rows; whether X takes it; whether there is a state before it
    __device__ __forceinline__ int first(int k) const { return (back ? K - 1 - k : k) * kRows; }
    __device__ __forceinline__ int count(int k) const { return (back ? k == 0 : k + 1 == K) ? rows - (K - 1) * kRows : kRows; }
    __device__ __forceinline__ bool takes(int k) const { return STATES || k + 1 < K || to != nullptr; }
    // The chunks that count in a state that the caller is given, from the first (in time), so that their weighted rows are three
    // numbers: not those of which the decay leaves less than e^-2.
    __device__ __forceinline__ int first_fine(const TcParams &a) const {
        bool given = !STATES && to;
        if (STATES)
            for (int x = 0; x < a.p.passes; ++x) given = given || (a.p.pass[x].kind == of && a.p.pass[x].last);
        if (!given) return INT_MAX;
        const float far = ((float)(back ? K * kRows + r0 : length - r0) - __fdividef(2.f, fabsf(rate))) * (1.f / kRows);  // (rate 0: all)
        return far >= 1.f ? (int)far : 0;
    }
    // of these, those of a head that keeps most of a state over a chunk: weights apart from the one of the middle row
    __device__ __forceinline__ bool centred() const { return !STATES && rate > -0.0025f; }
    __device__ __forceinline__ bool has(int k) const { return k > 0 || from != nullptr; }
};

// This thread's columns of a row of c times its weight w, as two bf16 numbers in two tiles.  `on`: the row counts (else
// zeros, whatever it holds).  With w = u + v in bf16 (2^-18 of w is left out), h = c u rounded, and l = (c u - h) + c v, of
// which the first part is exact: three instructions for two numbers.  (From fp32 products
// the states would be off by 2.4e-6 of themselves instead of 3.9e-6, and a chunk takes 3 to 8 % more.)
__device__ __forceinline__ void weight_row(const uint8_t *tile, uint8_t *hi, uint8_t *lo, int row, int part, float w, bool on) {
    constexpr int N = kSlice / 8;
    const __nv_bfloat16 u1 = __float2bfloat16_rn(w);
    const __nv_bfloat162 u = __bfloat162bfloat162(u1), v = __float2bfloat162_rn(w - __bfloat162float(u1));
    uint4 x4[N];
#pragma unroll
    for (int c = 0; c < N; ++c) x4[c] = on ? *reinterpret_cast<const uint4 *>(tile + chunk_at(row, N * part + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < N; ++c) {
        uint4 h4, l4;
        const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&x4[c]);
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&h4), *l = reinterpret_cast<__nv_bfloat162 *>(&l4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = __hmul2(x[i], u);
            l[i] = __hfma2(x[i], v, __hfma2(x[i], u, __hneg2(h[i])));
        }
        *reinterpret_cast<uint4 *>(hi + chunk_at(row, N * part + c)) = h4;
        *reinterpret_cast<uint4 *>(lo + chunk_at(row, N * part + c)) = l4;
    }
}
// What those two leave of the row, a third number, over the row itself.
__device__ __forceinline__ void rest_row(uint8_t *tile, const uint8_t *hi, const uint8_t *lo, int row, int part, float w) {
    constexpr int N = kSlice / 8;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const int at = chunk_at(row, N * part + c);
        uint4 *to = reinterpret_cast<uint4 *>(tile + at);
        const uint4 x4 = *to, h4 = *reinterpret_cast<const uint4 *>(hi + at), l4 = *reinterpret_cast<const uint4 *>(lo + at);
        auto rest = [&](uint32_t x, uint32_t h, uint32_t l) {
            const float a = fmaf(__uint_as_float(x << 16), w, -__uint_as_float(h << 16)) - __uint_as_float(l << 16);
            const uint32_t top = 0xffff0000u;
            const float b = fmaf(__uint_as_float(x & top), w, -__uint_as_float(h & top)) - __uint_as_float(l & top);
            return pack2(a, b);
        };
        *to = make_uint4(rest(x4.x, h4.x, l4.x), rest(x4.y, h4.y, l4.y), rest(x4.z, h4.z, l4.z), rest(x4.w, h4.w, l4.w));
    }
}

// What the issuing warp does it does as a whole, one lane of it elected for each product: with uniform control the descriptors
// are made by uniform instructions.  (Issued by a lane on a branch of its own a product took 75 to 140 cycles: 343 us for 4 x
// 16 heads, 16384, d = 128, against 255.)
__device__ __forceinline__ void product(uint32_t to, uint64_t a, uint64_t b, uint32_t id, uint32_t add) {
    asm volatile(
        "{\n .reg .pred e, p;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(to),
        "l"(a), "l"(b), "r"(id), "r"(add)
        : "memory");
}
__device__ __forceinline__ void product_tmem(uint32_t to, uint32_t a, uint64_t b, uint32_t id, uint32_t add) {
    asm volatile(
        "{\n .reg .pred e, p;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(to),
        "r"(a), "l"(b), "r"(id), "r"(add)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}
// False once a phase has not come within kTries tries of up to 2 us each (the error word is set on the way out).  In a few
// instructions: what waits take in the instruction cache is taken from the steps between them.
constexpr int kTries = 1 << 20;
__device__ __forceinline__ bool hold(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .s32 i;\n mov.s32 i, %3;\n"
        "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n @p bra over;\n"
        " sub.s32 i, i, 1;\n setp.gt.s32 q, i, 0;\n @q bra again;\n"
        "over:\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kTries)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool all_hold(uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, hold(bar, parity)); }

__device__ __forceinline__ void tmem_ld16(uint32_t at, float *v) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                   "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
template <int D, bool STATES, bool KEPT>
__global__ void __launch_bounds__(kThreads, 1) decay_kernel(const __grid_constant__ TcParams a) {
    using G = Geo<D, STATES>;
    constexpr int NS = G::kStages;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G::kBars);
    // full: a stage's tiles have landed; over: the products of its chunk are complete; p_ready: P is there and the o before has
    // been read; x_ready: so are X~, X and the weighted rows; x_full: so is what the chunk adds to X;
    // c_free: (of a chunk with third numbers) P c is complete; m_ready: they are in the place of c
    uint64_t *full = bars, *over = full + NS, *s_full = over + NS /* [2] */, *p_ready = s_full + 2, *x_ready = p_ready + 1 /* [2] */,
             *x_full = x_ready + 2 /* [2] */, *staged = x_full + 2, *sent = staged + 1, *done = sent + 1,
             *c_free = done + 1, *m_ready = c_free + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + G::kNBars);
    const DecayProblem &p = a.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    auto gave_up = [] { atomicOr(&g_decay_error, 1u); };
    if (smem_u32(sm) & 1023u) {  // (there is no room to move the tiles: never seen)
        if (threadIdx.x == 0) gave_up();
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) mbar_init(full + s, 1), mbar_init(over + s, 1);
        for (int s = 0; s < 2; ++s) mbar_init(s_full + s, 1), mbar_init(x_ready + s, kGroup), mbar_init(x_full + s, 1);
        mbar_init(p_ready, kGroup);
        mbar_init(staged, kGroup);
        mbar_init(sent, 1);
        mbar_init(done, 1);
        mbar_init(c_free, 1);
        mbar_init(m_ready, kGroup);
        fence_mbar_init();
    }
    if (warp == kWarpIssue) tmem_alloc(s_tmem, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
    grid_dependency_wait();
    grid_dependents_launch();

    Item<STATES> it;
    it.ask(a, blockIdx.x);
    auto stage = [&](int g) { return sm + G::kRing + g % NS * G::kStage; };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    auto around = [](int g) { return (uint32_t)((g / NS) & 1); };  // parity of a stage's barriers
    auto one = [](int g) { return (uint32_t)(g & 1); };            // of a barrier that each chunk passes,
    auto two = [](int g) { return (uint32_t)((g >> 1) & 1); };     // and of a pair of barriers

    if (!STATES && warp >= kWarpLoad) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOthers));
    if (warp == kWarpLoad) {
        int g = 0;
        bool ok = true;
        for (int index = blockIdx.x; index < a.items && ok; index += gridDim.x) {
            it.set(a, index);
            if (it.from) {  // the state that the item begins with, into L2: it is read some chunks from now
                const int bytes = p.d * min(p.d, kColumns) * 4;
                for (int o = 128 * lane; o < bytes; o += 128 * 32) {
                    const int at = p.d <= kColumns || it.turned ? it.half * bytes + o : o / 256 * (p.d * 4) + it.half * 256 + o % 256;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(it.from) + at));
                }
            }
            // STATES: b and c in the order of the kind, not turned
            const bool swap = STATES && it.q->turned;
            const TileMap &ma = a.a[it.which], &mb = swap ? a.c[it.which] : a.b[it.which], &mc = swap ? a.b[it.which] : a.c[it.which];
            for (int k = 0; k < it.K; ++k, ++g) {
                const int row = it.r0 + it.first(k), st = g % NS;
                uint8_t *to = stage(g);
                if (g >= NS && !(ok = all_hold(over + st, around(g - NS)))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(full + st, G::kStage);
                    if (!STATES) load_tile<D, kRows, kRows>(to + G::kA, ma, full + st, row, it.h, it.b);
                    load_tile<D, kRows, kRows>(to + G::kB, mb, full + st, row, it.h, it.b);
                    tma_load_4d(to + G::kC, &mc.map, full + st, kColumns * it.half, row, it.h * mc.by_head, it.b * mc.by_batch);
                }
                __syncwarp();
            }
        }
        // the CTA leaves only once its copies have landed
        for (int x = max(0, g - NS); x < g; ++x) ok = all_hold(full + x % NS, around(x)) && ok;
        if (!ok) gave_up();
    } else if (warp == kWarpIssue) {
        {
            const uint32_t base = smem_u32(sm);
            auto at = [&](int g) { return base + G::kRing + g % NS * G::kStage; };
            constexpr uint32_t idS = idesc_bf16_f32(kRows, kRows, false, false), idO = idesc_bf16_f32(kRows, kColumns, false, true),
                               idX = idesc_bf16_f32(kRows, 2 * kColumns, true, true);
            // What chunks add to X, b^T [hi | lo], in 128 columns whose halves are added by the rows (fresh: begun anew).  With 64
            // columns of b the product has 128 rows all the same: the upper ones are made of the tile of c behind b's, and are not read.
            auto product_x = [&](int g, uint32_t to, bool fresh) {
                const uint64_t b = smem_desc_sw128(at(g) + G::kB, kBlock, 1024), w = desc_mn(base + G::kW + (STATES ? (g & 1) * 2 * kTileC : 0));
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k) product(tmem + to, b + step_mn(k), w + step_mn(k), idX, !fresh || k > 0 ? 1u : 0u);
            };
            // and b^T times the third numbers, to the second half
            auto product_m = [&](int g, uint32_t to) {
                const uint64_t b = smem_desc_sw128(at(g) + G::kB, kBlock, 1024), m = desc_mn(at(g) + G::kC);
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k) product(tmem + to + kColumns, b + step_mn(k), m + step_mn(k), idO | 1u << 15, 1u);
            };
            int g = 0, scored = 0, fines = 0;  // scored: chunks whose S has been issued; fines: chunks with third numbers
            bool ok = true;
            for (int index = blockIdx.x; index < a.items && ok; index += gridDim.x) {
                it.set(a, index);
                const int first_fine = KEPT ? it.first_fine(a) : 0;
                const bool centred = it.centred();
                auto fine = [&](int k) { return KEPT && k >= first_fine; };
                for (int k = 0; k < it.K && ok; ++k, ++g) {
                    const int st = g % NS;
                    if constexpr (STATES) {
                        if (!(ok = all_hold(x_ready + (g & 1), two(g)))) break;
                        tc_fence_after();
                        product_x(g, 2 * kColumns * (k / kSums & 1), k % kSums == 0);
                        if (fine(k)) product_m(g, 2 * kColumns * (k / kSums & 1));
                        commit(x_full + (g & 1));
                        commit(over + st);
                    } else {
                        const bool partial = it.count(k) < kRows;
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            // S of this chunk, or, where its tiles have landed, of the next (which may be another item's)
                            bool score = scored == g;
                            if (score) {
                                if (!(ok = all_hold(full + scored % NS, around(scored)))) break;
                            } else {
                                score = part > 0 && scored == g + 1 && __all_sync(0xffffffffu, mbar_test(full + scored % NS, around(scored)));
                            }
                            if (score) {
                                tc_fence_after();
                                const uint64_t ad = desc_k(at(scored) + G::kA), bd = desc_k(at(scored) + G::kB);
#pragma unroll
                                for (int s = 0; s < D / 16; ++s) product(tmem + kColS, ad + step_k(s), bd + step_k(s), idS, s > 0 ? 1u : 0u);
                                commit(s_full + (scored & 1));
                                ++scored;
                            }
                            if (part == 0) {
                                // (rows of c behind the length are zeros by then)
                                if (partial && !(ok = all_hold(x_ready, one(g)))) break;
                                if (!(ok = all_hold(p_ready, one(g)))) break;
                                tc_fence_after();
                                const uint64_t cd = desc_mn(at(g) + G::kC);
#pragma unroll
                                for (int s = 0; s < kRows / 16; ++s)
                                    product_tmem(tmem + kColIn, tmem + kColP + 8 * s, cd + step_mn(s), idO, s > 0 ? 1u : 0u);
                                if (fine(k) && !centred) commit(c_free);
                            } else {
                                if (!partial && !(ok = all_hold(x_ready, one(g)))) break;
                                tc_fence_after();
                                if (it.takes(k)) product_x(g, kColAdd, true);
                                if (fine(k)) {
                                    if (!centred) {
                                        if (!(ok = all_hold(m_ready, one(fines)))) break;
                                        ++fines;
                                        tc_fence_after();
                                    }
                                    product_m(g, kColAdd);
                                }
                                commit(x_full);
                                if (it.has(k)) {
#pragma unroll
                                    for (int s = 0; s < D / 16; ++s)
                                        product(tmem + kColBy, desc_k(at(g) + G::kA) + step_k(s), desc_mn(base + G::kImg) + step_mn(s), idO, s > 0 ? 1u : 0u);
                                }
                                commit(over + st);
                            }
                        }
                    }
                }
            }
            commit(done);
            if (!all_hold(done, 0u) || !ok) gave_up();
        }
    } else if (warp == kWarpStore) {
        if (!STATES && lane == 0) {
            // o of a chunk (rows behind the length are zeros; what is not in the tensor is not written)
            int g = 0;
            bool ok = true;
            for (int index = blockIdx.x; index < a.items && ok; index += gridDim.x) {
                it.set(a, index);
                const TileMap &m = a.o[it.which];
                for (int k = 0; k < it.K; ++k, ++g) {
                    if (!(ok = hold(staged, one(g)))) break;
                    tma_store_4d(&m.map, sm + G::kOut, kColumns * it.half, it.r0 + it.first(k), it.h * m.by_head, it.b * m.by_batch);
                    bulk_commit_group();
                    bulk_wait_group_read0();
                    mbar_arrive(sent);
                }
            }
            bulk_wait_group0();
            if (!ok) gave_up();
        }
        __syncwarp();
    } else if (warp >= kWarpState && warp < kWarpLoad) {
        // ---------------------------------------------------------------------- the state, and the weighted rows of c
        if constexpr (!STATES) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsState));
        const int w4 = warp & 3, part = (warp - kWarpState) >> 2, row = w4 * 32 + lane;
        const uint32_t tX = tmem + ((uint32_t)(w4 * 32) << 16) + kColX + kSlice * part;
        const bool mine = w4 * 32 < D;  // the warp has rows of X
        int g = 0, fines = 0;
        bool ok = true;
        // this thread's part of a row of c
        auto zero_part = [&](uint8_t *c) {
            for (int x = 0; x < kSlice / 8; ++x) *reinterpret_cast<uint4 *>(c + chunk_at(row, kSlice / 8 * part + x)) = make_uint4(0, 0, 0, 0);
        };
        // 16 columns of this thread's part of X, with what the chunk before has added
        auto take_x = [&](int c, float *x, float f) {
            const uint64_t f2 = f32x2(f, f);
            float hi[16], lo[16];
            tmem_ld16(tX + c, x);
            tmem_ld16(tX + kColAdd - kColX + c, hi);
            tmem_ld16(tX + kColAdd - kColX + kColumns + c, lo);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                f32x2_split(fma_f32x2(f2, add_f32x2(f32x2(hi[i], hi[i + 1]), f32x2(lo[i], lo[i + 1])), f32x2(x[i], x[i + 1])), x[i], x[i + 1]);
        };
        for (int index = blockIdx.x; index < a.items && ok; index += gridDim.x) {
            it.set(a, index);
            const float rate = it.rate;
            const int first_fine = KEPT ? it.first_fine(a) : 0;
            const bool centred = it.centred();
            auto fine = [&](int k) { return KEPT && k >= first_fine; };
            const int c0 = it.half * kColumns + kSlice * part;  // this thread's columns of the state
            // four columns of this thread's row of the state outside (zeros where there is none)
            auto outside = [&](int c, float *x) {
                if (!it.from || row >= p.d || c0 + c >= p.d) {
                    x[0] = x[1] = x[2] = x[3] = 0.f;
                } else if (it.turned) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = it.from[(c0 + c + i) * p.d + row];
                } else {
                    *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(it.from + row * p.d + c0 + c);
                }
            };
            float y[kSlice], mid = 1.f;  // what is written to `to`; the weight that chunks are taken apart from
            if constexpr (STATES) {
#pragma unroll
                for (int i = 0; i < kSlice; ++i) y[i] = 0.f;
                // y plus the sum of kSums chunks
                auto add = [&](int sum) {
                    if (!mine) return;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kSlice; c += 16) {
                        float hi[16], lo[16];
                        tmem_ld16(tX - kColX + 2 * kColumns * (sum & 1) + c, hi);
                        tmem_ld16(tX - kColX + 2 * kColumns * (sum & 1) + kColumns + c, lo);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[c + i] += hi[i] + lo[i];
                    }
                    tc_fence_before();
                };
                for (int k = 0; k < it.K; ++k, ++g) {
                    const int first = it.first(k), count = it.count(k);
                    const float w = it.q->s * expf(rate * (float)max(it.back ? first + row + 1 : it.rows - 1 - first - row, 0));
                    if (!(ok = hold(full + g % NS, around(g)))) break;
                    if (g > 1 && !(ok = hold(x_full + (g & 1), two(g - 2)))) break;
                    uint8_t *hi = sm + G::kW + (g & 1) * 2 * kTileC;
                    uint8_t *c = stage(g) + G::kC;
                    weight_row(c, hi, hi + kTileC, row, part, w, row < count);
                    if (count < kRows) {  // zeros, whatever is there, in the other operand too
                        if (part == 0) zero_rows<D>(stage(g) + G::kB, row, count, kRows);
                        if (row >= count) zero_part(c);
                    }
                    if (fine(k)) rest_row(c, hi, hi + kTileC, row, part, w);
                    fence_proxy_async_smem();
                    arrive(x_ready + (g & 1));
                    if (k > 0 && k % kSums == 0) {
                        if (!(ok = hold(x_full + ((g - 1) & 1), two(g - 1)))) break;
                        add(k / kSums - 1);
                    }
                }
                if (!ok) break;
                if (it.K > 0) {
                    if (!(ok = hold(x_full + ((g - 1) & 1), two(g - 1)))) break;
                    add((it.K - 1) / kSums);
                }
            } else {
                // factors of a chunk: of X (rest: what fp32 leaves of it, owed: has left of those before), of this thread's row of c
                float keep = 0.f, rest = 0.f, owed = 0.f, weight = 0.f, was = 1.f;
                int counted = -1;
                for (int k = 0; k < it.K; ++k, ++g) {
                    const int count = it.count(k);
                    was = mid;
                    if (count != counted || (KEPT && k == first_fine)) {
                        counted = count;
                        const float far = (float)(it.back ? row + 1 : max(count - 1 - row, 0));
                        if (centred && fine(k)) weight = expf(rate * (far - 64.f)) - 1.f, mid = it.q->s * expf(rate * 64.f);
                        else weight = it.q->s * expf(rate * far);
                        keep = expf(rate * (float)count);
                        // (few factors do without: 128 x 12 x 197 would take 82 us instead of 77)
                        rest = it.K > 4 ? decay_rest(rate, (float)count, keep) : 0.f;
                    }
                    // the rows of c, once the product of the chunk before is complete
                    if (!(ok = hold(full + g % NS, around(g)))) break;
                    if (g > 0 && !(ok = hold(x_full, one(g - 1)))) break;
                    uint8_t *c = stage(g) + G::kC, *hi = sm + G::kW;
                    if (it.takes(k)) weight_row(c, hi, hi + kTileC, row, part, weight, row < count);
                    if (count < kRows) {
                        // zeros, whatever is there, in both operands of X and in that of P c (S may be reading b: what it makes of
                        // these rows is masked)
                        if (part == 0) zero_rows<D>(stage(g) + G::kB, row, count, kRows);
                        if (row >= count) zero_part(c);
                    }
                    // X~ and X, once a X~ of the chunk before is complete too
                    if (g > 0 && !(ok = hold(over + (g - 1) % NS, around(g - 1)))) break;
                    if ((k == 0 || it.has(k)) && mine) {
                        tc_fence_after();
                        const float by = decay_next(keep, rest, owed);
                        const uint64_t keep2 = f32x2(by, by);
#pragma unroll
                        for (int c = 0; c < kSlice; c += 16) {
                            float x[16];
                            if (k > 0) {
                                take_x(c, x, was);
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; i += 4) outside(c + i, x + i);
                            }
#pragma unroll
                            for (int i = 0; i < 16; i += 8)
                                *reinterpret_cast<uint4 *>(sm + G::kImg + chunk_at(row, (kSlice * part + c + i) / 8)) =
                                    make_uint4(pack2(x[i], x[i + 1]), pack2(x[i + 2], x[i + 3]), pack2(x[i + 4], x[i + 5]), pack2(x[i + 6], x[i + 7]));
                            uint32_t z[16];
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float y0, y1;
                                f32x2_split(mul_f32x2(f32x2(x[i], x[i + 1]), keep2), y0, y1);
                                z[i] = __float_as_uint(y0), z[i + 1] = __float_as_uint(y1);
                            }
                            tmem_st16(tX + c, z);
                        }
                        tmem_st_wait();
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    arrive(x_ready);
                    if (fine(k) && !centred) {
                        if (!(ok = hold(c_free, one(fines)))) break;
                        ++fines;
                        rest_row(c, hi, hi + kTileC, row, part, weight);
                        fence_proxy_async_smem();
                        arrive(m_ready);
                    }
                }
                // (the last product, before X is read here or X~ is written for the next item)
                if (!ok || (it.to && it.K > 0 && !(ok = hold(x_full, one(g - 1))))) break;
            }
            if (!it.to || !mine) continue;
            if constexpr (!STATES) {
                if (it.K > 0) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kSlice; c += 16) take_x(c, y + c, mid);
                } else {
#pragma unroll
                    for (int i = 0; i < kSlice; i += 4) outside(i, y + i);
                }
            }
            // By way of this warp's part of the weighted rows, whose product is complete, so that rows go out 128 bytes at a
            // time (each thread its own row, 16 bytes at a time: 1.5 us).  Rolled: what an item does once is mostly fetched (128 x
            // 12 x 197, d = 64: 80 us unrolled, 76).
            auto at = [&](int r, int x) { return reinterpret_cast<float4 *>(sm + G::kW + (x >> 2) * kTileC + chunk_at(r, 4 * part + (x & 3))); };
#pragma unroll
            for (int i = 0; i < 8; ++i) *at(row, i) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            __syncwarp();
            const int x = lane & 7;
#pragma unroll 1
            for (int i = 0; i < 32; i += 4) {
                const int r = w4 * 32 + i + (lane >> 3);
                if (r < p.d && c0 + 4 * x < p.d) *reinterpret_cast<float4 *>(it.to + r * p.d + c0 + 4 * x) = *at(r, x);
            }
            __syncwarp();
        }
        if (!ok) gave_up();
    } else if (!STATES && warp < kWarpState) {
        // ---------------------------------------------------------------------- P and o
        if constexpr (!STATES) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
        const int w4 = warp & 3, part = warp >> 2, row = w4 * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
        constexpr int kP = kRows / kParts;
        const int j0 = kP * part;
        uint64_t pf[kP / 2];
        float *table = reinterpret_cast<float *>(sm + G::kPow) + warp * 64;
        int index = (int)blockIdx.x - (int)gridDim.x, k = 0, counted = -1;
        int count = 0, count_o = 0;      // rows of this chunk, and of the one whose o comes next
        float by = 0.f, by_o = 0.f;      // factors of a X~
        bool has = false, has_o = false;
        bool ok = true;
        it.K = 0;
        for (int g = 0;; ++g) {
            // the next chunk, which may be another item's: its P comes before the o of the chunk before
            bool more = true;
            if (++k >= it.K) {
                do {
                    index += gridDim.x;
                    if (!(more = index < a.items)) break;
                    it.set(a, index);
                    if (it.K * kRows < it.end) {  // chunks of the segment from the length on
                        __nv_bfloat16 *O = (__nv_bfloat16 *)it.q->o.ptr + it.b * it.q->o.sb + it.h * it.q->o.sh + it.r0 * it.q->o.sn + it.half * kColumns;
                        const int per = p.d == 16 ? 1 : p.d == 32 ? 2 : 3, col = (int)threadIdx.x % (1 << per) * 8;
                        for (int x = it.K * kRows + ((int)threadIdx.x >> per); x < it.end; x += 32 * kGroup >> per)
                            *reinterpret_cast<uint4 *>(O + (long long)x * it.q->o.sn + col) = make_uint4(0, 0, 0, 0);
                    }
                } while (it.K == 0);
                if (more) {
                    // P's factors for this thread's columns, p g^(i - j) (backward g^(j - i)), 0 on the other side of the diagonal
                    const float rate2 = it.rate * kLog2e, scale = it.q->p;
                    // 32 columns of 32 rows have 63 distances (and one more, that is not read), in the order in which a row reads them
#pragma unroll
                    for (int y = 0; y < kP; y += 32) {
                        if (it.back ? j0 + y < w4 * 32 : j0 + y > w4 * 32) continue;  // (not read)
                        const int least = it.back ? j0 + y - w4 * 32 - 31 : w4 * 32 - j0 - y - 31;  // of lane 0 (backward 31) and column 31 (0)
                        __syncwarp();
#pragma unroll
                        for (int x = 0; x < 64; x += 32) {
                            const int far = it.back ? least + x + lane : least + 62 - x - lane;
                            table[x + lane] = far >= 0 ? scale * ex2(rate2 * (float)far) : 0.f;
                        }
                        __syncwarp();
                        const float *at = table + 31 - lane;
#pragma unroll
                        for (int x = 0; x < 32; x += 2) pf[(y + x) / 2] = f32x2(at[x], at[x + 1]);
                    }
                    k = 0, counted = -1;
                }
            }
            if (more) {
                has = it.has(k), count = it.count(k);
                if (count != counted) {
                    counted = count;
                    by = it.q->w * expf(it.rate * (float)(it.back ? max(count - 1 - row, 0) : row + 1));
                }
                if (!(ok = hold(s_full + (g & 1), two(g)))) break;
                tc_fence_after();
#pragma unroll
                for (int y = 0; y < kP; y += 32) {
                    uint32_t packed[16];
                    // (blocks on the other side of the diagonal are not read)
                    if (it.back ? j0 + y < w4 * 32 || j0 + y >= count : j0 + y > w4 * 32) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) packed[x] = 0u;
                    } else {
                        float s[32];
                        tmem_ld32(lanes + kColS + j0 + y, s);
                        tmem_ld_wait();
                        if (j0 + y + 32 > count) {  // (0 times what is there may be a NaN)
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (j0 + y + x >= count) s[x] = 0.f;
                        }
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            float s0, s1;
                            f32x2_split(mul_f32x2(f32x2(s[2 * x], s[2 * x + 1]), pf[(y + 2 * x) / 2]), s0, s1);
                            packed[x] = pack2(s0, s1);
                        }
                    }
                    tmem_st16(lanes + kColP + (j0 + y) / 2, packed);
                }
                tmem_st_wait();
            }
            uint32_t u[kSlice / 2];
            if (g > 0) {
                if (!(ok = hold(over + (g - 1) % NS, around(g - 1)))) break;
                tc_fence_after();
                const uint64_t f2 = f32x2(by_o, by_o);
#pragma unroll
                for (int c = 0; c < kSlice; c += 16) {
                    float in[16], x[16];
                    tmem_ld16(lanes + kColIn + kSlice * part + c, in);
                    if (has_o) {
                        tmem_ld16(lanes + kColBy + kSlice * part + c, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = 0.f;
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float y, z;
                        f32x2_split(fma_f32x2(f2, f32x2(x[2 * i], x[2 * i + 1]), f32x2(in[2 * i], in[2 * i + 1])), y, z);
                        u[c / 2 + i] = row < count_o ? pack2(y, z) : 0u;
                    }
                }
            }
            tc_fence_before();
            if (more) arrive(p_ready);
            if (g > 0) {
                if (g > 1 && !(ok = hold(sent, one(g - 2)))) break;  // the chunk before has left `out`
#pragma unroll
                for (int x = 0; x < kSlice / 8; ++x)
                    *reinterpret_cast<uint4 *>(sm + G::kOut + chunk_at(row, kSlice / 8 * part + x)) = make_uint4(u[4 * x], u[4 * x + 1], u[4 * x + 2], u[4 * x + 3]);
                fence_proxy_async_smem();
                arrive(staged);
            }
            if (!more) break;
            has_o = has, count_o = count, by_o = by;
        }
        if (!ok) gave_up();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpIssue) tmem_dealloc(tmem, kCols);
}

template <int D, bool STATES, bool KEPT>
cudaError_t launch(const DecayProblem &p, cudaStream_t stream) {
    TcParams a;
    a.p = p;
    for (int i = 0; i < p.passes; ++i) {
        const DecayPass &q = p.pass[i];
        if (!make_tile_map(&a.a[i], q.a, p.B, p.heads, p.n, p.d, kRows) || !make_tile_map(&a.b[i], q.b, p.B, p.heads, p.n, p.d, kRows) ||
            !make_tile_map(&a.c[i], q.c, p.B, p.heads, p.n, p.d, kRows) || (!STATES && !make_tile_map(&a.o[i], q.o, p.B, p.heads, p.n, p.d, kRows)))
            return cudaErrorInvalidValue;
    }
    const int segs = STATES ? p.segs - 1 : p.segs;
    a.halves = D / kColumns;
    a.items = (int)(p.slices() * segs * (STATES ? p.kinds : p.passes) * a.halves);
    a.by_segs = Divide((uint32_t)segs), a.by_heads = Divide((uint32_t)p.heads);
    static SmemOnce once;
    const cudaError_t e = once(decay_kernel<D, STATES, KEPT>, Geo<D, STATES>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(decay_kernel<D, STATES, KEPT>, dim3((unsigned)std::min(a.items, kPlanSMs)), dim3(kThreads), Geo<D, STATES>::kSmem, stream, a);
}

template <bool STATES>
cudaError_t launch(const DecayProblem &p, cudaStream_t stream) {
    bool kept = false;
    for (int i = 0; i < p.passes; ++i) kept = kept || p.pass[i].last;
    return p.d == 128 ? (kept ? launch<128, STATES, true>(p, stream) : launch<128, STATES, false>(p, stream))
                      : (kept ? launch<64, STATES, true>(p, stream) : launch<64, STATES, false>(p, stream));
}

}  // namespace

cudaError_t launch_decay_tc_states(const DecayProblem &p, cudaStream_t stream) { return launch<true>(p, stream); }
cudaError_t launch_decay_tc(const DecayProblem &p, cudaStream_t stream) { return launch<false>(p, stream); }
cudaError_t decay_read_and_clear_error(unsigned *out) {
    const unsigned zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(out, g_decay_error, sizeof(unsigned));
    return e == cudaSuccess ? cudaMemcpyToSymbol(g_decay_error, &zero, sizeof(unsigned)) : e;
}

}  // namespace anchor
