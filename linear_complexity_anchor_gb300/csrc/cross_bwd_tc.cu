// Cross attention backward in bf16 on the tensor cores (formulas in include/anchor_attn.h):
//   P = 2^(c S - lse), S = Q K^T;  dS = P o (dH V^T - D), D = dH . H;
//   dQ = scale dS K;  dV = P^T dH;  dK = scale dS^T Q.
//
// Two kernels, one that keeps queries and one that keeps keys, so that every gradient is summed in
// tensor memory by one CTA in a fixed order, without atomics.  S and dP are made twice for
// that: seven products where five would do.
//
//   queries   a tile of 128 rows of Q and dH stays, the keys of the entry stream by:
//             S = Q K^T, dP = dH V^T, dQ += dS K
//   keys      a tile of 128 rows of K and V stays, the queries of all heads that share it
//             stream by: S^T = K Q^T, dP^T = V dH^T, dV += P^T dH, dK += dS^T Q
//
// Eight row warps: warp w has lanes 32 (w % 4) .. + 31 of tensor memory (one row a thread) and
// columns 64 (w / 4) .. + 63.  P^T and dS go back to tensor memory as bf16 operands, each warp's
// over columns that it has read itself.  The products are issued so that the tensor cores have
// work while the rows are between two of their steps:
//   keys      after P^T(j): dV += P^T(j) dH, S^T(j + 1)      while the rows make dS^T(j)
//             after dS^T(j): dK += dS^T(j) Q, dP^T(j + 1)    while the rows make P^T(j + 1)
//   queries   after S(j) is read: S(j + 1);  after dS(j): dQ += dS(j) K, dP(j + 1)
// (a product that overwrites an operand is issued after the one that reads it).  S, dP, dV and dK
// fill tensor memory at d = 128.  P and dS are rounded to bf16, the operands' type; S, dP, P in dS,
// and all sums are fp32.
// States from the length on: P and dS are zero there by select, and rows of K that meet a zero of dS
// are zeroed in shared memory.
#include "cross_tc.cuh"

#include <math.h>

namespace anchor {

__device__ unsigned int g_cross_bwd_error;  // bit 0: a wait gave up

namespace {

using namespace cross_tc;

constexpr int kRowWarps = 8;
constexpr int kLoad = kRowWarps, kStat = kRowWarps + 1, kIssue = kRowWarps + 2;
constexpr int kThreads = 32 * (kRowWarps + 3);
constexpr uint32_t kColS = 0, kColP = 128, kColA = 256;  // S, dP, then the sums

template <int D>
struct Geo {
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kFix = 0, kRing = 2 * kTile<D>, kStatB = kRing + kStages * kTile<D>;  // 2 x (lse, D) of 128 columns
    static constexpr int kBars = kStatB + 2 * 2 * kRows * 4;
    static constexpr int kNBars = 2 * kStages + 11;
    static constexpr int kSmem = kBars + kNBars * 8 + 16 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct BwdParams {
    CrossProblem p;
    const float *delta;
    TileMap a, b;  // queries: K, V stream; keys: Q, dH stream
    TileMap fa, fb;  // keys: K, V stay
    int tiles;
};

// An operand of 128 contraction columns in tensor memory, bf16: the two halves over the first 32 of
// their own 64 columns.
__device__ __forceinline__ uint32_t half_step(uint32_t base, int k) { return base + (k < 4 ? 8 * k : 64 + 8 * (k - 4)); }

// KEYS: see above
template <int D, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) cross_bwd_kernel(const __grid_constant__ BwdParams a) {
    using G = Geo<D>;
    constexpr int ST = G::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G::kBars);
    uint64_t *full = bars, *empty = full + ST, *fix_full = empty + ST, *s_full = fix_full + 1, *dp_full = s_full + 1,
             *p_full = dp_full + 1, *ds_full = p_full + 1, *stat_full = ds_full + 1 /* [2] */, *stat_empty = stat_full + 2 /* [2] */,
             *acc = stat_empty + 2, *done = acc + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + G::kNBars);
    float *stat = reinterpret_cast<float *>(sm + G::kStatB);
    const CrossProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = (int)(blockIdx.x % a.tiles), bk = (int)(blockIdx.x / a.tiles);
    const int b = bk / p.kv, kh = bk - b * p.kv, r0 = tile * kRows;
    unsigned int *error = &g_cross_bwd_error;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(fix_full, KEYS ? 1 : kRowWarps);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, kRowWarps);
        mbar_init(ds_full, kRowWarps);
        for (int s = 0; s < 2; ++s) {
            mbar_init(stat_full + s, 1);
            mbar_init(stat_empty + s, kRowWarps);
        }
        mbar_init(acc, 1);
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == kIssue) tmem_alloc(s_tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dependency_wait();
    grid_dependents_launch();

    const int L = cross_length(p, b);
    // steps over the tiles that stream by: keys of the entry, or the queries of each head in turn
    const int per_head = (p.n + kRows - 1) / kRows;
    const int nt = KEYS ? (r0 < L ? p.group * per_head : 0) : (L + kRows - 1) / kRows;
    // columns of step j that exist, and the same in 16s
    auto width = [&](int j) { return KEYS ? min(kRows, p.n - (j % per_head) * kRows) : min(kRows, L - j * kRows); };
    auto width16 = [&](int j) { return (width(j) + 15) / 16 * 16; };

    if (warp == kLoad) {
        if (lane == 0 && nt > 0) {
            if (KEYS) {
                mbar_arrive_expect_tx(fix_full, 2 * kTile<D>);
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    tma_load_4d(sm + G::kFix + q * kBlock, &a.fa.map, fix_full, 64 * q, r0, kh * a.fa.by_head, b * a.fa.by_batch);
                    tma_load_4d(sm + G::kFix + kTile<D> + q * kBlock, &a.fb.map, fix_full, 64 * q, r0, kh * a.fb.by_head,
                                b * a.fb.by_batch);
                }
            }
            int i = 0;
            for (; i < 2 * nt; ++i) {
                const int st = i % ST, j = i / 2;
                if (i >= ST && !bwait(empty + st, (uint32_t)((i / ST - 1) & 1), error)) break;
                const int row = (KEYS ? j % per_head : j) * kRows, head = KEYS ? kh * p.group + j / per_head : kh;
                load_tile<D>(sm + G::kRing + st * kTile<D>, i & 1 ? a.b : a.a, full + st, row, head, b);
            }
            // the CTA leaves only once its copies have landed
            for (int j = max(0, i - ST); j < i; ++j) bwait(full + j % ST, (uint32_t)((j / ST) & 1), error);
            if (KEYS) bwait(fix_full, 0u, error);
        }
        __syncwarp();
    } else if (warp == kStat) {
        if (KEYS) {  // lse (in log2) and D of each step's columns; columns that do not exist: P = 0
            bool ok = true;
            for (int j = 0; j < nt && ok; ++j) {
                if (j >= 2) ok = bwait(stat_empty + (j & 1), (uint32_t)((j / 2 - 1) & 1), error);
                if (!ok) break;
                const int i0 = (j % per_head) * kRows;
                const long long f = ((long long)b * p.heads + kh * p.group + j / per_head) * p.n + i0;
                float *dst = stat + (j & 1) * 2 * kRows;
#pragma unroll
                for (int x = 0; x < kRows; x += 32) {
                    const bool in = i0 + x + lane < p.n;
                    dst[x + lane] = in ? p.lse[f + x + lane] * kLog2e : INFINITY;
                    dst[kRows + x + lane] = in ? a.delta[f + x + lane] : 0.f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(stat_full + (j & 1));
            }
        }
        __syncwarp();
    } else if (warp == kIssue) {
        if (lane == 0 && nt > 0) {
            const int ksteps = (p.d + 15) / 16;
            const uint32_t base = smem_u32(sm), ring = base + G::kRing;
            const uint32_t idA = idesc_bf16_f32(kRows, p.d < D ? p.d : D, false, true);
            const uint64_t f0 = desc_k(base + G::kFix), f1 = desc_k(base + G::kFix + kTile<D>);
            auto landed = [&](int i) {
                const bool ok = bwait(full + i % ST, (uint32_t)((i / ST) & 1), error);
                tc_fence_after();
                return ok;
            };
            // to = (the tile that stays) x (slot i of the ring)^T
            auto across = [&](uint32_t to, uint64_t fix, int i, uint64_t *bar) {
                const uint32_t id = idesc_bf16_f32(kRows, width16(i / 2), false, false);
                const uint64_t d = desc_k(ring + (i % ST) * kTile<D>);
                for (int k = 0; k < ksteps; ++k) umma_bf16(to, fix + step_k(k), d + step_k(k), id, k > 0 ? 1u : 0u);
                umma_commit(bar);
            };
            // sum += (operand in tensor memory) x (slot i of the ring)
            auto along = [&](uint32_t sum, uint32_t op, int i) {
                const int steps = width16(i / 2) / 16;
                const uint64_t d = desc_mn(ring + (i % ST) * kTile<D>);
                for (int k = 0; k < steps; ++k)
                    umma_bf16_tmem_a(sum, half_step(op, k), d + step_mn(k), idA, (i > 1 || k > 0) ? 1u : 0u);
            };
            bool ok = bwait(fix_full, 0u, error) && landed(0);
            if (ok) {
                across(tmem + kColS, f0, 0, s_full);
                ok = landed(1);
                if (ok) across(tmem + kColP, f1, 1, dp_full);
            }
            for (int j = 0; j < nt && ok; ++j) {
                // the rows have read S(j) (and left P^T(j) over it)
                if (!(ok = bwait(p_full, (uint32_t)(j & 1), error))) break;
                tc_fence_after();
                if (KEYS) {
                    along(tmem + kColA, tmem + kColS, 2 * j + 1);  // dV += P^T dH
                    umma_commit(empty + (2 * j + 1) % ST);
                }
                if (j + 1 < nt) {
                    if (!(ok = landed(2 * j + 2))) break;
                    across(tmem + kColS, f0, 2 * j + 2, s_full);
                }
                // the rows have left dS(j) over dP(j)
                if (!(ok = bwait(ds_full, (uint32_t)(j & 1), error))) break;
                tc_fence_after();
                along(tmem + kColA + (KEYS ? D : 0), tmem + kColP, 2 * j);  // dK += dS^T Q, dQ += dS K
                umma_commit(empty + 2 * j % ST);
                if (!KEYS) umma_commit(empty + (2 * j + 1) % ST);  // V: read by dP(j), long done
                if (j + 1 < nt) {
                    if (!(ok = landed(2 * j + 3))) break;
                    across(tmem + kColP, f1, 2 * j + 3, dp_full);
                }
            }
            if (ok) umma_commit(acc);
            umma_commit(done);
            bwait(done, 0u, error);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ rows
        const int half = warp >> 2, w4 = warp & 3, row = w4 * 32 + lane, r = r0 + row;
        const bool mine = r < (KEYS ? L : p.rows);  // a row that counts
        const uint32_t trow = tmem + ((uint32_t)(w4 * 32) << 16);
        const float c = p.scale * kLog2e;
        constexpr int kLanes = D / 8;
        float lse2 = INFINITY, dl = 0.f;
        if (!KEYS && nt > 0) {
            // half 0 loads the 128 rows of Q, half 1 those of dH
            const CrossView &v = half ? p.dH : p.Q;
            const long long at = mine ? cross_row(p, v, b, kh, r) : -1;
            uint8_t *dst = sm + G::kFix + half * kTile<D>;
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const int rr = i * (32 / kLanes) + lane / kLanes, ch = lane % kLanes;
                const long long o = __shfl_sync(0xffffffffu, at, rr);
                uint4 x = make_uint4(0, 0, 0, 0);
                if (o >= 0 && ch * 8 < p.d) x = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)v.ptr + o + ch * 8);
                *reinterpret_cast<uint4 *>(dst + chunk_at(w4 * 32 + rr, ch)) = x;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(fix_full);
            if (mine) {
                const long long f = cross_flat(p, b, kh, r);
                lse2 = p.lse[f] * kLog2e;
                dl = a.delta[f];
            }
        }
        bool ok = true;
        for (int j = 0; j < nt && ok; ++j) {
            const int cols = width(j) - 64 * half;  // of this half that exist (may be none)
            const uint32_t tS = trow + kColS + 64 * half, tP = trow + kColP + 64 * half;
            const float *st = stat + (j & 1) * 2 * kRows + 64 * half;
            float e[64];
            if (!bwait(s_full, (uint32_t)(j & 1), error)) { ok = false; break; }
            if (KEYS && !bwait(stat_full + (j & 1), (uint32_t)((j / 2) & 1), error)) { ok = false; break; }
            tc_fence_after();
            tmem_ld32(tS, e);
            if (cols > 32) tmem_ld32(tS + 32, e + 32);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 64; x += 4) {
                float4 s4 = make_float4(lse2, lse2, lse2, lse2);
                if (KEYS) s4 = *reinterpret_cast<const float4 *>(st + x);
                e[x] = ex2(fmaf(e[x], c, -s4.x));
                e[x + 1] = ex2(fmaf(e[x + 1], c, -s4.y));
                e[x + 2] = ex2(fmaf(e[x + 2], c, -s4.z));
                e[x + 3] = ex2(fmaf(e[x + 3], c, -s4.w));
            }
            if (!mine || (!KEYS && cols < 64)) {
#pragma unroll
                for (int x = 0; x < 64; ++x)
                    if (!mine || x >= cols) e[x] = 0.f;
            }
            if (KEYS) {
                uint32_t u[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) u[x] = pack2(e[2 * x], e[2 * x + 1]);
                tmem_st32(tS, u);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            // dS
            if (!bwait(dp_full, (uint32_t)(j & 1), error)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float g[32];
                uint32_t u[16];
                if (x == 1 && cols <= 32) break;
                tmem_ld32(tP + 32 * x, g);
                tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 32; y += 4) {
                    float4 d4 = make_float4(dl, dl, dl, dl);
                    if (KEYS) d4 = *reinterpret_cast<const float4 *>(st + kRows + 32 * x + y);
                    const float *q = e + 32 * x + y;
                    g[y] = q[0] * (g[y] - d4.x);
                    g[y + 1] = q[1] * (g[y + 1] - d4.y);
                    g[y + 2] = q[2] * (g[y + 2] - d4.z);
                    g[y + 3] = q[3] * (g[y + 3] - d4.w);
                }
                // (a masked state's dP may be anything: zero by select, not by the product)
                if (!mine || (!KEYS && cols < 64)) {
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (!mine || 32 * x + y >= cols) g[y] = 0.f;
                }
#pragma unroll
                for (int y = 0; y < 16; ++y) u[y] = pack2(g[2 * y], g[2 * y + 1]);
                tmem_st16(tP + 16 * x, u);
            }
            tmem_st_wait();
            if (!KEYS && j == nt - 1 && half == 0 && L % kRows && L < p.s) {
                // the last tile's rows of K that do not count (S has read them)
                if (!bwait(full + 2 * j % ST, (uint32_t)((2 * j / ST) & 1), error)) { ok = false; break; }
                zero_rows<D>(sm + G::kRing + (2 * j % ST) * kTile<D>, row, L % kRows, (L % kRows + 15) / 16 * 16);
                fence_proxy_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (KEYS) mbar_arrive(stat_empty + (j & 1));
                mbar_arrive(ds_full);
            }
        }
        if (ok && nt > 0) ok = bwait(acc, 0u, error);
        tc_fence_after();
        // rows out through shared memory (the tiles that stayed are not needed any more): keys: half 0
        // dV, half 1 dK; queries: each half its columns of dQ
        const bool second = KEYS && half == 1;
        const float by = KEYS && half == 0 ? 1.f : p.scale;
        uint8_t *stage = sm + G::kFix + (second ? kTile<D> : 0);
        const int from = KEYS ? 0 : half * (D / 2), to = KEYS ? D : from + D / 2;
        if (ok) {
#pragma unroll 1
            for (int x = from; x < to && x < p.d; x += 32) {
                float o[32];
                if (nt > 0) {
                    tmem_ld32(trow + kColA + (second ? D : 0) + x, o);
                    tmem_ld_wait();
                }
                const bool some = nt > 0 && mine;
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
            const bool exists = r < (KEYS ? p.s : p.rows);
            const long long at = !exists ? -1 : KEYS ? b * v.sb + kh * v.sh + (long long)r * v.sn : cross_row(p, v, b, kh, r);
            // 16-byte chunks of this warp's rows and columns, a row's chunks by neighbouring lanes
            constexpr int kW = KEYS ? D / 8 : D / 16;
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                const int rr = i * (32 / kW) + lane / kW, ch = from / 8 + lane % kW;
                const long long o = __shfl_sync(0xffffffffu, at, rr);
                if (o >= 0 && ch * 8 < p.d)
                    *reinterpret_cast<uint4 *>((__nv_bfloat16 *)v.ptr + o + ch * 8) =
                        *reinterpret_cast<const uint4 *>(stage + chunk_at(w4 * 32 + rr, ch));
            }
        }
        tc_fence_before();
        __syncwarp();
    }
    __syncthreads();
    if (warp == kIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool KEYS>
cudaError_t launch(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    using G = Geo<D>;
    BwdParams a;
    a.p = p;
    a.delta = delta;
    a.tiles = ((KEYS ? p.s : p.rows) + kRows - 1) / kRows;
    TileMap k, v, q, g;
    if (p.s > 0 && (!make_tile_map(&k, p.K, p.B, p.kv, p.s, p.d) || !make_tile_map(&v, p.V, p.B, p.kv, p.s, p.d)))
        return cudaErrorInvalidValue;
    if (KEYS && p.n > 0 && (!make_tile_map(&q, p.Q, p.B, p.heads, p.n, p.d) || !make_tile_map(&g, p.dH, p.B, p.heads, p.n, p.d)))
        return cudaErrorInvalidValue;
    a.a = KEYS ? q : k, a.b = KEYS ? g : v, a.fa = k, a.fb = v;
    const cudaError_t e = cudaFuncSetAttribute(cross_bwd_kernel<D, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_bwd_kernel<D, KEYS>, dim3(a.tiles * p.B * p.kv), dim3(kThreads), G::kSmem, stream, a);
}

template <int D>
cudaError_t backward(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    cudaError_t e = p.rows > 0 ? launch<D, false>(p, delta, stream) : cudaSuccess;
    if (e == cudaSuccess && p.s > 0) e = launch<D, true>(p, delta, stream);
    return e;
}

}  // namespace

cudaError_t launch_cross_tc_backward(const CrossProblem &p, const float *delta, cudaStream_t stream) {
    return p.d > 64 ? backward<128>(p, delta, stream) : backward<64>(p, delta, stream);
}

cudaError_t cross_bwd_read_and_clear_error(unsigned *out) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_cross_bwd_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_cross_bwd_error, &zero, sizeof(unsigned));
}

}  // namespace anchor
