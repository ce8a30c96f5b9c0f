// What the tensor-core kernels of cross attention share: bounded waits, 4-D tile loads, tiles in
// swizzled shared memory, descriptors.
//
// A tile is 128 rows (tiles that stream by also 64, at 64 columns) of 64 or 128 bf16 columns, in blocks of 64 columns: [128 rows][128 bytes]
// with the 128-byte swizzle (16-byte chunk c of row r at c ^ (r & 7)), as a TMA box lands.  One
// copy serves as a K-major operand (contraction over the columns) and as an MN-major one
// (contraction over the rows).  Heads of 16 and 32 columns are tiles of 64 whose other columns
// are not read.
#pragma once

#include "cross.cuh"
#include "ptx.cuh"

namespace anchor {
namespace cross_tc {

using namespace ptx;

constexpr int kRows = 128;
constexpr int kBlock = kRows * 128;  // bytes of a 64-column block
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int rows = kRows> constexpr int kTile = rows * D * 2;

// A view as a tensor map (d, rows, heads, batch): an axis that does not move (a stride of 0, or
// one entry) is an axis of one entry whose coordinate is multiplied by 0.
struct TileMap {
    CUtensorMap map;
    int by_head, by_batch;
};
bool make_tile_map(TileMap *m, const CrossView &v, int B, int heads, int rows, int d, int box_rows);

// bit 0 of the error word, and false, once a wait has lasted kWaitNs.  (In line: a call in the loops
// that wait costs them their registers, 62 -> 69 us in the forward of 8 heads, 9728 x 2048.)
__device__ __forceinline__ bool bwait(uint64_t *bar, uint32_t parity, unsigned int *error) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 2000)) {
        if (globaltimer_ns() - t0 > kWaitNs) {
            atomicOr(error, 1u);
            return false;
        }
    }
    return true;
}

// whether a phase is complete, without waiting
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
// a box into L2, nothing else
__device__ __forceinline__ void prefetch_tile(const CUtensorMap *map, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"((uint64_t)map), "r"(c0), "r"(c1),
                 "r"(c2), "r"(c3)
                 : "memory");
}
// a tile's rows from `row` on, of one head, in boxes of `box` rows; rows and columns outside the tensor
// are zero.  The caller has announced the bytes on `bar`.
template <int D, int rows, int box>
__device__ __forceinline__ void load_tile(uint8_t *dst, const TileMap &m, uint64_t *bar, int row, int head, int b) {
    static_assert(rows == kRows || D == 64, "a tile of more than one block has 128 rows");
#pragma unroll
    for (int q = 0; q < D / 64; ++q)
#pragma unroll
        for (int r = 0; r < rows; r += box)
            tma_load_4d(dst + q * kBlock + r * 128, &m.map, bar, 64 * q, row + r, head * m.by_head, b * m.by_batch);
}

// A warp's 32 rows of a view, `lanes` lanes of 16 bytes a row: calls f(i, row of the warp, offset of
// the row in the view, or -1) for its 32 / lanes rows of each of `lanes` passes.  `at`: the offset of
// this lane's own row.  Rows that follow one another (all but those around the end of a head) are
// addressed by their step, others by asking the lane that has them.
template <int lanes, typename F>
__device__ __forceinline__ void each_row(long long at, long long step, F f) {
    const int lane = threadIdx.x & 31, first = lane / lanes;
    const long long base = __shfl_sync(0xffffffffu, at, 0);
    if (__all_sync(0xffffffffu, base >= 0 && at == base + lane * step)) {
        long long o = base + first * step;
#pragma unroll
        for (int i = 0; i < lanes; ++i, o += (32 / lanes) * step) f(i, i * (32 / lanes) + first, o);
    } else {
#pragma unroll
        for (int i = 0; i < lanes; ++i) {
            const int row = i * (32 / lanes) + first;
            f(i, row, __shfl_sync(0xffffffffu, at, row));
        }
    }
}

// byte offset of 16-byte chunk c of row r
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (uint32_t)((c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// descriptors of a tile, and their advance for step k of 16 along the contraction
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return smem_desc_sw128(tile, 16, 1024); }        // over columns
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile) { return smem_desc_sw128(tile, kBlock, 1024); }   // over rows
__device__ __forceinline__ uint64_t step_k(int k) { return (uint64_t)(((k >> 2) * kBlock + (k & 3) * 32) >> 4); }
__device__ __forceinline__ uint64_t step_mn(int k) { return (uint64_t)(k * 16 * 128 >> 4); }

// Products issued by one thread.  A loop of known length is issued without a pause (descriptors
// in registers ahead of time); with a length that is read at run time each product waited on the
// address arithmetic of its own (128 cycles where the tensor pipe takes 64), so the common length
// has a loop of its own.
// to = A B^T: both tiles in shared memory, over `steps` 16s of their columns.  `meanwhile` runs
// behind the second product: the tensor pipe holds about two, so what takes the thread a hundred
// cycles costs nothing there.
template <int D, typename F>
__device__ __forceinline__ void product_k(uint32_t to, uint64_t a, uint64_t b, uint32_t id, int steps, F meanwhile) {
    if (steps == D / 16) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            umma_bf16(to, a + step_k(k), b + step_k(k), id, k > 0 ? 1u : 0u);
            if (k == 1) meanwhile();
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < steps; ++k) umma_bf16(to, a + step_k(k), b + step_k(k), id, k > 0 ? 1u : 0u);
        meanwhile();
    }
}
// sum (+)= A B: A bf16 in tensor memory, its columns in runs of 2 R (R columns of 32 bits, at the
// start of their own 2 R columns), B over `steps` 16s of its rows
template <int R, int rows>
__device__ __forceinline__ void product_mn(uint32_t sum, uint32_t a, uint64_t b, uint32_t id, int steps, bool add) {
    auto at = [&](int k) { return a + (uint32_t)(8 * k / R * 2 * R + 8 * k % R); };
    if (steps == rows / 16) {
#pragma unroll
        for (int k = 0; k < rows / 16; ++k) umma_bf16_tmem_a(sum, at(k), b + step_mn(k), id, k > 0 || add ? 1u : 0u);
    } else {
#pragma unroll 1
        for (int k = 0; k < steps; ++k) umma_bf16_tmem_a(sum, at(k), b + step_mn(k), id, k > 0 || add ? 1u : 0u);
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 columns of a warp's 32 lanes, for paths that have few registers to spare
__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// zeros in rows [from, to) of a tile, one row per thread t of 128
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int t, int from, int to) {
    if (t < from || t >= to) return;
#pragma unroll
    for (int q = 0; q < D / 64; ++q)
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(tile + q * kBlock + t * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
}

}  // namespace cross_tc
}  // namespace anchor
