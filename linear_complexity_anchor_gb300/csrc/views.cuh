// Strided [B][heads][n][d] views of the C ABI: their checks on the host, and the stream-ordered
// workspaces of the calls that take them.
#pragma once

#include "common.cuh"

#include <atomic>

namespace anchor {

// a view with its sizes
struct View {
    const char *ptr = nullptr;
    long long sb = 0, sh = 0, sn = 0;  // strides in elements
    long long B = 0, H = 0, N = 0;
    int d = 0, es = 0;

    long long extent() const { return ((B - 1) * sb + (H - 1) * sh + (N - 1) * sn + d) * es; }  // bytes, first to last
    bool same(const View &o) const {
        return ptr == o.ptr && B == o.B && H == o.H && N == o.N && d == o.d && es == o.es && (B < 2 || sb == o.sb) &&
               (H < 2 || sh == o.sh) && (N < 2 || sn == o.sn);
    }
};

View make_view(const anchor_attn_view_t &v, int B, int heads, int n, int d, int es);
// pointer and strides as the ABI asks; `writes`: no two rows share an element
anchor_attn_status_t check_view(const View &v, bool writes);
bool views_overlap(const View &a, const View &b);
inline bool bytes_overlap(const void *a, size_t an, const void *b, size_t bn) {
    return (uintptr_t)a < (uintptr_t)b + bn && (uintptr_t)b < (uintptr_t)a + an;
}

// Stream-ordered device memory from a pool of this library, one per device, that keeps up to
// kPoolKeep bytes between calls: the device's default pool gives its memory back at every
// synchronisation, and a call after one maps it again (one query of 32 heads over 65536 states, waited
// for: 66 us against 249; a backward of 8 x 12 heads, 1000 x 1000: 167 against 369).
constexpr unsigned long long kPoolKeep = 512ull << 20;
cudaError_t workspace_alloc(void **ptr, size_t bytes, cudaStream_t stream);
// what the current device's pool keeps goes back to the device
cudaError_t workspace_release();

// Allows a kernel `bytes` of dynamic shared memory, once per device (one object for each kernel).
struct SmemOnce {
    std::atomic<unsigned long long> done{0};  // bit: device
    template <typename Kernel> cudaError_t operator()(Kernel kernel, size_t bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

}  // namespace anchor
