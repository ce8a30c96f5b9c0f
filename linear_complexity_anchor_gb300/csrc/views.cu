// Checks of strided views and the workspace pool (see views.cuh).
#include "views.cuh"

#include <algorithm>
#include <mutex>

namespace anchor {

View make_view(const anchor_attn_view_t &v, int B, int heads, int n, int d, int es) {
    View r;
    r.ptr = (const char *)v.ptr;
    r.B = B, r.H = heads, r.N = n, r.d = d, r.es = es;
    r.sb = B > 1 ? v.batch : 0;
    r.sh = heads > 1 ? v.head : 0;
    r.sn = n > 1 ? v.row : 0;
    return r;
}

anchor_attn_status_t check_view(const View &v, bool writes) {
    if (!v.ptr || ((uintptr_t)v.ptr & 15u)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    const long long strides[3] = {v.sb, v.sh, v.sn}, sizes[3] = {v.B, v.H, v.N};
    long long room = (1LL << 60) / v.es;  // elements the view may span
    for (int i = 0; i < 3; ++i) {
        if (strides[i] < 0 || (strides[i] * v.es) % 16 != 0 || strides[i] > (1LL << 39) / v.es)
            return ANCHOR_ATTN_ERR_INVALID_ARG;
        if (strides[i] > 0 && sizes[i] - 1 > room / strides[i]) return ANCHOR_ATTN_ERR_INVALID_ARG;
        room -= (sizes[i] - 1) * strides[i];
    }
    if (room < v.d || (v.N > 1 && v.sn < v.d)) return ANCHOR_ATTN_ERR_INVALID_ARG;
    if (writes) {  // by growing stride, each axis steps over all that the ones before it span
        int order[3] = {0, 1, 2};
        std::sort(order, order + 3, [&](int a, int b) { return strides[a] < strides[b]; });
        long long span = v.d;
        for (int i : order) {
            if (sizes[i] < 2) continue;
            if (strides[i] < span) return ANCHOR_ATTN_ERR_INVALID_ARG;
            span += strides[i] * (sizes[i] - 1);
        }
    }
    return ANCHOR_ATTN_OK;
}

bool views_overlap(const View &a, const View &b) {
    if (!bytes_overlap(a.ptr, (size_t)a.extent(), b.ptr, (size_t)b.extent())) return false;
    // Parts of one buffer (queries, keys and values of one projection, in any order of the axes): with a
    // cell of `c` elements, if every stride of both that is not below c is a multiple of it, every row of
    // either lies within a fixed part of a cell, and the two parts may be apart.
    if (a.es != b.es) return true;
    const long long strides[6] = {a.sb, a.sh, a.sn, b.sb, b.sh, b.sn};
    for (long long c : strides) {
        if (c <= 0) continue;
        auto part = [&](const View &v) {  // elements of a cell that a row and its neighbours take; -1: no fixed part
            const long long st[3] = {v.sb, v.sh, v.sn}, sizes[3] = {v.B, v.H, v.N};
            long long span = v.d;
            for (int i = 0; i < 3; ++i) {
                if (sizes[i] < 2 || st[i] == 0) continue;
                if (st[i] < c) span += (sizes[i] - 1) * st[i];
                else if (st[i] % c) return -1LL;
            }
            return span;
        };
        const long long na = part(a), nb = part(b);
        if (na < 0 || nb < 0) continue;
        const long long delta = ((b.ptr - a.ptr) / a.es % c + c) % c;
        if (delta >= na && delta + nb <= c) return false;
    }
    return true;
}

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_pool_lock;
cudaMemPool_t g_pools[kMaxDevices] = {};
}  // namespace

cudaError_t workspace_alloc(void **ptr, size_t bytes, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaMemPool_t pool = nullptr;
    if (dev < kMaxDevices) {
        std::lock_guard<std::mutex> hold(g_pool_lock);
        if (!g_pools[dev]) {  // not made while a stream is captured: that call takes the default pool
            cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
            if (cudaStreamIsCapturing(stream, &cap) == cudaSuccess && cap == cudaStreamCaptureStatusNone) {
                cudaMemPoolProps props = {};
                props.allocType = cudaMemAllocationTypePinned;
                props.location.type = cudaMemLocationTypeDevice;
                props.location.id = dev;
                unsigned long long keep = kPoolKeep;
                if (cudaMemPoolCreate(&g_pools[dev], &props) != cudaSuccess) {
                    g_pools[dev] = nullptr;
                } else {
                    cudaMemPoolSetAttribute(g_pools[dev], cudaMemPoolAttrReleaseThreshold, &keep);
                }
            }
            cudaGetLastError();
        }
        pool = g_pools[dev];
    }
    return pool ? cudaMallocFromPoolAsync(ptr, bytes, pool, stream) : cudaMallocAsync(ptr, bytes, stream);
}

cudaError_t workspace_release() {
    std::lock_guard<std::mutex> hold(g_pool_lock);
    if (std::all_of(g_pools, g_pools + kMaxDevices, [](cudaMemPool_t p) { return p == nullptr; })) return cudaSuccess;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return dev < kMaxDevices && g_pools[dev] ? cudaMemPoolTrimTo(g_pools[dev], 0) : cudaSuccess;
}

}  // namespace anchor
