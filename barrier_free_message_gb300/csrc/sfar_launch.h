// sfar_launch.h -- what the host code of the paged caches' operators shares:
// checks of arguments, the launch, a handle's status.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <new>

#include "sfar.h"
#include "sfar_internal.h"

static inline size_t ceil_div(size_t x, size_t a) { return (x + a - 1) / a; }
static inline bool aligned(const void *p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }

struct Span {
    uintptr_t lo, hi;
    Span(const void *p, size_t bytes) : lo((uintptr_t)p), hi((uintptr_t)p + bytes) {}
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// Launches f as a programmatic dependent of the kernel before it on the
// stream (every kernel here begins with griddepcontrol.wait); plain: without.
static inline sfar_status launch(int dev, const void *f, dim3 grid, unsigned threads, size_t smem, void *args, sfar_stream_t s, bool plain = false,
                   unsigned cluster = 1)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)s;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (!plain) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    void *params[] = {args};
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != dev)
        cudaSetDevice(dev);
    const cudaError_t err = cudaLaunchKernelExC(&cfg, f, params);
    if (cur != dev && cur >= 0)
        cudaSetDevice(cur);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return SFAR_ERR_CUDA;
    }
    return SFAR_OK;
}

// The new block of a handle's status: nothing recorded, waits of a second.
static inline SfarCtl fresh_ctl()
{
    SfarCtl c;
    memset(&c, 0, sizeof c);
    c.timeout_ns = 1000000000ull;
    c.strag_rank = c.drop_rank = -1;
    c.f_rank = c.f_cta = c.f_peer = -1;
    return c;
}
// What a handle's status block on the device says, through its pinned copy and stream.
static inline sfar_status read_ctl(const SfarCtl *ctl, SfarCtl *host, cudaStream_t s, sfar_fault *info)
{
    if (cudaMemcpyAsync(host, ctl, 32, cudaMemcpyDeviceToHost, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return SFAR_ERR_CUDA;
    }
    const sfar_status code = (sfar_status)host->status;
    if (info) {
        info->code = code;
        info->rank = code ? host->f_rank : -1;
        info->cta = code ? host->f_cta : -1;
        info->peer = code ? host->f_peer : -1;
        info->epoch = code ? host->f_epoch : 0;
        info->where = code ? host->f_where : 0;
    }
    return code;
}

// Puts a timeout into a handle's status and 1 into its n counters, as a call that gave up may leave them.
static inline sfar_status record_failure(SfarCtl *ctl, int *counters, size_t n)
{
    SfarCtl c;
    std::unique_ptr<int[]> ones(new (std::nothrow) int[n]);
    if (!ones)
        return SFAR_ERR_OOM;
    std::fill_n(ones.get(), n, 1);
    if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(&c, ctl, sizeof c, cudaMemcpyDeviceToHost) != cudaSuccess)
        return SFAR_ERR_CUDA;
    c.status = SFAR_ERR_TIMEOUT;
    c.f_where = SFAR_WAIT_COPY;
    if (cudaMemcpy(ctl, &c, sizeof c, cudaMemcpyHostToDevice) != cudaSuccess ||
        cudaMemcpy(counters, ones.get(), n * sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
        return SFAR_ERR_CUDA;
    return SFAR_OK;
}

// The plan of a step over a pool of pages, for any handle that has one (sfar_kv_host.cu).
struct SfarPool {
    int dev, shift;
    size_t pages;
    SfarCtl *ctl;
    unsigned plan_ctas;                 // of a large plan's cluster
};
sfar_status sfar_pool_plan(const SfarPool &h, const int32_t *lens, const int32_t *delta, int32_t *table, int32_t *ring,
                           const int32_t *state, int32_t *lens_out, int32_t *state_out, int32_t *starts, int32_t *slots,
                           int32_t *taken, size_t requests, size_t table_width, size_t tokens, sfar_stream_t s);
// What the plan's kernel needs of the current device; false: it failed.
bool sfar_pool_prepare(unsigned *plan_ctas);
