// Helpers shared by the host runtime files: error reporting, the device guard
// of an API call, the allocation hook and the timing ring.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "ctx.h"

namespace scute {

inline scute_status fail(scute_ctx *c, scute_status s, const char *fmt, ...) {
    if (c) {
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(c->err, sizeof(c->err), fmt, ap);
        va_end(ap);
    }
    return s;
}

#define CU_TRY(ctx, expr)                                                                      \
    do {                                                                                       \
        cudaError_t _e = (expr);                                                               \
        if (_e != cudaSuccess) {                                                               \
            (void)cudaGetLastError();                                                          \
            if (_e == cudaErrorMemoryAllocation)                                               \
                return fail(ctx, SCUTE_ERR_OOM, "%s: %s", #expr, cudaGetErrorString(_e));      \
            return fail(ctx, SCUTE_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(_e));         \
        }                                                                                      \
    } while (0)

// Keeps the context's device current for the duration of one API call.
struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) {
            if (cudaSetDevice(dev) == cudaSuccess) changed = true;
        }
    }
    ~DeviceGuard() {
        if (changed) cudaSetDevice(prev);
    }
};

// Device allocation of the library (counts for scute_debug_fail_alloc).
cudaError_t dev_malloc(void **p, size_t bytes);

inline void count_launch(scute_ctx *c, int k) { c->launches += k; }

// Timing ring (scute_timing_*): while enabled, every launch (or launch pair)
// of the hot path is bracketed by an event pair on its stream, tagged with its
// kind.  Event records made while the stream is being captured become graph
// nodes, re-recorded on every replay.
struct TimedLaunch {
    scute_ctx *c;
    cudaStream_t st;
    int slot = -1;
    unsigned flags = cudaEventRecordDefault;
    cudaError_t begin() {
        if (!c->timing) return cudaSuccess;
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        cudaError_t e = cudaStreamIsCapturing(st, &cs);
        if (e != cudaSuccess) return e;
        if (cs == cudaStreamCaptureStatusActive) flags = cudaEventRecordExternal;
        slot = c->t_next;
        return cudaEventRecordWithFlags(c->ev[slot][0], st, flags);
    }
    cudaError_t end(int kind) {
        if (!c->timing || slot < 0) return cudaSuccess;
        const cudaError_t e = cudaEventRecordWithFlags(c->ev[slot][1], st, flags);
        c->ev_kind[slot] = kind;
        c->t_next = (slot + 1) % SCUTE_TIMING_SLOTS;
        if (c->t_used < SCUTE_TIMING_SLOTS) ++c->t_used;
        slot = -1;
        return e;
    }
};

}  // namespace scute
