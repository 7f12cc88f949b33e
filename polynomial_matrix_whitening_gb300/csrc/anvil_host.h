// anvil_host.h -- what the C ABI's translation units share on the host: the per-device
// set-up, CUDA error texts, launch profiling and the overlap checks (internal to libanvil).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "../../include/anvil.h"

namespace anvil {

// Keeps the text for anvil_last_cuda_error (per thread).
void set_error_text(const char* text);
anvil_status cuda_fail(cudaError_t e, const char* where);

struct DeviceState {
    bool ready = false;
    unsigned* err = nullptr;
    int sm_count = 0;
};
// Checks the device is sm_103, sets kernel attributes, finds the error word and the
// tensor-map encoder.  Once per device; no allocation, no synchronisation.
anvil_status device_setup(DeviceState** out);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
extern EncodeTiledFn g_encode;  // set by device_setup

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Range {
    uintptr_t lo, hi;
};
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Whether every row of a matrix (ld elements of es bytes apart) starts on a 16-byte boundary.
inline bool aligned16(const void* p, int64_t ld, int es, int64_t rows) {
    return !(reinterpret_cast<uintptr_t>(p) & 15) && (rows <= 1 || (ld * es) % 16 == 0);
}

// ---------------------------------------------------------------- launch profiling
struct Profiler {
    std::mutex mu;
    bool active = false;
    int cap = 0, used = 0;
    cudaEvent_t* ev = nullptr;  // 2 * cap events
    int* kind = nullptr;
};
extern Profiler g_prof;

// Runs `launch`, bracketed by two events on `stream` when profiling is on.  A timed
// launch holds the profiler's lock throughout, so anvil_profile_end on another thread
// cannot destroy its events in between.
template <class F>
cudaError_t profiled(int kind, cudaStream_t stream, F&& launch) {
    std::unique_lock<std::mutex> lock(g_prof.mu);
    if (!g_prof.active || g_prof.used >= g_prof.cap) {
        lock.unlock();
        return launch();
    }
    const int slot = g_prof.used++;
    g_prof.kind[slot] = kind;
    cudaError_t e;
    if ((e = cudaEventRecord(g_prof.ev[2 * slot], stream))) return e;
    if ((e = launch())) return e;
    return cudaEventRecord(g_prof.ev[2 * slot + 1], stream);
}

}  // namespace anvil
