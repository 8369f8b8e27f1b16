// Host helpers shared by the files that define the C entry points (muon_api.hip,
// train_api.hip): error reporting, the device check and per-launch timing.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "muon.h"

namespace muon {

// Set the calling thread's error message and return the status.
muon_status fail(muon_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
muon_status hip_fail(hipError_t e, const char* what);
void clear_error();

// Current device and its number of compute units; an error unless it is gfx950.
muon_status check_device(int* dev_out, int* cu_count);

constexpr size_t ALIGN = 256;
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Events around one launch, recorded while profiling is enabled.
struct ProfMark {
    hipEvent_t a = nullptr, b = nullptr;
};
ProfMark prof_begin(hipStream_t s);
void prof_end(int cls, const ProfMark& mark, hipStream_t s);

template <typename F>
muon_status timed_launch(int cls, hipStream_t s, const char* what, F launch) {
    const ProfMark mark = prof_begin(s);
    const hipError_t e = launch();
    if (e != hipSuccess) return hip_fail(e, what);
    prof_end(cls, mark, s);
    return MUON_OK;
}

}  // namespace muon
