// Host-side launchers of the routed kernels (include/qroute.h).  Arguments are
// validated by the C-ABI layer before these are called; each enqueues on `s`
// and returns the HIP status of the launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "route_grid.hpp"

namespace qgemv {

int64_t route_sort_workspace(int64_t n, int64_t e);
hipError_t launch_route_sort(const int32_t* ids, int64_t n, int64_t e, int32_t* order, int32_t* position,
                             int32_t* offsets, void* ws, hipStream_t s);
hipError_t launch_route_gather(const void* x, const int32_t* order, const float* weights, void* out, int dtype,
                               int64_t t, int64_t k, int64_t c, hipStream_t s);
hipError_t launch_route_combine(const void* rows, int rows_dtype, const int32_t* position, const float* weights,
                                void* y, int y_dtype, int64_t t, int64_t k, int64_t c, hipStream_t s);
hipError_t launch_route_combine_grad(const void* dy, int dy_dtype, const void* rows, int rows_dtype,
                                     const int32_t* position, const float* weights, void* drows, float* dweights,
                                     int64_t t, int64_t k, int64_t c, hipStream_t s);

// Largest span of the activations that a plan's rows are picked from.
constexpr int64_t kRouteMaxXBytes = int64_t(1) << 30;
hipError_t launch_routed(int fmt, const void* w, const void* x, const int32_t* order, const int32_t* offsets, void* y,
                         int y_dtype, int64_t t, int64_t choices, int64_t e, int64_t m, int64_t k,
                         int64_t expert_bytes, hipStream_t s);

// Low-rank adapters: y = c + scale (x A^T) B^T by the plan's rows.
int64_t lora_workspace(int64_t t, int64_t e, int64_t r, int64_t m, int64_t k);
hipError_t launch_lora(bool bf16, const void* x, const void* a, const void* b, const float* scale,
                       const int32_t* order, const int32_t* offsets, const void* c, void* y, int y_dtype, int64_t t,
                       int64_t e, int64_t r, int64_t m, int64_t k, void* ws, hipStream_t s);

}  // namespace qgemv
