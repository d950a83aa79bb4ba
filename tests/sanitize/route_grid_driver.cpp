// Drives the routed entry points (include/qroute.h) with sizes around their limits, the
// kernel launchers replaced by stubs that compute the launch's grid as the real ones
// do (route_grid.hpp): no accepted call may take 2^32 work items or more in one
// launch, and sizes on both sides of a limit get the right code.  Pointers are addresses
// that nothing reads.  Exits non-zero on the first mismatch.
#include <stdint.h>
#include <stdio.h>

#include "launch_route.hpp"
#include "qroute.h"

static int g_fail = 0, g_launches = 0;
static int64_t g_most = 0;

static hipError_t items(const char* what, int64_t n, int64_t a, int64_t b, int64_t c) {
  ++g_launches;
  if (n > g_most) g_most = n;
  if (n < 1 || n >= (int64_t(1) << 32)) {
    fprintf(stderr, "%s(%lld, %lld, %lld): %lld work items\n", what, (long long)a, (long long)b, (long long)c, (long long)n);
    g_fail = 1;
  }
  return hipSuccess;
}

namespace qgemv {

int64_t route_sort_workspace(int64_t, int64_t) { return 0; }
hipError_t launch_route_sort(const int32_t*, int64_t, int64_t, int32_t*, int32_t*, int32_t*, void*, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_route_gather(const void*, const int32_t*, const float*, void*, int, int64_t t, int64_t k, int64_t c,
                               hipStream_t) {
  return items("gather", route_move_workgroups(t * k, c) * kRouteMoveThreads, t, k, c);
}
hipError_t launch_route_combine(const void*, int, const int32_t*, const float*, void*, int, int64_t t, int64_t k, int64_t c,
                                hipStream_t) {
  return items("combine", route_move_workgroups(t, c) * kRouteMoveThreads, t, k, c);
}
hipError_t launch_route_combine_grad(const void*, int, const void*, int, const int32_t*, const float*, void*, float*,
                                     int64_t t, int64_t k, int64_t c, hipStream_t) {
  return items("combine_grad", route_grad_workgroups(t, c) * kRouteMoveThreads, t, k, c);
}
hipError_t launch_routed(int fmt, const void*, const void*, const int32_t*, const int32_t*, void*, int, int64_t t,
                         int64_t choices, int64_t e, int64_t m, int64_t, int64_t, hipStream_t) {
  return items("product", routed_work_items(routed_plan(fmt, t * choices, e, m)), t * choices, m, e);
}
int64_t lora_workspace(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }
hipError_t launch_lora(bool, const void*, const void*, const void*, const float*, const int32_t*, const int32_t*,
                       const void*, void*, int, int64_t, int64_t, int64_t, int64_t, int64_t, void*, hipStream_t) {
  return hipSuccess;
}

}  // namespace qgemv

// address i, far from the others (a call's arrays reach at most 2^59 bytes)
template <typename T = void>
static T* at(int i) {
  return reinterpret_cast<T*>(uintptr_t(i + 1) << 60);
}

static int gather(int64_t t, int64_t k, int64_t c) {
  return qroute_gather(at(0), at<int32_t>(1), nullptr, at(3), 1, t, k, c, nullptr);
}
static int combine(int64_t t, int64_t k, int64_t c) {
  return qroute_combine(at(0), 1, at<int32_t>(1), at<float>(2), at(3), 0, t, k, c, nullptr);
}
static int grad(int64_t t, int64_t k, int64_t c) {
  return qroute_combine_grad(at(0), 0, at(1), 1, at<int32_t>(2), at<float>(3), at(4), at<float>(5), t, k, c, nullptr);
}
static int product(int fmt, int64_t n, int64_t e, int64_t m, int64_t k) {
  auto* const f = fmt == 0 ? qgemm_q4k_routed : fmt == 1 ? qgemm_nvfp4_routed : qgemm_tq1_routed;
  return f(at(0), at(2), nullptr, at<int32_t>(3), at(4), 0, n, 1, e, m, k, nullptr);
}

static void expect(const char* what, int got, int want) {
  if (got != want) {
    fprintf(stderr, "%s -> %d, not %d\n", what, got, want);
    g_fail = 1;
  }
}

int main() {
  // the row movers' limit T*k*(C + 16) <= 2^35, from both sides, for every number of rows
  for (int r = 0; r <= 24; ++r)
    for (int64_t rows : {(int64_t(1) << r) - 1, int64_t(1) << r, (int64_t(1) << r) + 1})
      for (int64_t k : {int64_t(1), int64_t(3), int64_t(64)}) {
        const int64_t t = rows / k;
        if (t < 1 || t * k > QROUTE_MAX_N) continue;
        const int64_t most = (int64_t(1) << 35) / (t * k) - 16;  // the largest C
        for (int64_t c = most - 9; c <= most + 9; ++c) {
          const int want = c <= most && c <= (1 << 24) ? QGEMV_OK : QGEMV_E_SHAPE;
          if (c < 1) continue;
          expect("gather", gather(t, k, c), want);
          expect("combine", combine(t, k, c), want);
          expect("combine_grad", grad(t, k, c), want);
        }
        for (int64_t c : {1, 8, 1024, 1025, 2032, 1 << 24}) {
          const int want = t * k * (c + 16) <= int64_t(1) << 35 ? QGEMV_OK : QGEMV_E_SHAPE;
          expect("gather", gather(t, k, c), want);
          expect("combine", combine(t, k, c), want);
          expect("combine_grad", grad(t, k, c), want);
        }
      }
  // products: none is refused that the header promises, and none accepted that a launch
  // cannot take (the stub's check)
  int refused = 0;
  for (int fmt = 0; fmt < 3; ++fmt)
    for (int nb = 0; nb <= 24; ++nb)
      for (int64_t n : {int64_t(1) << nb, int64_t(3) << nb, (int64_t(1) << nb) + 5})
        for (int64_t e : {1, 2, 7, 64, 1000, 1024})
          for (int mb = 0; mb <= 24; ++mb)
            for (int64_t m : {(int64_t(1) << mb) - 1, int64_t(1) << mb, (int64_t(5) << mb) / 4 + 3})
              for (int64_t k : {256, 4096, 16384, 1 << 20}) {
                if (n > QROUTE_MAX_N || m < 1 || m > (1 << 24)) continue;
                const int rc = product(fmt, n, e, m, k);
                const int64_t used = n < e ? n : e;
                if ((m + 63) / 64 * (n / 16 + used) < (1 << 23)) expect("product", rc, QGEMV_OK);
                if (rc != QGEMV_OK) {
                  expect("product", rc, QGEMV_E_SHAPE);
                  ++refused;
                }
              }
  if (refused == 0 || g_launches == 0 || g_most < (int64_t(1) << 32) - (int64_t(1) << 24)) {
    fprintf(stderr, "the limits were not reached: %d refused, %d launches, at most %lld items\n", refused, g_launches,
            (long long)g_most);
    g_fail = 1;
  }
  if (!g_fail) printf("route grids: ok\n");
  return g_fail;
}
