// C ABI of the routed calls: argument validation in plain host code, then the
// launches on the caller's stream.  See include/qroute.h for the contract.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "abi_checks.hpp"
#include "launch_route.hpp"
#include "qroute.h"

namespace {

using namespace qgemv;

// T tokens of k choices
int check_slots(int64_t t, int64_t k) {
  if (t < 0 || k < 1 || k > QROUTE_MAX_K || t > QROUTE_MAX_N / k) return QGEMV_E_SHAPE;
  return QGEMV_OK;
}

int check_rows(int64_t t, int64_t k, int64_t c) {
  const int rc = check_slots(t, k);
  if (rc != QGEMV_OK) return rc;
  if (c < 0 || c > kMaxK) return QGEMV_E_SHAPE;
  if (t * k * (c + 16) > kRouteMaxElems) return QGEMV_E_SHAPE;
  return QGEMV_OK;
}

int gemm_routed(Fmt f, RouteFmt rf, const void* w, const void* x, const int32_t* order, const int32_t* offsets, void* y,
                int32_t y_dtype, int64_t t, int64_t k, int64_t e, int64_t m, int64_t kk, hipStream_t s) {
  int rc = check_slots(t, k);
  if (rc == QGEMV_OK) rc = check_shape(f, m, kk);
  if (rc != QGEMV_OK) return rc;
  if (e < 1 || e > QROUTE_MAX_E || m > kMaxK || kk > kPrefillMaxK) return QGEMV_E_SHAPE;
  if (f == kNvfp4 && kk % 64 != 0) return QGEMV_E_SHAPE;  // whole 64-weight steps
  const int64_t n = t * k;
  if (n > 0 && m > 0 && routed_work_items(routed_plan(rf, n, e, m)) > kMaxWorkItems) return QGEMV_E_SHAPE;
  if (order && t * kk * 2 > kRouteMaxXBytes) return QGEMV_E_SHAPE;
  if (!valid_dtype(y_dtype)) return QGEMV_E_DTYPE;
  if (t == 0 || m == 0) return QGEMV_OK;
  if (!w || !x || !offsets || !y) return QGEMV_E_NULL;
  if (misaligned(w, 16) || misaligned(x, 16) || misaligned(y, 16) || misaligned(order, 4) || misaligned(offsets, 4))
    return QGEMV_E_ALIGN;
  const int64_t wb = weight_bytes(f, m, kk), yb = n * m * dtype_size(y_dtype);
  if (overlap(y, yb, w, e * wb) || overlap(y, yb, x, (order ? t : n) * kk * 2) || overlap(y, yb, offsets, 4 * (e + 1)) ||
      (order && overlap(y, yb, order, 4 * n)))
    return QGEMV_E_ALIAS;
  return finish(launch_routed(rf, w, x, order, offsets, y, y_dtype, t, k, e, m, kk, wb, s));
}

int check_lora(int64_t t, int64_t e, int64_t r, int64_t m, int64_t k) {
  if (t < 0 || t > QROUTE_MAX_N || e < 1 || e > QROUTE_MAX_E || r <= 0 || r > QLORA_MAX_R || r % 8 != 0 || m < 0 ||
      m > kMaxK || k <= 0 || k > kPrefillMaxK || k % 8 != 0 || t * k * 2 > kRouteMaxXBytes)
    return QGEMV_E_SHAPE;
  return QGEMV_OK;
}

int lora(bool bf16, const void* x, const void* a, const void* b, const float* scale, const int32_t* order,
         const int32_t* offsets, const void* c, void* y, int32_t y_dtype, int64_t t, int64_t e, int64_t r, int64_t m,
         int64_t k, void* ws, int64_t ws_bytes, hipStream_t s) {
  const int rc = check_lora(t, e, r, m, k);
  if (rc != QGEMV_OK) return rc;
  if (!valid_dtype(y_dtype)) return QGEMV_E_DTYPE;
  if (t == 0 || m == 0) return QGEMV_OK;
  if (!x || !a || !b || !order || !offsets || !y || !ws) return QGEMV_E_NULL;
  if (misaligned(x, 16) || misaligned(a, 16) || misaligned(b, 16) || misaligned(c, 16) || misaligned(y, 16) ||
      misaligned(scale, 4) || misaligned(order, 4) || misaligned(offsets, 4) || misaligned(ws, 256))
    return QGEMV_E_ALIGN;
  const int64_t need = lora_workspace(t, e, r, m, k), yb = t * m * dtype_size(y_dtype);
  if (ws_bytes < need) return QGEMV_E_WORKSPACE;
  const struct {
    const void* p;
    int64_t bytes;
  } in[] = {{x, t * k * 2},     {a, e * r * k * 2},       {b, e * m * r * 2}, {scale, scale ? 4 * e : 0},
            {order, 4 * t},     {offsets, 4 * (e + 1)}};
  for (const auto& i : in)
    if (i.bytes > 0 && (overlap(y, yb, i.p, i.bytes) || overlap(ws, need, i.p, i.bytes))) return QGEMV_E_ALIAS;
  if (overlap(ws, need, y, yb)) return QGEMV_E_ALIAS;
  if (c && c != y && (overlap(y, yb, c, yb) || overlap(ws, need, c, yb))) return QGEMV_E_ALIAS;
  return finish(launch_lora(bf16, x, a, b, scale, order, offsets, c, y, y_dtype, t, e, r, m, k, ws, s));
}

}  // namespace

extern "C" {

int64_t qroute_workspace_bytes(int64_t n, int64_t E) {
  if (n < 0 || n > QROUTE_MAX_N || E < 1 || E > QROUTE_MAX_E) return QGEMV_E_SHAPE;
  return route_sort_workspace(n, E);
}

int qroute_sort(const int32_t* ids, int64_t n, int64_t E, int32_t* order, int32_t* position, int32_t* offsets,
                void* ws, int64_t ws_bytes, struct ihipStream_t* s) {
  const int64_t need = qroute_workspace_bytes(n, E);
  if (need < 0) return (int)need;
  if (!offsets || (n > 0 && (!ids || !order || !position))) return QGEMV_E_NULL;
  if (misaligned(ids, 4) || misaligned(order, 4) || misaligned(position, 4) || misaligned(offsets, 4))
    return QGEMV_E_ALIGN;
  const int64_t nb = 4 * n, ob = 4 * (E + 1);
  if (overlap(order, nb, ids, nb) || overlap(position, nb, ids, nb) || overlap(order, nb, position, nb) ||
      overlap(offsets, ob, ids, nb) || overlap(offsets, ob, order, nb) || overlap(offsets, ob, position, nb))
    return QGEMV_E_ALIAS;
  if (need > 0) {
    if (!ws) return QGEMV_E_NULL;
    if (misaligned(ws, 256)) return QGEMV_E_ALIGN;
    if (ws_bytes < need) return QGEMV_E_WORKSPACE;
    if (overlap(ws, need, ids, nb) || overlap(ws, need, order, nb) || overlap(ws, need, position, nb) ||
        overlap(ws, need, offsets, ob))
      return QGEMV_E_ALIAS;
  }
  return finish(launch_route_sort(ids, n, E, order, position, offsets, ws, s));
}

int qroute_gather(const void* x, const int32_t* order, const float* weights, void* out, int32_t dtype, int64_t T,
                  int64_t k, int64_t C, struct ihipStream_t* s) {
  const int rc = check_rows(T, k, C);
  if (rc != QGEMV_OK) return rc;
  if (!valid_dtype(dtype)) return QGEMV_E_DTYPE;
  if (T == 0 || C == 0) return QGEMV_OK;
  if (!x || !order || !out) return QGEMV_E_NULL;
  if (misaligned(x, 16) || misaligned(out, 16) || misaligned(order, 4) || misaligned(weights, 4)) return QGEMV_E_ALIGN;
  const int64_t n = T * k, sz = dtype_size(dtype), ob = n * C * sz;
  if (overlap(out, ob, x, T * C * sz) || overlap(out, ob, order, 4 * n) || (weights && overlap(out, ob, weights, 4 * n)))
    return QGEMV_E_ALIAS;
  return finish(launch_route_gather(x, order, weights, out, dtype, T, k, C, s));
}

int qroute_combine(const void* rows, int32_t rows_dtype, const int32_t* position, const float* weights, void* y,
                   int32_t y_dtype, int64_t T, int64_t k, int64_t C, struct ihipStream_t* s) {
  const int rc = check_rows(T, k, C);
  if (rc != QGEMV_OK) return rc;
  if (!valid_dtype(rows_dtype) || !valid_dtype(y_dtype)) return QGEMV_E_DTYPE;
  if (T == 0 || C == 0) return QGEMV_OK;
  if (!rows || !position || !y) return QGEMV_E_NULL;
  if (misaligned(rows, 16) || misaligned(y, 16) || misaligned(position, 4) || misaligned(weights, 4))
    return QGEMV_E_ALIGN;
  const int64_t n = T * k, yb = T * C * dtype_size(y_dtype);
  if (overlap(y, yb, rows, n * C * dtype_size(rows_dtype)) || overlap(y, yb, position, 4 * n) ||
      (weights && overlap(y, yb, weights, 4 * n)))
    return QGEMV_E_ALIAS;
  return finish(launch_route_combine(rows, rows_dtype, position, weights, y, y_dtype, T, k, C, s));
}

int qroute_combine_grad(const void* dy, int32_t dy_dtype, const void* rows, int32_t rows_dtype,
                        const int32_t* position, const float* weights, void* drows, float* dweights, int64_t T,
                        int64_t k, int64_t C, struct ihipStream_t* s) {
  const int rc = check_rows(T, k, C);
  if (rc != QGEMV_OK) return rc;
  if (!valid_dtype(dy_dtype) || !valid_dtype(rows_dtype)) return QGEMV_E_DTYPE;
  if (T == 0) return QGEMV_OK;
  if (!position || !weights || !dweights || (C > 0 && (!dy || !rows || !drows))) return QGEMV_E_NULL;
  if (misaligned(dy, 16) || misaligned(rows, 16) || misaligned(drows, 16) || misaligned(position, 4) ||
      misaligned(weights, 4) || misaligned(dweights, 4))
    return QGEMV_E_ALIGN;
  const int64_t n = T * k, db = T * C * dtype_size(dy_dtype), rb = n * C * dtype_size(rows_dtype);
  const struct {
    const void* p;
    int64_t bytes;
  } in[] = {{dy, db}, {rows, rb}, {position, 4 * n}, {weights, 4 * n}};
  for (const auto& i : in)
    if (overlap(drows, rb, i.p, i.bytes) || overlap(dweights, 4 * n, i.p, i.bytes)) return QGEMV_E_ALIAS;
  if (overlap(drows, rb, dweights, 4 * n)) return QGEMV_E_ALIAS;
  return finish(launch_route_combine_grad(dy, dy_dtype, rows, rows_dtype, position, weights, drows, dweights, T, k, C, s));
}

int qgemm_q4k_routed(const void* w, const void* x, const int32_t* order, const int32_t* offsets, void* y, int32_t y_dtype,
                     int64_t T, int64_t k, int64_t E, int64_t M, int64_t K, struct ihipStream_t* s) {
  return gemm_routed(kQ4k, kRouteQ4k, w, x, order, offsets, y, y_dtype, T, k, E, M, K, s);
}
int qgemm_nvfp4_routed(const void* w, const void* x, const int32_t* order, const int32_t* offsets, void* y, int32_t y_dtype,
                     int64_t T, int64_t k, int64_t E, int64_t M, int64_t K, struct ihipStream_t* s) {
  return gemm_routed(kNvfp4, kRouteNvfp4, w, x, order, offsets, y, y_dtype, T, k, E, M, K, s);
}
int qgemm_tq1_routed(const void* w, const void* x, const int32_t* order, const int32_t* offsets, void* y, int32_t y_dtype,
                     int64_t T, int64_t k, int64_t E, int64_t M, int64_t K, struct ihipStream_t* s) {
  return gemm_routed(kTq1, kRouteTq1, w, x, order, offsets, y, y_dtype, T, k, E, M, K, s);
}

int64_t qlora_workspace_bytes(int64_t T, int64_t E, int64_t r, int64_t M, int64_t K) {
  const int rc = check_lora(T, E, r, M, K);
  return rc != QGEMV_OK ? rc : lora_workspace(T, E, r, M, K);
}
int qlora_f16(const void* x, const void* a, const void* b, const float* scale, const int32_t* order,
              const int32_t* offsets, const void* c, void* y, int32_t y_dtype, int64_t T, int64_t E, int64_t r,
              int64_t M, int64_t K, void* ws, int64_t ws_bytes, struct ihipStream_t* s) {
  return lora(false, x, a, b, scale, order, offsets, c, y, y_dtype, T, E, r, M, K, ws, ws_bytes, s);
}
int qlora_bf16(const void* x, const void* a, const void* b, const float* scale, const int32_t* order,
               const int32_t* offsets, const void* c, void* y, int32_t y_dtype, int64_t T, int64_t E, int64_t r,
               int64_t M, int64_t K, void* ws, int64_t ws_bytes, struct ihipStream_t* s) {
  return lora(true, x, a, b, scale, order, offsets, c, y, y_dtype, T, E, r, M, K, ws, ws_bytes, s);
}

}  // extern "C"
