// pkv_validate.h -- host-side validation shared by the entry points of
// libpkv: checks of a tensor's type, extents, strides and alignment, and the
// helpers that turn a failure into a status with its message.  Messages are
// built only when a check fails.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "pkv.h"
#include "pkv_kernels.h"

namespace pkv {

inline pkv_status fail(pkv_status st, const std::string& msg) { return record_failure(st, msg); }

inline pkv_status cuda_fail(cudaError_t e, const char* where) {
  cudaGetLastError();  // clear a sticky launch error of this thread
  return fail(PKV_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

inline const char* dtype_name(pkv_dtype d) {
  switch (d) {
    case PKV_F32: return "f32";
    case PKV_BF16: return "bf16";
    case PKV_FP8_E4M3: return "fp8_e4m3";
    case PKV_I32: return "i32";
    case PKV_I64: return "i64";
  }
  return "?";
}

inline int esize(pkv_dtype d) {
  switch (d) {
    case PKV_F32: return 4;
    case PKV_BF16: return 2;
    case PKV_FP8_E4M3: return 1;
    case PKV_I32: return 4;
    case PKV_I64: return 8;
  }
  return 0;
}

inline std::string describe(const char* name, const pkv_tensor* t) {
  std::string s = std::string(name) + " (" + dtype_name(t->dtype) + ", shape [";
  for (int i = 0; i < t->ndim && i < 4; ++i) s += (i ? ", " : "") + std::to_string(t->shape[i]);
  return s + (t->ndim > 4 ? ", ..])" : "])");
}

inline pkv_status need(bool ok, const std::string& msg) {
  return ok ? PKV_OK : fail(PKV_ERR_INVALID_ARGUMENT, msg);
}

#define PKV_TRY(expr)                 \
  do {                                \
    pkv_status _s = (expr);           \
    if (_s != PKV_OK) return _s;      \
  } while (0)

#define PKV_NEED(ok, msg)                                          \
  do {                                                             \
    if (!(ok)) return pkv::fail(PKV_ERR_INVALID_ARGUMENT, (msg));  \
  } while (0)

inline pkv_status check_tensor(const char* name, const pkv_tensor* t, int ndim) {
  if (t == nullptr) return fail(PKV_ERR_INVALID_ARGUMENT, std::string(name) + " is NULL");
  if (t->ndim != ndim)
    return fail(PKV_ERR_INVALID_ARGUMENT,
                describe(name, t) + ": expected " + std::to_string(ndim) + " dimensions");
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] < 0) return fail(PKV_ERR_INVALID_ARGUMENT, describe(name, t) + ": negative extent");
  int64_t n = 1;
  for (int i = 0; i < ndim; ++i) n *= t->shape[i];
  if (n > 0 && t->data == nullptr) return fail(PKV_ERR_INVALID_ARGUMENT, std::string(name) + ": data is NULL");
  return PKV_OK;
}

inline bool contiguous(const pkv_tensor* t) {
  int64_t expect = 1;
  for (int i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] != 1 && t->stride[i] != expect) return false;
    expect *= t->shape[i];
  }
  return true;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline pkv_status check_vector_i32(const char* name, const pkv_tensor* t, int64_t len) {
  PKV_TRY(check_tensor(name, t, 1));
  PKV_NEED(t->dtype == PKV_I32, describe(name, t) + ": must be i32");
  PKV_NEED(t->shape[0] == len, describe(name, t) + ": expected length " + std::to_string(len));
  PKV_NEED(t->shape[0] <= 1 || t->stride[0] == 1, describe(name, t) + ": must be contiguous");
  return PKV_OK;
}

inline pkv_status check_block_tables(const pkv_tensor* bt, int64_t B) {
  PKV_TRY(check_tensor("block_tables", bt, 2));
  PKV_NEED(bt->dtype == PKV_I32, describe("block_tables", bt) + ": must be i32");
  PKV_NEED(bt->shape[0] == B,
           describe("block_tables", bt) + ": first extent must be B = " + std::to_string(B));
  PKV_NEED(bt->shape[1] >= 1, describe("block_tables", bt) + ": needs at least one column");
  PKV_NEED(bt->shape[1] <= 1 || bt->stride[1] == 1, "block_tables: column stride must be 1");
  PKV_NEED(bt->shape[0] <= 1 || bt->stride[0] >= bt->shape[1], "block_tables: rows overlap");
  return PKV_OK;
}

inline pkv_status check_caches(const pkv_tensor* kc, const pkv_tensor* vc) {
  PKV_TRY(check_tensor("k_cache", kc, 4));
  PKV_TRY(check_tensor("v_cache", vc, 4));
  PKV_NEED(kc->dtype == vc->dtype, "k_cache and v_cache dtypes differ");
  for (int i = 0; i < 4; ++i) PKV_NEED(kc->shape[i] == vc->shape[i], "k_cache and v_cache shapes differ");
  PKV_NEED(kc->dtype == PKV_F32 || kc->dtype == PKV_BF16 || kc->dtype == PKV_FP8_E4M3,
           describe("k_cache", kc) + ": cache dtype must be f32, bf16 or fp8_e4m3");
  PKV_NEED(contiguous(kc) && contiguous(vc), "caches must be contiguous [num_blocks, block_size, Hkv, D]");
  PKV_NEED(kc->shape[1] >= 1, "block_size must be >= 1");
  PKV_NEED(kc->shape[2] >= 1 && kc->shape[3] >= 1, "Hkv and D must be >= 1");
  PKV_NEED(kc->shape[0] <= INT32_MAX, "num_blocks beyond int32");
  PKV_NEED(aligned(kc->data, 16) && aligned(vc->data, 16), "cache data must be 16-byte aligned");
  return PKV_OK;
}

inline int log2_exact(int64_t v) {
  if (v <= 0 || (v & (v - 1))) return -1;
  int k = 0;
  while ((int64_t(1) << k) < v) ++k;
  return k;
}

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace pkv
