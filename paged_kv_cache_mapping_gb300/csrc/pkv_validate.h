// pkv_validate.h -- host-side validation shared by the entry points of
// libpkv: checks of a tensor's type, extents, strides and alignment, and the
// helpers that turn a failure into a status with its message.  Messages are
// built only when a check fails.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <string>
#include <utility>

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

constexpr int kTreeKeySlack = 256;  // key numbers, in 32 bits, run up to two tiles past a sequence (the next tile's pages)

inline pkv_status check_index_vector(const char* name, const pkv_tensor* t, int64_t len) {
  PKV_TRY(check_tensor(name, t, 1));
  PKV_NEED(t->dtype == PKV_I32 || t->dtype == PKV_I64, describe(name, t) + ": must be i32 or i64");
  PKV_NEED(t->shape[0] == len, describe(name, t) + ": expected length " + std::to_string(len));
  PKV_NEED(len <= 1 || t->stride[0] == 1, describe(name, t) + ": must be contiguous");
  return PKV_OK;
}

// [T, H, D] rows: unit stride in D, 16-byte aligned
inline pkv_status check_rows(const char* name, const pkv_tensor* t) {
  const int es = esize(t->dtype);
  PKV_NEED(t->stride[2] == 1 || t->shape[2] == 1, std::string(name) + " must have unit stride in D");
  PKV_NEED(aligned(t->data, 16) && (t->stride[0] * es) % 16 == 0 && (t->stride[1] * es) % 16 == 0,
           std::string(name) + " rows must be 16-byte aligned (data and strides)");
  return PKV_OK;
}

inline pkv_status check_scales(float k_scale, float v_scale) {
  PKV_NEED(k_scale > 0.f && v_scale > 0.f && isfinite(k_scale) && isfinite(v_scale),
           "fp8 scales must be positive and finite");
  return PKV_OK;
}

// Lengths, counts and tables of a step: B sequences.
inline pkv_status check_step(const pkv_tensor* cu_seqlens_q, const pkv_tensor* seq_lens, int64_t& B) {
  PKV_TRY(check_tensor("seq_lens", seq_lens, 1));
  B = seq_lens->shape[0];
  PKV_NEED(B <= (1 << 24), "B beyond 2^24 sequences");
  PKV_TRY(check_vector_i32("seq_lens", seq_lens, B));
  PKV_TRY(check_vector_i32("cu_seqlens_q", cu_seqlens_q, B + 1));
  return PKV_OK;
}

// groups of requests: first, behind the last, prefix tokens
inline pkv_status check_groups(const pkv_tensor* g, int64_t B) {
  PKV_TRY(check_tensor("groups", g, 2));
  PKV_NEED(g->dtype == PKV_I32, describe("groups", g) + ": must be i32");
  PKV_NEED(g->shape[0] == B && g->shape[1] == 3, describe("groups", g) + ": must be [B, 3], B = " + std::to_string(B));
  PKV_NEED(contiguous(g), "groups must be contiguous");
  return PKV_OK;
}

// nodes a sequence may have: the caller's bound, else every row
inline int64_t max_nodes_of(int32_t max_q_len, int64_t T) {
  return max_q_len > 0 ? std::min<int64_t>(max_q_len, T) : T;
}

// The address range that a tensor spans (lo == hi: it has no elements).
struct Span {
  uintptr_t lo = 0, hi = 0;
  bool meets(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};
inline Span span_of(const pkv_tensor* t) {
  int64_t first = 0, last = 0;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] == 0) return {};
    const int64_t d = (t->shape[i] - 1) * t->stride[i];
    (d < 0 ? first : last) += d;
  }
  const uintptr_t at = reinterpret_cast<uintptr_t>(t->data);
  return {at + first * esize(t->dtype), at + (last + 1) * esize(t->dtype)};
}

// Whether the address ranges that two tensors span have a byte in common.
inline bool spans_overlap(const pkv_tensor* a, const pkv_tensor* b) { return span_of(a).meets(span_of(b)); }

// What a call writes must not overlap what its CTAs still read.
inline pkv_status check_apart(const char* name, const pkv_tensor* out, std::initializer_list<std::pair<const char*, const pkv_tensor*>> others) {
  for (const auto& o : others)
    PKV_NEED(!spans_overlap(out, o.second), std::string(name) + " must not overlap " + o.first);
  return PKV_OK;
}

// Rows of a packed batch over the paged caches, as the attention of trees and of
// shared prefixes takes them: checks, then everything of p that follows from these.
// kv: 0 = f32, 1 = bf16, 2 = e4m3.
inline pkv_status check_paged_rows(const pkv_tensor* q, const pkv_tensor* cu_seqlens_q, const pkv_tensor* seq_lens,
                                   const pkv_tensor* block_tables, const pkv_tensor* k_cache, const pkv_tensor* v_cache,
                                   float scale, float k_scale, float v_scale, const pkv_tensor* out, TreeParams& p, int& kv) {
  int64_t B;
  PKV_TRY(check_tensor("q", q, 3));
  PKV_TRY(check_tensor("out", out, 3));
  PKV_TRY(check_step(cu_seqlens_q, seq_lens, B));
  PKV_TRY(check_block_tables(block_tables, B));
  PKV_TRY(check_caches(k_cache, v_cache));
  const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t NB = k_cache->shape[0], bs = k_cache->shape[1], Hkv = k_cache->shape[2];
  PKV_NEED(T <= INT32_MAX, "T beyond int32");
  PKV_NEED(k_cache->shape[3] == D, "q and cache head dims differ");
  PKV_NEED(Hq >= 1 && Hq % Hkv == 0, "Hq must be a positive multiple of Hkv");
  PKV_NEED(Hq <= (1 << 16), "Hq beyond 65536");
  PKV_NEED(out->shape[0] == T && out->shape[1] == Hq && out->shape[2] == D, describe("out", out) + " must have q's shape");
  PKV_NEED(out->dtype == PKV_F32 || out->dtype == PKV_BF16, "out must be f32 or bf16");
  PKV_NEED(block_tables->shape[1] * bs <= INT32_MAX - kTreeKeySlack, "max_blocks * block_size beyond int32");
  PKV_NEED(NB >= 1, "the cache has no blocks");
  if (q->dtype != PKV_F32 && T > (int64_t(1) << 30) / Hq)
    return fail(PKV_ERR_UNSUPPORTED, "T * Hq beyond 2^30 (a sequence's rows and work items are numbered in 32 bits)");
  if (NB * bs > INT32_MAX / Hkv)
    return fail(PKV_ERR_UNSUPPORTED, "num_blocks * block_size * Hkv beyond int32 (rows are numbered in 32 bits)");
  if (q->dtype == PKV_F32 && k_cache->dtype == PKV_F32)
    kv = 0;
  else if (q->dtype == PKV_BF16 && k_cache->dtype == PKV_BF16)
    kv = 1;
  else if (q->dtype == PKV_BF16 && k_cache->dtype == PKV_FP8_E4M3)
    kv = 2;
  else
    return fail(PKV_ERR_UNSUPPORTED, std::string("q ") + dtype_name(q->dtype) + " with a " +
                                         dtype_name(k_cache->dtype) + " cache");
  if (kv == 0)
    PKV_NEED(D % 32 == 0 && D <= 256, "f32 attention needs D a multiple of 32, at most 256");
  else if (D != 64 && D != 128)
    return fail(PKV_ERR_UNSUPPORTED, "bf16/fp8 attention is built for D = 64 and D = 128");
  PKV_TRY(check_rows("q", q));
  PKV_NEED(out->stride[2] == 1 || D == 1, "out must have unit stride in D");
  const int oes = esize(out->dtype);
  PKV_NEED(aligned(out->data, 16) && (out->stride[0] * oes) % 8 == 0 && (out->stride[1] * oes) % 8 == 0,
           "out rows must be 8-byte aligned (data and strides)");
  if (kv == 2) PKV_TRY(check_scales(k_scale, v_scale));
  PKV_NEED(scale == scale, "scale is NaN");
  p.q = q->data;
  p.q_st = q->stride[0];
  p.q_sh = q->stride[1];
  p.out = out->data;
  p.T = T;
  p.o_st = out->stride[0];
  p.o_sh = out->stride[1];
  p.cu_q = static_cast<const int32_t*>(cu_seqlens_q->data);
  p.seq_lens = static_cast<const int32_t*>(seq_lens->data);
  p.bt = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.max_blocks = static_cast<int32_t>(block_tables->shape[1]);
  p.B = static_cast<int32_t>(B);
  p.k_cache = k_cache->data;
  p.v_cache = v_cache->data;
  p.num_blocks = NB;
  p.bs = static_cast<int32_t>(bs);
  p.bs_shift = log2_exact(bs);
  p.Hq = static_cast<int32_t>(Hq);
  p.Hkv = static_cast<int32_t>(Hkv);
  p.G = static_cast<int32_t>(Hq / Hkv);
  p.D = static_cast<int32_t>(D);
  const float kLog2e = 1.4426950408889634f;
  p.qk_scale_log2 = scale * (kv == 2 ? k_scale : 1.0f) * kLog2e;
  p.v_scale = kv == 2 ? v_scale : 1.0f;
  return PKV_OK;
}

inline pkv_status check_workspace(const void* workspace, size_t bytes, size_t need_bytes) {
  if (bytes < need_bytes)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL,
                "workspace needs " + std::to_string(need_bytes) + " bytes, got " + std::to_string(bytes));
  PKV_NEED(need_bytes == 0 || (workspace != nullptr && aligned(workspace, 256)), "workspace must be 256-byte aligned");
  return PKV_OK;
}

}  // namespace pkv
