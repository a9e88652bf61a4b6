// pkv_spec_api.cu -- C entry points of a speculative decoding step (declared
// in include/pkv.h): host-side validation and launches of the rotary append,
// the tree mask, the tree attention and the path commit.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <utility>

#include "pkv.h"
#include "pkv_kernels.h"
#include "pkv_validate.h"

using namespace pkv;

namespace {

pkv_status check_mask(const char* name, const pkv_tensor* m, int64_t T) {
  PKV_TRY(check_tensor(name, m, 2));
  PKV_NEED(m->dtype == PKV_I32, describe(name, m) + ": must be i32");
  PKV_NEED(m->shape[0] == T, describe(name, m) + ": first extent must be T = " + std::to_string(T));
  PKV_NEED(m->shape[1] >= 1 && m->shape[1] <= (1 << 20), describe(name, m) + ": needs 1 .. 2^20 words a row");
  PKV_NEED(m->shape[1] <= 1 || m->stride[1] == 1, std::string(name) + ": column stride must be 1");
  PKV_NEED(m->shape[0] <= 1 || m->stride[0] >= m->shape[1], std::string(name) + ": rows overlap");
  return PKV_OK;
}

// Whether a row of a [T, H, D] and one of b [U, J, D] (unit stride in D) have a
// byte in common.  Views of one buffer whose rows interleave (the q, k and v parts
// of a fused projection) span the same addresses without sharing any: where both
// have the same strides the rows are compared, difference of heads by difference
// of heads; views of other strides that span the same addresses count as shared.
bool rows_overlap(const pkv_tensor* a, const pkv_tensor* b) {
  if (!spans_overlap(a, b)) return false;
  const int64_t es = esize(a->dtype), row = a->shape[2] * es;
  const bool tokens = a->shape[0] > 1 || b->shape[0] > 1, heads = a->shape[1] > 1 || b->shape[1] > 1;
  auto stride = [&](int i) { return (a->shape[i] > 1 ? a : b)->stride[i]; };  // one row alone has no stride
  for (int i = 0; i < 2; ++i)
    if (a->shape[i] > 1 && b->shape[i] > 1 && a->stride[i] != b->stride[i]) return true;
  const int64_t st = tokens ? stride(0) * es : 0, sh = heads ? stride(1) * es : 0;
  const int64_t d0 = static_cast<const char*>(b->data) - static_cast<const char*>(a->data);
  for (int64_t h = -(a->shape[1] - 1); h <= b->shape[1] - 1; ++h) {
    const int64_t d = d0 + h * sh;  // from a row of a to the row of b h heads on, the same token
    int64_t t = st == 0 ? 0 : -d / st;
    for (int64_t u = t - 1; u <= t + 1; ++u) {
      const int64_t at = std::min(std::max(u, -(a->shape[0] - 1)), b->shape[0] - 1);
      const int64_t off = d + at * st;
      if (off < row && -off < row) return true;
    }
  }
  return false;
}

}  // namespace

extern "C" {

pkv_status pkv_rope_init(const pkv_rope_params* a, pkv_rope* rope) {
  PKV_NEED(a != nullptr, "params is NULL");
  PKV_NEED(rope != nullptr, "rope is NULL");
  PKV_NEED(a->rot_dim >= 2 && a->rot_dim <= 2 * PKV_ROPE_MAX_PAIRS && a->rot_dim % 2 == 0,
           "rot_dim must be even, 2 .. 256");
  PKV_NEED(a->base > 1.0 && isfinite(a->base), "base must be finite and > 1");
  PKV_NEED(a->scaling >= PKV_ROPE_PLAIN && a->scaling <= PKV_ROPE_SMOOTH, "unknown rope scaling");
  const bool scaled = a->scaling != PKV_ROPE_PLAIN;
  PKV_NEED(!scaled || (a->factor > 0.0 && isfinite(a->factor)), "factor must be finite and > 0");
  const bool banded = a->scaling == PKV_ROPE_BY_PARTS || a->scaling == PKV_ROPE_SMOOTH;
  PKV_NEED(!banded || (a->original_max_position > 0.0 && isfinite(a->original_max_position)),
           "original_max_position must be finite and > 0");
  PKV_NEED(a->attention_factor >= 0.0 && isfinite(a->attention_factor), "attention_factor must be finite and >= 0");
  const double pi2 = 6.283185307179586476925286766559;
  PKV_NEED(!banded || (a->fast >= 0.0 && a->slow >= 0.0), "fast and slow must be >= 0");
  const double fast = a->fast > 0.0 ? a->fast : (a->scaling == PKV_ROPE_SMOOTH ? 4.0 : 32.0);
  const double slow = a->slow > 0.0 ? a->slow : 1.0;
  PKV_NEED(!banded || (isfinite(fast) && isfinite(slow) && fast > slow), "fast must be finite and above slow");
  const double r = a->rot_dim, L = a->original_max_position, f = a->factor;
  double base = a->base;
  if (a->scaling == PKV_ROPE_NTK && a->rot_dim > 2) base *= pow(f, r / (r - 2.0));
  PKV_NEED(base > 0.0 && isfinite(base), "the scaled base leaves the numbers");
  double lo = 0.0, hi = 0.0;
  if (a->scaling == PKV_ROPE_BY_PARTS) {  // the pair index that makes t turns over L positions, rounded outwards
    auto at = [&](double t) { return r * log(L / (t * pi2)) / (2.0 * log(base)); };
    lo = std::max(floor(at(fast)), 0.0);
    hi = std::min(ceil(at(slow)), r - 1.0);
  }
  pkv_rope out{};
  for (int i = 0; i < a->rot_dim / 2; ++i) {
    double w = pow(base, -2.0 * i / r);
    if (a->scaling == PKV_ROPE_LINEAR) w /= f;
    if (a->scaling == PKV_ROPE_BY_PARTS) {
      const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      w = w * (1.0 - ramp) + w / f * ramp;
    }
    if (a->scaling == PKV_ROPE_SMOOTH) {
      const double keep = std::min(std::max((L * w / pi2 - slow) / (fast - slow), 0.0), 1.0);
      w = w * keep + w / f * (1.0 - keep);
    }
    PKV_NEED(isfinite(w), "an angle per position is not finite");
    const double turn = w / pi2;
    out.turns[i] = static_cast<uint64_t>(ldexp(turn - floor(turn), 64));  // a fraction below 1: fits 64 bits
  }
  double amp = a->attention_factor > 0.0 ? a->attention_factor : 1.0;
  if (a->attention_factor == 0.0 && a->scaling == PKV_ROPE_BY_PARTS) amp = f > 1.0 ? 0.1 * log(f) + 1.0 : 1.0;
  PKV_NEED(amp <= FLT_MAX, "attention_factor beyond fp32");
  out.amplitude = static_cast<float>(amp);
  out.rot_dim = a->rot_dim;
  out.interleaved = a->interleaved != 0;
  out.ready = 1;
  *rope = out;
  return PKV_OK;
}

pkv_status pkv_rope_append(const pkv_tensor* q, const pkv_tensor* k, const pkv_tensor* v,
                           const pkv_tensor* positions, const pkv_tensor* slot_mapping, const pkv_rope* rope,
                           pkv_tensor* q_out, pkv_tensor* k_cache, pkv_tensor* v_cache, float k_scale,
                           float v_scale, void* stream) {
  PKV_TRY(check_tensor("q", q, 3));
  PKV_TRY(check_tensor("q_out", q_out, 3));
  PKV_TRY(check_tensor("k", k, 3));
  PKV_TRY(check_tensor("v", v, 3));
  PKV_TRY(check_caches(k_cache, v_cache));
  PKV_NEED(rope != nullptr, "rope is NULL");
  PKV_NEED(rope->ready == 1 && rope->rot_dim >= 2 && rope->rot_dim <= 2 * PKV_ROPE_MAX_PAIRS && rope->rot_dim % 2 == 0,
           "rope was not made by pkv_rope_init");
  const int64_t T = q->shape[0], Hq = q->shape[1], Hkv = k_cache->shape[2], D = k_cache->shape[3];
  PKV_NEED(q->shape[2] == D, describe("q", q) + ": head dim differs from the cache's " + std::to_string(D));
  PKV_NEED(Hq >= 1 && Hq <= (1 << 16) && Hkv <= (1 << 16), "1 .. 65536 heads");
  PKV_NEED(k->shape[0] == T && k->shape[1] == Hkv && k->shape[2] == D,
           describe("k", k) + " must be [T, Hkv, D] of q and the cache");
  for (int i = 0; i < 3; ++i) {
    PKV_NEED(k->shape[i] == v->shape[i], "k and v shapes differ");
    PKV_NEED(q->shape[i] == q_out->shape[i], "q and q_out shapes differ");
  }
  PKV_NEED(k->dtype == q->dtype && v->dtype == q->dtype && q_out->dtype == q->dtype, "q, q_out, k and v dtypes differ");
  PKV_NEED(T <= INT32_MAX, "T beyond int32");
  PKV_TRY(check_index_vector("positions", positions, T));
  PKV_TRY(check_index_vector("slot_mapping", slot_mapping, T));
  const bool fp8 = k_cache->dtype == PKV_FP8_E4M3;
  int src_kind;
  if (q->dtype == PKV_F32 && (k_cache->dtype == PKV_F32 || fp8))
    src_kind = 0;
  else if (q->dtype == PKV_BF16 && (k_cache->dtype == PKV_BF16 || fp8))
    src_kind = 1;
  else
    return fail(PKV_ERR_UNSUPPORTED, std::string("rotary append of ") + dtype_name(q->dtype) + " rows into a " +
                                         dtype_name(k_cache->dtype) + " cache");
  PKV_NEED(D % 8 == 0 && D <= 256, "rotary append needs D a multiple of 8, at most 256");
  PKV_NEED(rope->rot_dim <= D, "rot_dim beyond D");
  PKV_TRY(check_rows("q", q));
  PKV_TRY(check_rows("q_out", q_out));
  PKV_TRY(check_rows("k", k));
  PKV_TRY(check_rows("v", v));
  // rows are rotated by many CTAs: a row of q_out may be the same row of q, but not another one, nor of k or v
  const bool in_place = q->data == q_out->data && (T <= 1 || q->stride[0] == q_out->stride[0]) && (Hq <= 1 || q->stride[1] == q_out->stride[1]);
  PKV_NEED(in_place || !rows_overlap(q, q_out), "q_out may be q itself, but must not overlap it otherwise");
  PKV_NEED(!rows_overlap(k, q_out) && !rows_overlap(v, q_out), "q_out must not overlap k or v");
  if (fp8) PKV_TRY(check_scales(k_scale, v_scale));
  unsigned int* err = nullptr;
  int sms = 0;
  PKV_TRY(device_state(&err, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return PKV_OK;
  RopeParams p{};
  p.q = q->data;
  p.k = k->data;
  p.v = v->data;
  p.q_out = q_out->data;
  p.q_st = q->stride[0];
  p.q_sh = q->stride[1];
  p.k_st = k->stride[0];
  p.k_sh = k->stride[1];
  p.v_st = v->stride[0];
  p.v_sh = v->stride[1];
  p.o_st = q_out->stride[0];
  p.o_sh = q_out->stride[1];
  p.positions = positions->data;
  p.slots = slot_mapping->data;
  p.pos_i64 = positions->dtype == PKV_I64;
  p.slots_i64 = slot_mapping->dtype == PKV_I64;
  p.k_cache = k_cache->data;
  p.v_cache = v_cache->data;
  p.T = T;
  p.Hq = static_cast<int32_t>(Hq);
  p.Hkv = static_cast<int32_t>(Hkv);
  p.D = static_cast<int32_t>(D);
  p.num_slots = k_cache->shape[0] * k_cache->shape[1];
  p.k_inv_scale = fp8 ? 1.0f / k_scale : 1.0f;  // IEEE fp32 division on the host, as in pkv_append
  p.v_inv_scale = fp8 ? 1.0f / v_scale : 1.0f;
  p.err = err;
  p.rope = *rope;
  const cudaError_t e = launch_rope_append(p, src_kind, fp8, sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "rotary append launch");
  return finish(st, "pkv_rope_append");
}

pkv_status pkv_tree_mask(const pkv_tensor* parents, const pkv_tensor* cu_seqlens_q, const pkv_tensor* seq_lens,
                         pkv_tensor* tree_mask, pkv_tensor* positions, void* stream) {
  int64_t B;
  PKV_TRY(check_step(cu_seqlens_q, seq_lens, B));
  PKV_TRY(check_tensor("parents", parents, 1));
  const int64_t T = parents->shape[0];
  PKV_NEED(T <= INT32_MAX, "T beyond int32");
  PKV_TRY(check_vector_i32("parents", parents, T));
  PKV_TRY(check_mask("tree_mask", tree_mask, T));
  PKV_TRY(check_vector_i32("positions", positions, T));
  // sequences are independent CTAs, and nodes read their ancestors' links
  PKV_TRY(check_apart("tree_mask", tree_mask,
                      {{"parents", parents}, {"cu_seqlens_q", cu_seqlens_q}, {"seq_lens", seq_lens}, {"positions", positions}}));
  PKV_TRY(check_apart("positions", positions, {{"parents", parents}, {"cu_seqlens_q", cu_seqlens_q}, {"seq_lens", seq_lens}}));
  unsigned int* err = nullptr;
  int sms = 0;
  PKV_TRY(device_state(&err, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B == 0 || T == 0) return PKV_OK;
  const cudaError_t e = launch_tree_mask(
      static_cast<const int32_t*>(parents->data), static_cast<const int32_t*>(cu_seqlens_q->data),
      static_cast<const int32_t*>(seq_lens->data), static_cast<int32_t>(B), T, static_cast<int32_t*>(tree_mask->data),
      tree_mask->stride[0], static_cast<int32_t>(tree_mask->shape[1]), static_cast<int32_t*>(positions->data), err, st);
  if (e != cudaSuccess) return cuda_fail(e, "tree mask launch");
  return finish(st, "pkv_tree_mask");
}

pkv_status pkv_tree_commit(const pkv_tensor* accepted, const pkv_tensor* accepted_lens,
                           const pkv_tensor* cu_seqlens_q, const pkv_tensor* seq_lens,
                           const pkv_tensor* block_tables, pkv_tensor* k_cache, pkv_tensor* v_cache,
                           pkv_tensor* new_seq_lens, void* stream) {
  int64_t B;
  PKV_TRY(check_step(cu_seqlens_q, seq_lens, B));
  PKV_TRY(check_tensor("accepted", accepted, 2));
  PKV_NEED(accepted->dtype == PKV_I32, describe("accepted", accepted) + ": must be i32");
  PKV_NEED(accepted->shape[0] == B, describe("accepted", accepted) + ": first extent must be B = " + std::to_string(B));
  PKV_NEED(accepted->shape[1] <= INT32_MAX, "accepted: row beyond int32");
  PKV_NEED(accepted->shape[1] <= 1 || accepted->stride[1] == 1, "accepted: column stride must be 1");
  PKV_TRY(check_vector_i32("accepted_lens", accepted_lens, B));
  PKV_TRY(check_block_tables(block_tables, B));
  PKV_TRY(check_caches(k_cache, v_cache));
  const int64_t bs = k_cache->shape[1], Hkv = k_cache->shape[2], D = k_cache->shape[3];
  PKV_NEED(block_tables->shape[1] * bs <= INT32_MAX, "max_blocks * block_size beyond int32");
  PKV_NEED(bs <= INT32_MAX, "block_size beyond int32");
  PKV_NEED(D % 8 == 0, "commit needs D a multiple of 8");
  if (new_seq_lens != nullptr) {
    PKV_TRY(check_vector_i32("new_seq_lens", new_seq_lens, B));
    // a sequence's first CTA writes it while the others may still read these
    PKV_TRY(check_apart("new_seq_lens", new_seq_lens,
                        {{"seq_lens", seq_lens}, {"accepted", accepted}, {"accepted_lens", accepted_lens},
                         {"cu_seqlens_q", cu_seqlens_q}, {"block_tables", block_tables}, {"k_cache", k_cache}, {"v_cache", v_cache}}));
  }
  unsigned int* err = nullptr;
  int sms = 0;
  PKV_TRY(device_state(&err, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B == 0) return PKV_OK;
  CommitParams p{};
  p.accepted = static_cast<const int32_t*>(accepted->data);
  p.accepted_stride = accepted->stride[0];
  p.A = static_cast<int32_t>(accepted->shape[1]);
  p.accepted_lens = static_cast<const int32_t*>(accepted_lens->data);
  p.cu_q = static_cast<const int32_t*>(cu_seqlens_q->data);
  p.seq_lens = static_cast<const int32_t*>(seq_lens->data);
  p.bt = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.max_blocks = static_cast<int32_t>(block_tables->shape[1]);
  p.B = static_cast<int32_t>(B);
  p.bs = static_cast<int32_t>(bs);
  p.num_blocks = k_cache->shape[0];
  p.k_cache = static_cast<char*>(k_cache->data);
  p.v_cache = static_cast<char*>(v_cache->data);
  p.row_bytes = Hkv * D * esize(k_cache->dtype);
  p.new_lens = new_seq_lens != nullptr ? static_cast<int32_t*>(new_seq_lens->data) : nullptr;
  p.err = err;
  const cudaError_t e = launch_tree_commit(p, st);
  if (e != cudaSuccess) return cuda_fail(e, "tree commit launch");
  return finish(st, "pkv_tree_commit");
}

pkv_status pkv_tree_attention_workspace_size(const pkv_tensor* q, const pkv_tensor* block_tables,
                                             const pkv_tensor* k_cache, int32_t max_q_len, size_t* bytes) {
  PKV_TRY(check_tensor("q", q, 3));
  PKV_TRY(check_tensor("block_tables", block_tables, 2));
  PKV_TRY(check_tensor("k_cache", k_cache, 4));
  PKV_NEED(bytes != nullptr, "bytes is NULL");
  *bytes = 0;
  if (k_cache->dtype == PKV_F32) return PKV_OK;
  const int64_t B = block_tables->shape[0], Hkv = k_cache->shape[2], G = Hkv > 0 ? q->shape[1] / Hkv : 1;
  const int64_t rows = B * tree_tc_rows_per_seq(B, Hkv, G, max_nodes_of(max_q_len, q->shape[0]),
                                                block_tables->shape[1] * k_cache->shape[1], k_cache->dtype == PKV_FP8_E4M3);
  *bytes = align_up(sizeof(float) * rows * q->shape[1] * (q->shape[2] + 1), 256);
  return PKV_OK;
}

pkv_status pkv_tree_attention(const pkv_tensor* q, const pkv_tensor* cu_seqlens_q, const pkv_tensor* seq_lens,
                              const pkv_tensor* block_tables, const pkv_tensor* k_cache, const pkv_tensor* v_cache,
                              const pkv_tensor* tree_mask, float scale, float k_scale, float v_scale,
                              int32_t max_q_len, pkv_tensor* out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  TreeParams p{};
  int kv;
  PKV_TRY(check_paged_rows(q, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache, scale, k_scale, v_scale, out, p, kv));
  PKV_TRY(check_mask("tree_mask", tree_mask, p.T));
  PKV_NEED(max_q_len <= 0 || 32 * tree_mask->shape[1] >= max_q_len, "tree_mask: fewer than max_q_len bits a row");
  size_t ws_need = 0;
  PKV_TRY(pkv_tree_attention_workspace_size(q, block_tables, k_cache, max_q_len, &ws_need));
  PKV_TRY(check_workspace(workspace, workspace_bytes, ws_need));
  p.mask = static_cast<const int32_t*>(tree_mask->data);
  p.mask_stride = tree_mask->stride[0];
  const int64_t max_q = max_nodes_of(max_q_len, p.T);
  p.max_nodes = static_cast<int32_t>(std::min<int64_t>(32 * tree_mask->shape[1], max_q));
  int sms = 0;
  PKV_TRY(device_state(&p.err, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.T == 0 || p.B == 0) return PKV_OK;
  const int out_kind = out->dtype == PKV_BF16;
  const cudaError_t e = kv == 0 ? launch_tree_f32(p, out_kind, st)
                                : launch_tree_tc(p, kv == 2, out_kind, max_q, block_tables->shape[1] * p.bs, workspace, sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  return finish(st, "pkv_tree_attention");
}

}  // extern "C"
