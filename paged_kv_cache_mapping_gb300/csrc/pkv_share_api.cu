// pkv_share_api.cu -- C entry points for requests that grow, shrink and share
// prompts (declared in include/pkv.h): host-side validation and launches of the
// step's tables, the shared prefixes and the attention that uses them.
#include <algorithm>

#include "pkv.h"
#include "pkv_kernels.h"
#include "pkv_validate.h"

using namespace pkv;

extern "C" {

pkv_status pkv_step_tables(const pkv_tensor* seq_lens, const pkv_tensor* new_seq_lens, const pkv_tensor* shared_blocks,
                           int32_t block_size, pkv_tensor* block_tables, pkv_tensor* free_blocks,
                           const pkv_tensor* free_count, pkv_tensor* new_free_count, pkv_tensor* cu_seqlens_q,
                           pkv_tensor* slot_mapping, pkv_tensor* positions, void* stream) {
  int64_t B;
  PKV_TRY(check_step(cu_seqlens_q, seq_lens, B));
  PKV_TRY(check_vector_i32("new_seq_lens", new_seq_lens, B));
  if (shared_blocks != nullptr) PKV_TRY(check_vector_i32("shared_blocks", shared_blocks, B));
  PKV_TRY(check_block_tables(block_tables, B));
  PKV_NEED(block_size >= 1, "block_size must be >= 1");
  PKV_NEED(block_tables->shape[1] <= INT32_MAX / block_size, "max_blocks * block_size beyond int32");
  PKV_TRY(check_tensor("free_blocks", free_blocks, 1));
  PKV_TRY(check_vector_i32("free_blocks", free_blocks, free_blocks->shape[0]));
  PKV_NEED(free_blocks->shape[0] < INT32_MAX, "free_blocks beyond int32");
  PKV_TRY(check_vector_i32("free_count", free_count, 1));
  PKV_TRY(check_vector_i32("new_free_count", new_free_count, 1));
  PKV_TRY(check_tensor("slot_mapping", slot_mapping, 1));
  const int64_t T = slot_mapping->shape[0];
  PKV_NEED(T < INT32_MAX, "T beyond int32");
  PKV_TRY(check_index_vector("slot_mapping", slot_mapping, T));
  if (positions != nullptr) PKV_TRY(check_vector_i32("positions", positions, T));
  // CTAs are still reading while others write; only the count is read by all before it is written
  const struct {
    const char* name;
    const pkv_tensor* t;
    bool out;
  } args[] = {{"seq_lens", seq_lens, false},        {"new_seq_lens", new_seq_lens, false}, {"shared_blocks", shared_blocks, false},
              {"free_count", free_count, false},    {"block_tables", block_tables, true},  {"free_blocks", free_blocks, true},
              {"cu_seqlens_q", cu_seqlens_q, true}, {"slot_mapping", slot_mapping, true},  {"positions", positions, true},
              {"new_free_count", new_free_count, true}};
  constexpr int kArgs = sizeof(args) / sizeof(args[0]);
  Span spans[kArgs];
  for (int i = 0; i < kArgs; ++i) {
    if (args[i].t != nullptr) spans[i] = span_of(args[i].t);
    for (int j = 0; args[i].out && j < i; ++j)
      PKV_NEED(!spans[i].meets(spans[j]) || (args[i].t == new_free_count && args[j].t == free_count),
               std::string(args[i].name) + " must not overlap " + args[j].name);
  }
  if (B > kMaxRequests) return fail(PKV_ERR_UNSUPPORTED, "more than " + std::to_string(kMaxRequests) + " requests");
  StepTablesParams p{};
  int sms = 0;
  PKV_TRY(device_state(&p.err, &sms));
  p.seq_lens = static_cast<const int32_t*>(seq_lens->data);
  p.new_seq_lens = static_cast<const int32_t*>(new_seq_lens->data);
  p.shared_blocks = shared_blocks != nullptr ? static_cast<const int32_t*>(shared_blocks->data) : nullptr;
  p.bs = block_size;
  p.by_bs = fast_div(static_cast<uint32_t>(block_size));
  p.bt = static_cast<int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.max_blocks = static_cast<int32_t>(block_tables->shape[1]);
  p.B = static_cast<int32_t>(B);
  p.free_blocks = static_cast<int32_t*>(free_blocks->data);
  p.F = free_blocks->shape[0];
  p.free_count = static_cast<const int32_t*>(free_count->data);
  p.new_free_count = static_cast<int32_t*>(new_free_count->data);
  p.cu_q = static_cast<int32_t*>(cu_seqlens_q->data);
  p.slots = slot_mapping->data;
  p.positions = positions != nullptr ? static_cast<int32_t*>(positions->data) : nullptr;
  p.T = T;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_step_tables(p, slot_mapping->dtype == PKV_I64, st);
  if (e != cudaSuccess) return cuda_fail(e, "step tables launch");
  return finish(st, "pkv_step_tables");
}

pkv_status pkv_shared_prefixes(const pkv_tensor* cu_seqlens_q, const pkv_tensor* seq_lens, const pkv_tensor* block_tables,
                               int32_t block_size, int32_t min_tokens, pkv_tensor* groups, void* stream) {
  int64_t B;
  PKV_TRY(check_step(cu_seqlens_q, seq_lens, B));
  PKV_TRY(check_block_tables(block_tables, B));
  PKV_NEED(block_size >= 1, "block_size must be >= 1");
  PKV_NEED(block_tables->shape[1] <= INT32_MAX / block_size, "max_blocks * block_size beyond int32");
  PKV_NEED(min_tokens >= 1, "min_tokens must be >= 1");
  PKV_TRY(check_groups(groups, B));
  PKV_TRY(check_apart("groups", groups, {{"cu_seqlens_q", cu_seqlens_q}, {"seq_lens", seq_lens}, {"block_tables", block_tables}}));
  if (B > kMaxRequests) return fail(PKV_ERR_UNSUPPORTED, "more than " + std::to_string(kMaxRequests) + " requests");
  PrefixParams p{};
  int sms = 0;
  PKV_TRY(device_state(&p.err, &sms));
  if (B == 0) return PKV_OK;
  p.cu_q = static_cast<const int32_t*>(cu_seqlens_q->data);
  p.seq_lens = static_cast<const int32_t*>(seq_lens->data);
  p.bt = static_cast<const int32_t*>(block_tables->data);
  p.bt_stride = block_tables->stride[0];
  p.max_blocks = static_cast<int32_t>(block_tables->shape[1]);
  p.B = static_cast<int32_t>(B);
  p.bs = block_size;
  p.min_tokens = min_tokens;
  p.groups = static_cast<int32_t*>(groups->data);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_shared_prefixes(p, st);
  if (e != cudaSuccess) return cuda_fail(e, "shared prefixes launch");
  return finish(st, "pkv_shared_prefixes");
}

pkv_status pkv_shared_attention_workspace_size(const pkv_tensor* q, const pkv_tensor* block_tables, const pkv_tensor* k_cache,
                                               int32_t max_q_len, int32_t max_group_len, size_t* bytes) {
  PKV_TRY(check_tensor("q", q, 3));
  PKV_TRY(check_tensor("block_tables", block_tables, 2));
  PKV_TRY(check_tensor("k_cache", k_cache, 4));
  PKV_NEED(bytes != nullptr, "bytes is NULL");
  *bytes = 0;
  const int64_t T = q->shape[0], B = block_tables->shape[0], Hkv = k_cache->shape[2], G = Hkv > 0 ? q->shape[1] / Hkv : 1;
  if (k_cache->dtype == PKV_F32 || T == 0 || B == 0) return PKV_OK;
  int64_t words;
  const int64_t rows = shared_rows(T, B, Hkv, G, max_nodes_of(max_q_len, T), max_nodes_of(max_group_len, T),
                                   block_tables->shape[1] * k_cache->shape[1], k_cache->dtype == PKV_FP8_E4M3, &words);
  *bytes = align_up(sizeof(float) * rows * q->shape[1] * (q->shape[2] + 1) + sizeof(int32_t) * words, 256);
  return PKV_OK;
}

pkv_status pkv_shared_attention(const pkv_tensor* q, const pkv_tensor* cu_seqlens_q, const pkv_tensor* seq_lens,
                                const pkv_tensor* block_tables, const pkv_tensor* groups, const pkv_tensor* k_cache,
                                const pkv_tensor* v_cache, float scale, float k_scale, float v_scale, int32_t max_q_len,
                                int32_t max_group_len, pkv_tensor* out, void* workspace, size_t workspace_bytes, void* stream) {
  TreeParams p{};
  int kv;
  PKV_TRY(check_paged_rows(q, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache, scale, k_scale, v_scale, out, p, kv));
  PKV_TRY(check_groups(groups, p.B));
  size_t ws_need = 0;
  PKV_TRY(pkv_shared_attention_workspace_size(q, block_tables, k_cache, max_q_len, max_group_len, &ws_need));
  PKV_TRY(check_workspace(workspace, workspace_bytes, ws_need));
  const int64_t max_q = max_nodes_of(max_q_len, p.T), max_group = max_nodes_of(max_group_len, p.T);
  p.max_nodes = static_cast<int32_t>(max_q);
  int sms = 0;
  PKV_TRY(device_state(&p.err, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.T == 0 || p.B == 0) return PKV_OK;
  const int out_kind = out->dtype == PKV_BF16;
  const int32_t* g = static_cast<const int32_t*>(groups->data);
  const cudaError_t e = kv == 0 ? launch_shared_f32(p, g, max_group, out_kind, st)
                                : launch_shared_tc(p, g, kv == 2, out_kind, max_q, max_group, block_tables->shape[1] * p.bs, workspace, sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "shared attention launch");
  return finish(st, "pkv_shared_attention");
}

}  // extern "C"
