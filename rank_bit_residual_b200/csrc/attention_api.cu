// attention_api.cu - the C ABI of the attention operators between two linears:
// argument checks and launches. No call here allocates device memory.
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"

namespace svdq {

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;   // of the norm and the append
constexpr int64_t kMaxPrompt = int64_t(1) << 24;   // rows, keys, sequences and heads of attention
constexpr int kMaxHeads = 1 << 15;
constexpr float kMaxScale = 8.507059e37f;   // 2^126: times log2(e) it is still finite

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A tensor that must be there.
svdq_status check_heads(const svdq_heads& x, int head_dim, int elem_bytes) {
  if (!x.data || x.heads < 1 || x.token_ld < head_dim || x.head_ld < head_dim) return SVDQ_EINVAL;
  if (x.heads > kMaxHeads) return SVDQ_EUNSUPPORTED;
  if (!aligned16(x.data) || (x.token_ld * elem_bytes) % 16 != 0 || (x.head_ld * elem_bytes) % 16 != 0)
    return SVDQ_EUNSUPPORTED;
  return SVDQ_OK;
}

bool absent(const svdq_heads& x) { return x.data == nullptr && x.heads == 0; }

svdq_status check_dim(int head_dim, int most) {
  if (head_dim < 1) return SVDQ_EINVAL;
  return head_dim % 8 == 0 && head_dim <= most ? SVDQ_OK : SVDQ_EUNSUPPORTED;
}

svdq_status check_rope(const svdq_rope& r, int head_dim, const int64_t* positions) {
  if (r.rot_dim < 0 || r.rot_dim > head_dim || r.rot_dim % 2 != 0) return SVDQ_EINVAL;
  if (r.rot_dim == 0) return SVDQ_OK;
  if (!r.turns || !positions || (r.interleaved != 0 && r.interleaved != 1) || !std::isfinite(r.amplitude))
    return SVDQ_EINVAL;
  return SVDQ_OK;
}

svdq_status check_cache(const svdq_kv_cache* c, int most) {
  if (!c || !c->k || !c->v || c->pages < 1 || c->page_size < 1 || c->heads < 1) return SVDQ_EINVAL;
  const svdq_status s = check_dim(c->head_dim, most);
  if (s != SVDQ_OK) return s;
  if (c->slot_ld < c->head_dim || c->head_ld < c->head_dim || c->page_ld < c->head_dim) return SVDQ_EINVAL;
  if (c->heads > kMaxHeads || c->pages > (int64_t(1) << 31) - 1) return SVDQ_EUNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || c->page_ld % 8 || c->slot_ld % 8 || c->head_ld % 8)
    return SVDQ_EUNSUPPORTED;
  return SVDQ_OK;
}

svdq_status check_weights(const void* q_weight, const void* k_weight, svdq_dtype dt, float eps) {
  if (dt != SVDQ_BF16 && dt != SVDQ_F32) return SVDQ_EINVAL;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return SVDQ_EINVAL;
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return SVDQ_EUNSUPPORTED;
  return SVDQ_OK;
}

// x and its output, or neither.
svdq_status check_pair(const svdq_heads& x, const svdq_heads& out, int head_dim, int elem_bytes) {
  if (absent(x) && absent(out)) return SVDQ_OK;
  svdq_status s = check_heads(x, head_dim, elem_bytes);
  if (s != SVDQ_OK) return s;
  if (out.heads != x.heads) return SVDQ_EINVAL;
  s = check_heads(out, head_dim, elem_bytes);
  if (s != SVDQ_OK) return s;
  if (out.data == x.data && (out.token_ld != x.token_ld || out.head_ld != x.head_ld)) return SVDQ_EINVAL;
  return SVDQ_OK;
}

svdq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SVDQ_OK : SVDQ_ECUDA; }

svdq_status check_decode_sizes(int32_t batch, int32_t heads, int32_t kv_heads, int32_t head_dim) {
  if (batch < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0) return SVDQ_EINVAL;
  if (heads > kMaxHeads || int64_t(batch) * heads > (int64_t(1) << 30)) return SVDQ_EUNSUPPORTED;
  return check_dim(head_dim, 128);
}

svdq_status check_prompt_sizes(int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t batch, int64_t q_tokens,
                               int64_t k_tokens) {
  if (batch < 0 || q_tokens < 0 || k_tokens < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
    return SVDQ_EINVAL;
  const svdq_status s = check_dim(head_dim, 128);
  if (s != SVDQ_OK) return s;
  if (heads > kMaxHeads || q_tokens > kMaxPrompt || k_tokens > kMaxPrompt || batch > kMaxPrompt ||
      heads * (q_tokens / 64 + batch) > (int64_t(1) << 30))
    return SVDQ_EUNSUPPORTED;
  return SVDQ_OK;
}

}  // namespace

}  // namespace svdq

using namespace svdq;

extern "C" {

svdq_status svdq_qk_norm_rope(svdq_heads q, svdq_heads k, svdq_dtype dtype, int64_t tokens, int32_t head_dim,
                              const int64_t* positions, svdq_rope rope, const void* q_weight,
                              const void* k_weight, svdq_dtype weight_dtype, float eps, svdq_heads q_out,
                              svdq_heads k_out, svdq_stream_t stream) {
  if ((dtype != SVDQ_BF16 && dtype != SVDQ_F32) || tokens < 0) return SVDQ_EINVAL;
  svdq_status s = check_dim(head_dim, 256);
  if (s != SVDQ_OK) return s;
  if ((s = check_weights(q_weight, k_weight, weight_dtype, eps)) != SVDQ_OK) return s;
  if (tokens == 0) return SVDQ_OK;
  if (tokens > kMaxTokens) return SVDQ_EUNSUPPORTED;
  const int es = dtype == SVDQ_BF16 ? 2 : 4;
  if ((s = check_rope(rope, head_dim, positions)) != SVDQ_OK) return s;
  if ((s = check_pair(q, q_out, head_dim, es)) != SVDQ_OK) return s;
  if ((s = check_pair(k, k_out, head_dim, es)) != SVDQ_OK) return s;
  if (q.heads + k.heads == 0) return SVDQ_OK;
  HeadsArgs a{};
  a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
  a.positions = positions, a.rope = rope, a.q_weight = q_weight, a.k_weight = k_weight;
  a.weight_bf16 = weight_dtype == SVDQ_BF16;
  a.eps = eps, a.tokens = tokens, a.head_dim = head_dim;
  return from_cuda(launch_heads(a, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

svdq_status svdq_kv_append(const svdq_kv_cache* cache, svdq_heads k, svdq_heads v, const int64_t* slots,
                           int64_t tokens, const int64_t* positions, svdq_rope rope, const void* k_weight,
                           svdq_dtype weight_dtype, float eps, svdq_heads q, const void* q_weight,
                           svdq_heads q_out, svdq_heads k_out, svdq_stream_t stream) {
  if (tokens < 0) return SVDQ_EINVAL;
  svdq_status s = check_cache(cache, 256);
  if (s != SVDQ_OK) return s;
  if ((s = check_weights(q_weight, k_weight, weight_dtype, eps)) != SVDQ_OK) return s;
  if (tokens == 0) return SVDQ_OK;
  if (tokens > kMaxTokens) return SVDQ_EUNSUPPORTED;
  const int dim = cache->head_dim;
  if (!slots) return SVDQ_EINVAL;
  if ((s = check_rope(rope, dim, positions)) != SVDQ_OK) return s;
  if ((s = check_heads(k, dim, 2)) != SVDQ_OK) return s;
  if ((s = check_heads(v, dim, 2)) != SVDQ_OK) return s;
  if (k.heads != cache->heads || v.heads != cache->heads) return SVDQ_EINVAL;
  if ((s = check_pair(q, q_out, dim, 2)) != SVDQ_OK) return s;
  if (!absent(k_out) && (s = check_pair(k, k_out, dim, 2)) != SVDQ_OK) return s;
  HeadsArgs a{};
  a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.k_out = k_out;
  a.cache = *cache, a.slots = slots;
  a.positions = positions, a.rope = rope, a.q_weight = q_weight, a.k_weight = k_weight;
  a.weight_bf16 = weight_dtype == SVDQ_BF16;
  a.eps = eps, a.tokens = tokens, a.head_dim = dim;
  a.status = device_status_word();
  return from_cuda(launch_heads(a, SVDQ_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

svdq_status svdq_attention_prompt_workspace_size(int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t batch,
                                                 int64_t q_tokens, int64_t k_tokens, size_t* bytes) {
  if (!bytes) return SVDQ_EINVAL;
  const svdq_status s = check_prompt_sizes(heads, kv_heads, head_dim, batch, q_tokens, k_tokens);
  if (s != SVDQ_OK) return s;
  *bytes = batch == 0 || q_tokens == 0 ? 0 : prompt_scratch_bytes(heads, kv_heads, head_dim, batch, q_tokens, k_tokens);
  return SVDQ_OK;
}

svdq_status svdq_attention_prompt(svdq_heads q, svdq_heads k, svdq_heads v, const int32_t* cu_q,
                                  const int32_t* cu_k, int32_t batch, int64_t q_tokens, int64_t k_tokens,
                                  int32_t head_dim, int32_t causal, float scale, svdq_heads out,
                                  void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  if ((causal != 0 && causal != 1) || !(std::fabs(scale) < kMaxScale)) return SVDQ_EINVAL;
  svdq_status s = check_prompt_sizes(q.heads, k.heads, head_dim, batch, q_tokens, k_tokens);
  if (s != SVDQ_OK) return s;
  if (batch == 0 || q_tokens == 0) return SVDQ_OK;
  if ((!cu_q || !cu_k) && batch != 1) return SVDQ_EINVAL;
  if ((s = check_pair(q, out, head_dim, 2)) != SVDQ_OK) return s;
  if (absent(q) || out.data == q.data || k.heads != v.heads) return SVDQ_EINVAL;
  // no keys at all: the tensors need not exist, the rows become zero
  if (k_tokens > 0) {
    if ((s = check_heads(k, head_dim, 2)) != SVDQ_OK) return s;
    if ((s = check_heads(v, head_dim, 2)) != SVDQ_OK) return s;
  }
  const size_t need = prompt_scratch_bytes(q.heads, k.heads, head_dim, batch, q_tokens, k_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SVDQ_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return SVDQ_EUNSUPPORTED;
  bool bad = false;
  const cudaError_t e = launch_prompt(q, k, v, cu_q, cu_k, batch, q_tokens, k_tokens, head_dim, causal != 0, scale,
                                      out, workspace, reinterpret_cast<cudaStream_t>(stream), &bad);
  if (bad) return SVDQ_EUNSUPPORTED;
  return from_cuda(e);
}

svdq_status svdq_attention_decode_workspace_size(int32_t batch, int32_t heads, int32_t kv_heads,
                                                 int32_t head_dim, size_t* bytes) {
  if (!bytes) return SVDQ_EINVAL;
  const svdq_status s = check_decode_sizes(batch, heads, kv_heads, head_dim);
  if (s != SVDQ_OK) return s;
  *bytes = paged_scratch_bytes(batch, heads, kv_heads, head_dim);
  return SVDQ_OK;
}

svdq_status svdq_attention_decode(svdq_heads q, const svdq_kv_cache* cache, const int32_t* page_table,
                                  int64_t table_ld, const int32_t* kv_len, int32_t batch, float scale,
                                  svdq_heads out, void* workspace, size_t workspace_bytes,
                                  svdq_stream_t stream) {
  svdq_status s = check_cache(cache, 128);
  if (s != SVDQ_OK) return s;
  if (!(std::fabs(scale) < kMaxScale) || table_ld < 0) return SVDQ_EINVAL;
  if ((s = check_decode_sizes(batch, q.heads, cache->heads, cache->head_dim)) != SVDQ_OK) return s;
  if (batch == 0) return SVDQ_OK;
  if (!kv_len || (!page_table && table_ld > 0) || absent(q)) return SVDQ_EINVAL;
  if ((s = check_pair(q, out, cache->head_dim, 2)) != SVDQ_OK) return s;
  if (out.data == q.data) return SVDQ_EINVAL;
  if (!workspace || workspace_bytes < paged_scratch_bytes(batch, q.heads, cache->heads, cache->head_dim))
    return SVDQ_EWORKSPACE;
  if (!aligned16(workspace)) return SVDQ_EUNSUPPORTED;
  const int64_t limit = (int64_t(1) << 31) - 1;   // of a sequence's keys, whatever the table could hold
  const int64_t most = table_ld > limit / cache->page_size ? limit : table_ld * cache->page_size;
  if (!paged_fits(batch, q.heads, cache->heads, most)) return SVDQ_EUNSUPPORTED;
  return from_cuda(launch_paged(q, *cache, page_table, table_ld, kv_len, batch, scale, out, workspace,
                                reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
