// C-ABI entry points of the block-scaled caches and of the sampled
// verification: host checks, then the launchers.
#include <cmath>

#include "pa_internal.h"

using pa::fail;

namespace {

bool mis(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// A block-scaled cache's shape.
pa_status check_scaled(const pa_cache_desc* d, const char* fn) {
  const pa_status st = pa::check_desc(d, fn);
  if (st != PA_OK) return st;
  if (d->kv_dtype != PA_DTYPE_FP8_E4M3)
    return fail(PA_ERR_UNSUPPORTED, "%s: a block-scaled cache holds FP8_E4M3 codes", fn);
  return PA_OK;
}

// Query rows that share a stream of K/V: a token's heads of one kv head take a
// power of two of them.  Below 128 they hold a whole sequence's, which the planner
// relies on: it has one item per (sequence, kv head) there.
constexpr int32_t kMaxHeads = 32;
int32_t item_rows(int32_t num_q_heads, int32_t max_q_len, const pa_cache_desc* d) {
  int64_t heads = 1;
  while (heads < num_q_heads / d->num_kv_heads) heads *= 2;
  const int64_t rows = heads * max_q_len;
  if (rows <= 40 && heads <= 8 && rows > 32) return 40;  // (whole tokens)
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
}

pa_status check_attention(int32_t num_q_heads, int32_t max_q_len, const pa_cache_desc* desc) {
  const char* fn = "pa_block_scaled_attention";
  const pa_status st = check_scaled(desc, fn);
  if (st != PA_OK) return st;
  if (num_q_heads <= 0 || num_q_heads % desc->num_kv_heads)
    return fail(PA_ERR_INVALID, "%s: num_q_heads must be a positive multiple of num_kv_heads", fn);
  if (num_q_heads / desc->num_kv_heads > kMaxHeads)
    return fail(PA_ERR_UNSUPPORTED, "%s: more than %d query heads per kv head", fn, kMaxHeads);
  if (max_q_len < 0) return fail(PA_ERR_INVALID, "%s: max_q_len < 0", fn);
  if (max_q_len > 65535) return fail(PA_ERR_UNSUPPORTED, "%s: max_q_len above 65535", fn);
  return PA_OK;
}

// Per CTA two sets of partial rows (o, m, l) and 32 bytes on the item it leaves
// unfinished.
size_t attention_workspace(int32_t rows, int32_t sms, const pa_cache_desc* d) {
  const size_t ctas = static_cast<size_t>(sms);
  return (ctas * (2 * rows * (d->head_dim + 2) * sizeof(float) + 32) + 255) & ~static_cast<size_t>(255);
}

}  // namespace

extern "C" {

pa_status pa_block_scaled_append(const void* k, const void* v, int32_t in_dtype, int64_t k_stride, int64_t v_stride,
                                 const int32_t* q_start, int32_t num_tokens, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t B, void* k_cache,
                                 void* v_cache, float* k_scale, float* v_scale, const pa_cache_desc* desc,
                                 void* stream) {
  const char* fn = "pa_block_scaled_append";
  const pa_status st = check_scaled(desc, fn);
  if (st != PA_OK) return st;
  if (in_dtype != PA_DTYPE_F16 && in_dtype != PA_DTYPE_BF16 && in_dtype != PA_DTYPE_F32)
    return fail(PA_ERR_INVALID, "%s: in_dtype must be F16, BF16 or F32", fn);
  if (num_tokens < 0 || B < 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID, "%s: num_tokens, B or max_blocks_per_seq out of range", fn);
  const int64_t row = static_cast<int64_t>(desc->num_kv_heads) * desc->head_dim, step = in_dtype == PA_DTYPE_F32 ? 4 : 8;
  if (k_stride < row || v_stride < row || k_stride % step || v_stride % step)
    return fail(PA_ERR_INVALID, "%s: k_stride / v_stride below a row or not a multiple of 16 bytes", fn);
  if (2 * static_cast<int64_t>(desc->num_kv_heads) > 8 * 65535 || B > INT32_MAX / 4 ||
      max_blocks_per_seq > INT32_MAX / PA_BLOCK_SIZE)
    return fail(PA_ERR_UNSUPPORTED, "%s: too many heads, sequences or blocks", fn);
  if (num_tokens == 0 || B == 0) return PA_OK;
  if (!k || !v || !q_start || !block_tables || !context_lens || !k_cache || !v_cache || !k_scale || !v_scale)
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(k, 16) || mis(v, 16) || mis(k_cache, 16) || mis(v_cache, 16) || mis(q_start, 4) || mis(block_tables, 4) ||
      mis(context_lens, 4) || mis(k_scale, 4) || mis(v_scale, 4))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  pa::ScaledAppendLaunch a;
  a.k = k;
  a.v = v;
  a.in_dtype = in_dtype;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_start = q_start;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.T = num_tokens;
  a.B = B;
  a.max_blocks = max_blocks_per_seq;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return pa::launch_scaled_append(a, desc, stream);
}

size_t pa_block_scaled_attention_workspace_size(int32_t num_q_heads, int32_t max_q_len, const pa_cache_desc* desc) {
  if (check_attention(num_q_heads, max_q_len, desc) != PA_OK) return 0;
  return attention_workspace(item_rows(num_q_heads, max_q_len, desc), pa::sm_count(), desc);
}

pa_status pa_block_scaled_attention(const void* q, int32_t q_dtype, int64_t q_stride, const int32_t* q_start,
                                    int32_t num_tokens, int32_t max_q_len, const void* k_cache, const void* v_cache,
                                    const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                    int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t max_context_len,
                                    int32_t B, int32_t num_q_heads, float scale, void* out, int32_t out_dtype,
                                    const pa_cache_desc* desc, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  const char* fn = "pa_block_scaled_attention";
  const pa_status st = check_attention(num_q_heads, max_q_len, desc);
  if (st != PA_OK) return st;
  if (q_dtype != PA_DTYPE_F16 && q_dtype != PA_DTYPE_BF16)
    return fail(PA_ERR_INVALID, "%s: q_dtype must be F16 or BF16", fn);
  if (out_dtype != q_dtype && out_dtype != PA_DTYPE_F32)
    return fail(PA_ERR_INVALID, "%s: out_dtype must be q_dtype or F32", fn);
  if (num_tokens < 0 || B < 0 || max_context_len < 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID, "%s: negative size or max_blocks_per_seq <= 0", fn);
  if (num_tokens > 0 && max_q_len == 0) return fail(PA_ERR_INVALID, "%s: max_q_len is 0 with tokens", fn);
  if (max_blocks_per_seq > INT32_MAX / PA_BLOCK_SIZE) return fail(PA_ERR_UNSUPPORTED, "%s: table too wide", fn);
  if (!std::isfinite(scale)) return fail(PA_ERR_INVALID, "%s: scale is not finite", fn);
  if (q_stride < static_cast<int64_t>(num_q_heads) * desc->head_dim || q_stride % 8)
    return fail(PA_ERR_INVALID, "%s: q_stride below a row or not a multiple of 16 bytes", fn);
  if (B == 0 || num_tokens == 0) return PA_OK;
  if (!q || !q_start || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens || !out)
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(q, 16) || mis(k_cache, 16) || mis(v_cache, 16) || mis(out, 16) || mis(q_start, 4) || mis(block_tables, 4) ||
      mis(context_lens, 4) || mis(k_scale, 4) || mis(v_scale, 4))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  // units of work (two for every 128-key chunk of an item, ten for its start and end at most)
  // are counted in 32 bits
  int64_t G = 1;
  while (G < num_q_heads / desc->num_kv_heads) G *= 2;
  const int32_t item = item_rows(num_q_heads, max_q_len, desc), sms = pa::sm_count();
  const int64_t units = 2 * (static_cast<int64_t>(max_context_len) / 128 + 1) + 10;
  const int64_t items = static_cast<int64_t>(num_tokens) * G / item + B;
  if (items * desc->num_kv_heads > INT32_MAX / 2 / units)
    return fail(PA_ERR_UNSUPPORTED, "%s: more than 2^30 units of work", fn);
  if (static_cast<int64_t>(num_tokens) * num_q_heads > INT32_MAX)
    return fail(PA_ERR_UNSUPPORTED, "%s: too many query rows", fn);
  const size_t need = attention_workspace(item, sms, desc);
  if (!workspace || !pa::aligned16(workspace) || workspace_bytes < need)
    return fail(PA_ERR_INVALID, "%s: workspace NULL, misaligned or %zu of %zu bytes", fn, workspace_bytes, need);
  pa::ScaledAttentionLaunch a;
  a.q = q;
  a.q_dtype = q_dtype;
  a.q_stride = q_stride;
  a.q_start = q_start;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.max_blocks = max_blocks_per_seq;
  a.context_lens = context_lens;
  a.max_context_len = max_context_len;
  a.max_q_len = max_q_len;
  a.B = B;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.Hkv = desc->num_kv_heads;
  a.num_blocks = desc->num_blocks;
  a.scale = scale;
  a.out = out;
  a.out_dtype = out_dtype;
  a.workspace = workspace;
  a.n_cta = sms;
  a.item_rows = item;
  return pa::launch_scaled_attention(a, stream);
}

pa_status pa_block_scaled_copy(void* dst_k, void* dst_v, float* dst_k_scale, float* dst_v_scale,
                               int32_t dst_num_blocks, const void* src_k, const void* src_v,
                               const float* src_k_scale, const float* src_v_scale, int32_t src_num_blocks,
                               const int64_t* pairs, int64_t num_pairs, const pa_cache_desc* desc, void* stream) {
  const char* fn = "pa_block_scaled_copy";
  const pa_status st = check_scaled(desc, fn);
  if (st != PA_OK) return st;
  if (num_pairs < 0) return fail(PA_ERR_INVALID, "%s: num_pairs < 0", fn);
  if (dst_num_blocks <= 0 || src_num_blocks <= 0) return fail(PA_ERR_INVALID, "%s: pool sizes must be > 0", fn);
  if (num_pairs > INT32_MAX || desc->num_kv_heads > 65535 * 8)
    return fail(PA_ERR_UNSUPPORTED, "%s: too many pairs or heads", fn);
  if (num_pairs == 0) return PA_OK;
  if (!dst_k || !dst_v || !dst_k_scale || !dst_v_scale || !src_k || !src_v || !src_k_scale || !src_v_scale || !pairs)
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(dst_k, 16) || mis(dst_v, 16) || mis(src_k, 16) || mis(src_v, 16) || mis(pairs, 8) || mis(dst_k_scale, 4) ||
      mis(dst_v_scale, 4) || mis(src_k_scale, 4) || mis(src_v_scale, 4))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  return pa::launch_scaled_copy(dst_k, dst_v, dst_k_scale, dst_v_scale, dst_num_blocks, src_k, src_v, src_k_scale,
                                src_v_scale, src_num_blocks, pairs, num_pairs, desc, stream);
}

pa_status pa_draft_verify(const int64_t* tokens, const float* target_probs, int64_t target_stride,
                          const float* draft_probs, int64_t draft_stride, int32_t vocab, const float* uniform,
                          const int32_t* parents, const int32_t* q_start, int32_t num_tokens, int32_t B,
                          int32_t max_path, int32_t* path, int32_t* path_len, int64_t* next_token, void* stream) {
  const char* fn = "pa_draft_verify";
  if (num_tokens < 0 || B < 0 || max_path <= 0)
    return fail(PA_ERR_INVALID, "%s: num_tokens, B or max_path out of range", fn);
  if (vocab < 1 || target_stride < vocab || (draft_probs && draft_stride < vocab))
    return fail(PA_ERR_INVALID, "%s: vocab < 1 or a stride below it", fn);
  if (vocab > 1 << 19) return fail(PA_ERR_UNSUPPORTED, "%s: vocab above 2^19", fn);
  if (B > INT32_MAX / 16) return fail(PA_ERR_UNSUPPORTED, "%s: too many sequences", fn);
  if (draft_probs && parents)
    return fail(PA_ERR_UNSUPPORTED, "%s: draft_probs with parents (sampled drafts are chains)", fn);
  if (B == 0) return PA_OK;
  if (!q_start || !path || !path_len || !next_token || (num_tokens > 0 && (!tokens || !target_probs || !uniform)))
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(tokens, 8) || mis(target_probs, 4) || mis(draft_probs, 4) || mis(uniform, 4) || mis(parents, 4) ||
      mis(q_start, 4) || mis(path, 4) || mis(path_len, 4) || mis(next_token, 8))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  pa::VerifyLaunch a;
  a.tokens = tokens;
  a.target = target_probs;
  a.draft = draft_probs;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.V = vocab;
  a.uniform = uniform;
  a.parents = parents;
  a.q_start = q_start;
  a.T = num_tokens;
  a.B = B;
  a.max_path = max_path;
  a.path = path;
  a.path_len = path_len;
  a.next_token = next_token;
  return pa::launch_draft_verify(a, stream);
}

}  // extern "C"
