// C-ABI entry points of the drafted-tree step: host checks, then the
// launchers; and the tree's mask and depths from its parents.
#include <cmath>
#include <cstring>

#include "pa_internal.h"

using pa::fail;

namespace {

bool mis(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Rows a node takes in a tile: its heads per kv head, up to a power of two.
int32_t node_rows(int32_t num_q_heads, const pa_cache_desc* d) {
  int32_t r = 1;
  while (r < num_q_heads / d->num_kv_heads) r *= 2;
  return r;
}
pa_status check_tree(int32_t T, int32_t num_q_heads, int32_t max_q_len, const pa_cache_desc* desc) {
  pa_status st = pa::check_desc(desc, "pa_tree_attention");
  if (st != PA_OK) return st;
  if (T < 0 || num_q_heads <= 0 || max_q_len < 0)
    return fail(PA_ERR_INVALID, "pa_tree_attention: negative size or num_q_heads <= 0");
  if (T > 0 && max_q_len == 0) return fail(PA_ERR_INVALID, "pa_tree_attention: max_q_len is 0 with tokens");
  if (max_q_len > 65535) return fail(PA_ERR_UNSUPPORTED, "pa_tree_attention: max_q_len above 65535");
  if (num_q_heads % desc->num_kv_heads)
    return fail(PA_ERR_INVALID, "pa_tree_attention: num_q_heads must be a multiple of num_kv_heads");
  if (num_q_heads / desc->num_kv_heads > 128)
    return fail(PA_ERR_UNSUPPORTED, "pa_tree_attention: more than 128 query heads per kv head");
  return PA_OK;
}

// Query rows of one (sequence, kv head) at most, and the rows of a set of
// partial rows: an item's, at most 256.
int64_t tree_rows(int32_t num_q_heads, int32_t max_q_len, const pa_cache_desc* d) {
  return static_cast<int64_t>(max_q_len) * node_rows(num_q_heads, d);
}
int32_t slot_rows(int64_t rows) { return rows <= 64 ? 64 : rows <= 128 ? 128 : 256; }
// Per CTA two sets of partial rows (o, m, l) and 32 bytes on the item it leaves
// unfinished.
size_t tree_workspace(int64_t rows, const pa_cache_desc* d) {
  const size_t ctas = static_cast<size_t>(pa::sm_count());
  return (ctas * (2 * slot_rows(rows) * (d->head_dim + 2) * sizeof(float) + 32) + 255) & ~static_cast<size_t>(255);
}

}  // namespace

extern "C" {

pa_status pa_rope_cache_write(const void* q, const void* k, const void* v, int32_t in_dtype, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const int64_t* positions, const double* inv_freq,
                              int32_t rot_dim, int32_t interleaved, float factor, const int64_t* slot_mapping,
                              int64_t num_tokens, int32_t num_q_heads, void* q_out, int32_t q_out_dtype,
                              int64_t q_out_stride, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                              const pa_cache_desc* desc, void* stream) {
  const char* fn = "pa_rope_cache_write";
  pa_status st = pa::check_desc(desc, fn);
  if (st != PA_OK) return st;
  if (num_tokens < 0 || num_tokens > INT32_MAX) return fail(PA_ERR_INVALID, "%s: num_tokens out of range", fn);
  if (num_q_heads < 0) return fail(PA_ERR_INVALID, "%s: num_q_heads < 0", fn);
  const int32_t D = desc->head_dim, Hkv = desc->num_kv_heads;
  if (rot_dim <= 0 || rot_dim > D || rot_dim % 16)
    return fail(PA_ERR_INVALID, "%s: rot_dim must be a multiple of 16 in 16 .. head_dim", fn);
  if (interleaved != 0 && interleaved != 1) return fail(PA_ERR_INVALID, "%s: interleaved must be 0 or 1", fn);
  if (!std::isfinite(factor)) return fail(PA_ERR_INVALID, "%s: factor is not finite", fn);
  const bool q8 = pa::quantised(desc->kv_dtype);
  if (in_dtype != PA_DTYPE_F16 && in_dtype != PA_DTYPE_BF16 && in_dtype != PA_DTYPE_F32)
    return fail(PA_ERR_INVALID, "%s: in_dtype must be F16, BF16 or F32", fn);
  if (!q8 && in_dtype != desc->kv_dtype && in_dtype != PA_DTYPE_F32)
    return fail(PA_ERR_INVALID, "%s: in_dtype must equal kv_dtype or be F32", fn);
  if (num_q_heads > 0 && (in_dtype == PA_DTYPE_F32 ? q_out_dtype != PA_DTYPE_F16 && q_out_dtype != PA_DTYPE_BF16 &&
                                                         q_out_dtype != PA_DTYPE_F32
                                                   : q_out_dtype != in_dtype))
    return fail(PA_ERR_INVALID, "%s: q_out_dtype must equal in_dtype (F16, BF16 or F32 for F32 inputs)", fn);
  if (q8 ? !k_scale || !v_scale || !pa::aligned16(k_scale) || !pa::aligned16(v_scale) : k_scale || v_scale)
    return fail(PA_ERR_INVALID, "%s: FP8 / INT8 caches take 16-byte aligned scales, others none", fn);
  // 16-byte vectors: a token's row starts on a multiple of 16 bytes
  const int64_t in_step = in_dtype == PA_DTYPE_F32 ? 4 : 8, out_step = q_out_dtype == PA_DTYPE_F32 ? 4 : 8;
  if (k_stride < static_cast<int64_t>(Hkv) * D || v_stride < static_cast<int64_t>(Hkv) * D || k_stride % in_step ||
      v_stride % in_step)
    return fail(PA_ERR_INVALID, "%s: k_stride / v_stride below a row or not a multiple of 16 bytes", fn);
  if (num_q_heads > 0 &&
      (q_stride < static_cast<int64_t>(num_q_heads) * D || q_out_stride < static_cast<int64_t>(num_q_heads) * D ||
       q_stride % in_step || q_out_stride % out_step))
    return fail(PA_ERR_INVALID, "%s: q_stride / q_out_stride below a row or not a multiple of 16 bytes", fn);
  if (static_cast<int64_t>(num_q_heads) * (D / 16) + 2 * static_cast<int64_t>(Hkv) * (D / 16) > (1 << 23))
    return fail(PA_ERR_UNSUPPORTED, "%s: too many heads", fn);
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !positions || !inv_freq || !slot_mapping || !k_cache || !v_cache ||
      (num_q_heads > 0 && (!q || !q_out)))
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(k, 16) || mis(v, 16) || mis(k_cache, 16) || mis(v_cache, 16) ||
      (num_q_heads > 0 && (mis(q, 16) || mis(q_out, 16))) || mis(positions, 8) || mis(inv_freq, 8) ||
      mis(slot_mapping, 8))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  if (num_q_heads > 0 && q_out == q && (q_out_stride != q_stride || q_out_dtype != in_dtype))
    return fail(PA_ERR_INVALID, "%s: in place, q_out has q's stride and type", fn);
  pa::RopeLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.in_dtype = in_dtype;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved;
  a.factor = factor;
  a.slots = slot_mapping;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.q_out = q_out;
  a.q_out_dtype = q_out_dtype;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return pa::launch_rope_write(a, desc, stream);
}

size_t pa_tree_attention_workspace_size(int32_t num_q_heads, int32_t max_q_len, const pa_cache_desc* desc) {
  if (check_tree(0, num_q_heads, max_q_len, desc) != PA_OK) return 0;
  return tree_workspace(tree_rows(num_q_heads, max_q_len, desc), desc);
}

pa_status pa_tree_attention(const void* q, int32_t q_dtype, const int32_t* q_start, int32_t num_tokens,
                            int32_t max_q_len, const int64_t* tree_mask, int32_t mask_words, const void* k_cache,
                            const void* v_cache, const float* k_scale, const float* v_scale,
                            const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                            int32_t max_context_len, int32_t B, int32_t num_q_heads, float scale, void* out,
                            int32_t out_dtype, const pa_cache_desc* desc, void* workspace, size_t workspace_bytes,
                            void* stream) {
  const char* fn = "pa_tree_attention";
  pa_status st = check_tree(num_tokens, num_q_heads, max_q_len, desc);
  if (st != PA_OK) return st;
  if (B < 0 || max_context_len < 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID, "%s: B, max_context_len or max_blocks_per_seq out of range", fn);
  if (max_blocks_per_seq > INT32_MAX / PA_BLOCK_SIZE) return fail(PA_ERR_UNSUPPORTED, "%s: table too wide", fn);
  if (mask_words < (max_q_len + 63) / 64)
    return fail(PA_ERR_INVALID, "%s: mask_words below ceil(max_q_len / 64)", fn);
  if (!std::isfinite(scale)) return fail(PA_ERR_INVALID, "%s: scale is not finite", fn);
  const bool q8 = pa::quantised(desc->kv_dtype);
  if (q8 ? q_dtype != PA_DTYPE_F16 && q_dtype != PA_DTYPE_BF16 : q_dtype != desc->kv_dtype)
    return fail(PA_ERR_INVALID, "%s: q_dtype must equal kv_dtype (F16 or BF16 for an FP8 / INT8 cache)", fn);
  if (q8 ? !k_scale || !v_scale || !pa::aligned16(k_scale) || !pa::aligned16(v_scale) : k_scale || v_scale)
    return fail(PA_ERR_INVALID, "%s: FP8 / INT8 caches take 16-byte aligned scales, others none", fn);
  if (out_dtype != q_dtype && out_dtype != PA_DTYPE_F32)
    return fail(PA_ERR_INVALID, "%s: out_dtype must be q_dtype or F32", fn);
  if (B == 0 || num_tokens == 0) return PA_OK;
  if (!q || !q_start || !tree_mask || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(q, 16) || mis(k_cache, 16) || mis(v_cache, 16) || mis(out, 16) || mis(tree_mask, 8) || mis(q_start, 4) ||
      mis(block_tables, 4) || mis(context_lens, 4))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  // units of work (128-key chunks of every item, and 4 for its start and end) are counted in 32 bits
  const int64_t G = node_rows(num_q_heads, desc), chunks = static_cast<int64_t>(max_context_len) / 128 + 5;
  const int64_t items = static_cast<int64_t>(num_tokens) * G / 64 + B;
  if (items * desc->num_kv_heads > INT32_MAX / 2 / chunks)
    return fail(PA_ERR_UNSUPPORTED, "%s: more than 2^30 units of work", fn);
  if (static_cast<int64_t>(num_tokens) * num_q_heads > INT32_MAX)
    return fail(PA_ERR_UNSUPPORTED, "%s: too many query rows for one grid", fn);
  const int64_t rows = tree_rows(num_q_heads, max_q_len, desc);
  const size_t need = tree_workspace(rows, desc);
  if (!workspace || !pa::aligned16(workspace) || workspace_bytes < need)
    return fail(PA_ERR_INVALID, "%s: workspace NULL, misaligned or %zu of %zu bytes", fn, workspace_bytes, need);
  pa::TreeLaunch a;
  a.q = q;
  a.q_dtype = q_dtype;
  a.q_start = q_start;
  a.mask = tree_mask;
  a.words = mask_words;
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
  a.D = desc->head_dim;
  a.num_blocks = desc->num_blocks;
  a.kv_dtype = desc->kv_dtype;
  a.scale = scale;
  a.out = out;
  a.out_dtype = out_dtype;
  a.workspace = workspace;
  a.n_cta = pa::sm_count();
  a.rows = rows;
  a.slot_rows = slot_rows(rows);
  return pa::launch_tree(a, stream);
}

pa_status pa_tree_mask(const int32_t* parents, int32_t n, int32_t mask_words, int64_t* mask, int32_t* depths) {
  if (n < 0 || (n > 0 && (!parents || !mask)))
    return fail(PA_ERR_INVALID, "pa_tree_mask: n < 0 or null pointer");
  if (mask_words < (static_cast<int64_t>(n) + 63) / 64)
    return fail(PA_ERR_INVALID, "pa_tree_mask: mask_words below ceil(n / 64)");
  for (int32_t i = 0; i < n; ++i)
    if (parents[i] < -1 || parents[i] >= i)
      return fail(PA_ERR_INVALID, "pa_tree_mask: parent %d of node %d is not an earlier node", parents[i], i);
  const size_t row = static_cast<size_t>(mask_words);
  for (int32_t i = 0; i < n; ++i) {
    int64_t* m = mask + i * row;
    const int32_t p = parents[i];
    if (p >= 0)
      std::memcpy(m, mask + p * row, row * sizeof(int64_t));
    else
      std::memset(m, 0, row * sizeof(int64_t));
    m[i >> 6] = static_cast<int64_t>(static_cast<uint64_t>(m[i >> 6]) | (uint64_t{1} << (i & 63)));
    if (depths) depths[i] = p >= 0 ? depths[p] + 1 : 0;
  }
  return PA_OK;
}

pa_status pa_tree_accept(const int64_t* draft_tokens, const int64_t* target_tokens, const int32_t* parents,
                         const int32_t* q_start, int32_t num_tokens, int32_t B, int32_t max_path, int32_t* path,
                         int32_t* path_len, int64_t* next_token, void* stream) {
  const char* fn = "pa_tree_accept";
  if (num_tokens < 0 || B < 0 || max_path <= 0)
    return fail(PA_ERR_INVALID, "%s: num_tokens, B or max_path out of range", fn);
  if (B == 0) return PA_OK;
  if (!q_start || !path || !path_len || !next_token ||
      (num_tokens > 0 && (!draft_tokens || !target_tokens || !parents)))
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(draft_tokens, 8) || mis(target_tokens, 8) || mis(parents, 4) || mis(q_start, 4) || mis(path, 4) ||
      mis(path_len, 4) || mis(next_token, 8))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  return pa::launch_tree_accept(draft_tokens, target_tokens, parents, q_start, num_tokens, B, max_path, path,
                                path_len, next_token, stream);
}

pa_status pa_tree_commit(void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* q_start,
                         const int32_t* path, int32_t max_path, const int32_t* path_len, int32_t B,
                         int32_t* new_lens, const pa_cache_desc* desc, void* stream) {
  const char* fn = "pa_tree_commit";
  pa_status st = pa::check_desc(desc, fn);
  if (st != PA_OK) return st;
  if (B < 0 || max_blocks_per_seq <= 0 || max_path <= 0)
    return fail(PA_ERR_INVALID, "%s: B, max_blocks_per_seq or max_path out of range", fn);
  if (max_blocks_per_seq > INT32_MAX / PA_BLOCK_SIZE || desc->num_blocks > INT32_MAX / PA_BLOCK_SIZE)
    return fail(PA_ERR_UNSUPPORTED, "%s: more than 2^31 slots", fn);
  if (2 * static_cast<int64_t>(desc->num_kv_heads) * desc->head_dim > (1 << 23))
    return fail(PA_ERR_UNSUPPORTED, "%s: too many heads", fn);
  const bool q8 = pa::quantised(desc->kv_dtype);
  if (q8 ? !k_scale || !v_scale || !pa::aligned16(k_scale) || !pa::aligned16(v_scale) : k_scale || v_scale)
    return fail(PA_ERR_INVALID, "%s: FP8 / INT8 caches take 16-byte aligned scales, others none", fn);
  if (B == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !q_start || !path || !path_len)
    return fail(PA_ERR_INVALID, "%s: null pointer", fn);
  if (mis(k_cache, 16) || mis(v_cache, 16) || mis(block_tables, 4) || mis(context_lens, 4) || mis(q_start, 4) ||
      mis(path, 4) || mis(path_len, 4) || mis(new_lens, 4))
    return fail(PA_ERR_INVALID, "%s: misaligned pointer", fn);
  if (new_lens && new_lens < context_lens + B && context_lens < new_lens + B)
    return fail(PA_ERR_INVALID, "%s: new_lens overlaps context_lens", fn);
  pa::CommitLaunch a;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.max_blocks = max_blocks_per_seq;
  a.context_lens = context_lens;
  a.q_start = q_start;
  a.path = path;
  a.max_path = max_path;
  a.path_len = path_len;
  a.B = B;
  a.new_lens = new_lens;
  return pa::launch_tree_commit(a, desc, stream);
}

}  // extern "C"
