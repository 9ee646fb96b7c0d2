// Attention of a drafted tree over a paged cache, on tcgen05 (sm_103a).
//
// What it computes ("LLM推理引擎深度实战：从PagedAttention到分布式推理部署",
// section 6.1: the target model checks the drafted tokens in one pass; here the
// draft is a tree).  The n nodes of sequence b are the last n tokens of its
// L-token context, their K/V already in the cache.  Node i sees every key of
// the context before the tree and the nodes its mask row names:
//     out_i = sum_t p_it V_t / sum_t p_it,   p_it = exp(scale q_i . K_t)
// over t < L - n and over t = L - n + j with bit j of mask row i set.
//
// Rows and work.  The query rows of one (sequence, kv head) are the pairs
// (node, head of the group), the group padded to a power of two; they all read
// the same K/V, so an item is up to 64, 128 or 256 of them (Lay::ITEM), and
// streams the context in chunks of 128 keys (8 blocks).  One unit of work is one
// chunk of one item (an item's start and end count as kItem more); the launch
// has one persistent CTA per SM, and CTA k takes units [k u, (k + 1) u) of the
// batch in order, u = ceil(units / CTAs): every CTA streams the same number of
// chunks whatever the lengths.  (Items of the same kv head side by side where the
// planner finds that they line up.)  The lengths stay on the device: each CTA counts
// the units itself from context_lens and q_start.  An item that spans CTAs
// leaves partial rows (o, m, l), at most two sets per CTA, merged by tree_merge
// with log-sum-exp weights.
//
// Inside a CTA (tree_common.cuh):
//   warp 0       producer: Q rows and the K and V chunks into a ring of slots
//                by TMA (128-byte swizzle, one box per block); with 1-byte
//                caches warp 2 issues half of each chunk's boxes;
//   warp 1       issues the MMAs from one thread;
//   warp 3       planner: the CTA's pieces of items, published a few ahead, and
//                their mask words;
//   warps 4-7,   two softmax warpgroups, each with a tile: a score buffer and an
//   8-11         O accumulator in tensor memory;
//   warps 12-15  1-byte caches only: convert landed codes to the 16-bit layouts
//                the MMAs read.
// Two kernels differ in what a softmax thread owns.  Up to 64 rows of a kv head, 32
// with bf16 queries (tree_keys.cuh): a key, with transposed products, so that work is
// in proportion to the rows.  More (tree_rows.cuh): a row, with products of 128 rows.
// At 64 rows (16 sequences of 32 kv heads, contexts of 2048 .. 4096 tokens) the
// first takes 143 us, 86 % of the copy rate, and the second would compute on twice
// the rows; at 128 rows (64 sequences of 8 kv heads, mean context 2064) the first,
// with two tiles of 64 rows, took 163 us where the second took 109 (both with one
// bf16 for a weight).
//
// P is rounded to V's 16-bit type (the queries', which 1-byte codes are converted
// to), which the product shares, and normalised by the sum of the rounded weights
// (1-byte caches: weight x V scale is rounded, and the sum is of the weights before
// it), so a row that rests on one key returns that key's value.  A bf16 weight would
// have 8 bits: it is carried as two bf16 halves (off by 2^-17, as in the other
// attention calls) and V multiplied by both.  One bf16 took 110 us for 120 (64
// sequences of 8 kv heads, 128 rows) and 321 for 428 (512 rows), at errors of 2^-9 of a
// row in float32 outputs, and in bf16 ones of 1.3 times those of an exact softmax.
// References, l and O are float32.
//
// What bounds it: HBM while the rows per kv head stay below ~290 (4 D flops
// per key and row against 4 D bytes per key at 16 bits), the exponentials and
// the MMAs above that, shared memory with 1-byte caches.  The hot loops are kept
// short and the rest out of their way: the instruction cache, not the issue rate,
// limits a kernel of this many roles.
//
// Values in masked places: a masked exponent is replaced; V rows past the
// context's end are zeroed in shared memory, and a node's V row that holds an
// infinity or NaN (a slot nothing was ever written to) is zeroed too and added
// to O by hand for the rows that do see it, so it reaches no other row.
#include <cudaTypedefs.h>

#include <mutex>

#include "kv_map.h"
#include "pa_internal.h"
#include "tree_keys.cuh"
#include "tree_rows.cuh"

namespace pa {
namespace {

constexpr int kMaxDevices = 64;

// Merge of the items that span CTAs: block (k, y) takes rows 8 y .. 8 y + 7 of
// the item that CTA k left unfinished, one warp per row; lane i holds part i's
// (m, l), 32 parts at a time.
constexpr int kMergeRows = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeRows) tree_merge(const __grid_constant__ TreeArgs a) {
  constexpr int V = D / 32;
  const int lane = static_cast<int>(threadIdx.x & 31), k0 = static_cast<int>(blockIdx.x);
  const int row = static_cast<int>(blockIdx.y) * kMergeRows + static_cast<int>(threadIdx.x >> 5);
  dev::grid_dependency_wait();
  // parts, first slot, first query row, row of the tree | kv head, rows, CTAs from part to part
  const int4 s0 = a.split[2 * k0], s1 = a.split[2 * k0 + 1];
  const int h = (s0.w + row) & ((1 << a.gl) - 1);
  if (s0.x == 0 || row >= s1.y || h >= a.G) return;
  auto slot_row = [&](int i) { return static_cast<size_t>(i == 0 ? s0.y : 2 * (k0 + i * s1.z)) * a.slot_rows + row; };
  float M = -INFINITY, ls = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < s0.x; i0 += 32) {
    const int n = min(32, s0.x - i0);
    auto row_of = [&](int i, float2 (&f)[V / 2]) {
      const float* src = a.part_o + slot_row(i0 + i) * D + lane * V;
#pragma unroll
      for (int v = 0; v < V / 2; ++v) f[v] = *reinterpret_cast<const float2*>(src + 2 * v);
    };
    auto add = [&](float wi, const float2 (&f)[V / 2]) {
#pragma unroll
      for (int v = 0; v < V / 2; ++v) {
        acc[2 * v] = fmaf(wi, f[v].x, acc[2 * v]);
        acc[2 * v + 1] = fmaf(wi, f[v].y, acc[2 * v + 1]);
      }
    };
    float2 early[4][V / 2];  // the first rows are on their way with the weights
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) row_of(i, early[i]);
    const float mv = lane < n ? a.part_m[slot_row(i0 + lane)] : -INFINITY;
    const float lv = lane < n ? a.part_l[slot_row(i0 + lane)] : 0.f;
    const float nm = fmaxf(M, warp_max(mv));
    if (nm == -INFINITY) continue;  // no key in any of them
    const float again = dev::ex2(M - nm), w = lane < n ? dev::ex2(mv - nm) : 0.f;
    M = nm;
    float wl = w * lv;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) wl += __shfl_xor_sync(FULL, wl, off);
    ls = ls * again + wl;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= again;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) add(__shfl_sync(FULL, w, i), early[i]);
#pragma unroll 4
    for (int i = 4; i < n; ++i) {
      float2 f[V / 2];
      row_of(i, f);
      add(__shfl_sync(FULL, w, i), f);
    }
  }
  const float inv = M == -INFINITY ? 0.f : 1.f / ls;
  const size_t at =
      static_cast<size_t>((s0.z + ((s0.w + row) >> a.gl)) * a.Hq + s1.x * a.G + h) * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    if (a.out_f32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + v) = make_float2(acc[v] * inv, acc[v + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at + v) = dev::pack2<T>(acc[v] * inv, acc[v + 1] * inv);
  }
}

// ---- launch ------------------------------------------------------------------
pa_status encode_map(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* p, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!fn) return fail(PA_ERR_CUDA, "pa_tree_attention: cuTensorMapEncodeTiled unavailable");
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(m, dt, rank, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(PA_ERR_CUDA, "pa_tree_attention: tensor map encode failed (%d)", static_cast<int>(r));
  return PA_OK;
}
// TMA map over a 16-bit cache of head_dim 128 whose box is one (block, kv
// head) tile, landing as [group of 8 tokens][span of 64 dims][8][128 B]: the
// 8-row groups of a span are evenly spaced over a run of tiles, as one UMMA
// operand of many tiles wants them.
pa_status make_group_map(CUtensorMap* m, const void* cache, int Hkv, int num_blocks, CUtensorMapDataType dt) {
  const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(2) * Hkv, static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[4] = {256, 128, 2048, static_cast<cuuint64_t>(4096) * Hkv};
  const cuuint32_t box[5] = {64, 8, 2, 2, 1};
  return encode_map(m, dt, 5, cache, dims, strides, box);
}
// TMA map over q [T][Hq][D] whose box is a 64-dim span of gp heads (a group,
// padded to a power of two) of as many nodes as make 32 rows.
pa_status make_q_map(CUtensorMap* m, const void* q, int D, int Hq, int T, int gp, CUtensorMapDataType dt) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(D) * 2 * Hq};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(gp), static_cast<cuuint32_t>(gp < 32 ? 32 / gp : 1)};
  return encode_map(m, dt, 3, q, dims, strides, box);
}

template <typename KT, typename T, int D, bool ROWS>
pa_status launch_t(const TreeLaunch& l, CUtensorMapDataType dt, cudaStream_t stream) {
  using L = Lay<KT, T, D, ROWS>;
  const auto kernel = [] {
    if constexpr (ROWS)
      return tree_rows<KT, T, D>;
    else
      return tree_keys<KT, T, D>;
  }();
  constexpr int EB = static_cast<int>(sizeof(KT));
  TreeArgs a;
  a.q = l.q;
  a.q_start = l.q_start;
  a.mask = reinterpret_cast<const uint64_t*>(l.mask);
  a.block_tables = l.block_tables;
  a.context_lens = l.context_lens;
  a.k_scale = l.k_scale;
  a.v_scale = l.v_scale;
  a.out = l.out;
  a.B = l.B;
  a.T = l.T;
  a.Hq = l.Hq;
  a.Hkv = l.Hkv;
  a.G = l.Hq / l.Hkv;
  a.max_blocks = l.max_blocks;
  a.num_blocks = l.num_blocks;
  a.max_context_len = l.max_context_len;
  a.max_q_len = l.max_q_len;
  a.words = l.words;
  a.n_cta = l.n_cta;
  a.gl = 0;
  while ((1 << a.gl) < a.G) ++a.gl;
  const float mag = l.scale < 0.f ? -l.scale : l.scale;
  // a scale of 0 stays 0 for every finite score and leaves masked ones at -inf
  a.scale_log2 = mag * 1.4426950408889634f > 1e-30f ? mag * 1.4426950408889634f : 1e-30f;
  a.negate = l.scale < 0.f ? 1u : 0u;
  a.out_f32 = l.out_dtype == PA_DTYPE_F32;
  // few units: many CTAs and a longer merge against long runs (one sequence of 600
  // tokens, 8 kv heads: 13.3 us for 15.9 at 5)
  a.min_units = 2;
  a.item_rows = L::ITEM;
  a.slot_rows = l.slot_rows;
  const size_t rows = static_cast<size_t>(2) * a.n_cta * a.slot_rows;
  a.part_o = static_cast<float*>(l.workspace);
  a.part_m = a.part_o + rows * D;
  a.part_l = a.part_m + rows;
  a.split = reinterpret_cast<int4*>(a.part_l + rows);

  CUtensorMap tmK, tmV, tmQ;
  for (int v = 0; v < 2; ++v) {
    CUtensorMap* m = v ? &tmV : &tmK;
    const void* cache = v ? l.v_cache : l.k_cache;
    const pa_status st = D * EB == 256
                             ? make_group_map(m, cache, l.Hkv, l.num_blocks, dt)
                             : make_kv_map(m, cache, l.Hkv, l.num_blocks, D * EB, EB, dt, "pa_tree_attention");
    if (st != PA_OK) return st;
  }
  const pa_status sq = make_q_map(&tmQ, l.q, D, l.Hq, l.T, 1 << a.gl,
                                  std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
  if (sq != PA_OK) return sq;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices)
    return fail(PA_ERR_CUDA, "pa_tree_attention: no CUDA device");
  static std::once_flag once[kMaxDevices];
  static cudaError_t setup[kMaxDevices];
  std::call_once(once[dev], [dev, kernel] {
    setup[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    // the registers that the roles ask for have to be the launch's, or they would wait for them forever
    constexpr int WANT = 256 * L::HIGH + (L::THREADS - 256) * L::LOW;
    cudaFuncAttributes fa;
    if (setup[dev] == cudaSuccess) setup[dev] = cudaFuncGetAttributes(&fa, kernel);
    if (setup[dev] == cudaSuccess && fa.numRegs * L::THREADS < WANT) setup[dev] = cudaErrorInvalidConfiguration;
  });
  if (setup[dev] != cudaSuccess)
    return fail(PA_ERR_CUDA, "pa_tree_attention: %s", cudaGetErrorString(setup[dev]));
  cudaError_t e = launch_dependent(kernel, dim3(static_cast<unsigned>(a.n_cta)), dim3(L::THREADS),
                                   L::BYTES, stream, tmK, tmV, tmQ, a);
  if (e == cudaSuccess && l.max_context_len > kKeys)
    e = launch_dependent(tree_merge<T, D>, dim3(static_cast<unsigned>(a.n_cta), a.slot_rows / kMergeRows),
                         dim3(32 * kMergeRows), 0, stream, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_tree_attention launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

// A thread per key while one kv head's rows fit its items (64, with bf16 weights
// 32), else a thread per row (products and exponentials are then in 128s of rows).
template <typename KT, typename T, int D>
pa_status launch_d(const TreeLaunch& l, CUtensorMapDataType dt, cudaStream_t stream) {
  return l.rows > Lay<KT, T, D, false>::ITEM ? launch_t<KT, T, D, true>(l, dt, stream) : launch_t<KT, T, D, false>(l, dt, stream);
}

}  // namespace

pa_status launch_tree(const TreeLaunch& l, void* stream_ptr) {
  cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
  if (l.kv_dtype == PA_DTYPE_F16)
    return l.D == 64 ? launch_d<__half, __half, 64>(l, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, st)
                     : launch_d<__half, __half, 128>(l, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, st);
  if (l.kv_dtype == PA_DTYPE_BF16)
    return l.D == 64 ? launch_d<__nv_bfloat16, __nv_bfloat16, 64>(l, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, st)
                     : launch_d<__nv_bfloat16, __nv_bfloat16, 128>(l, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, st);
  const bool f16 = l.q_dtype == PA_DTYPE_F16;  // 1-byte codes, head_dim 128 (checked by the caller)
  if (l.kv_dtype == PA_DTYPE_INT8)
    return f16 ? launch_d<int8_t, __half, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st)
               : launch_d<int8_t, __nv_bfloat16, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st);
  return f16 ? launch_d<uint8_t, __half, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st)
             : launch_d<uint8_t, __nv_bfloat16, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st);
}

pa_status read_errors_tree(uint32_t* flags, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_err, sizeof(v));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_tree_err, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_device_errors: %s", cudaGetErrorString(e));
  *flags = v;
  return PA_OK;
}

}  // namespace pa
