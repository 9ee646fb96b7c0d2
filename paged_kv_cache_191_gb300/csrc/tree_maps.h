// Tensor maps of the attention kernels that multiply whole chunks of a paged cache.
#pragma once

#include <cudaTypedefs.h>

#include "kv_map.h"

namespace pa {
namespace {

inline pa_status encode_map(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* p, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box, const char* what) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!fn) return fail(PA_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", what);
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(m, dt, rank, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(PA_ERR_CUDA, "%s: tensor map encode failed (%d)", what, static_cast<int>(r));
  return PA_OK;
}
// TMA map over a 16-bit cache of head_dim 128 whose box is one (block, kv
// head) tile, landing as [group of 8 tokens][span of 64 dims][8][128 B]: the
// 8-row groups of a span are evenly spaced over a run of tiles, as one UMMA
// operand of many tiles wants them.
inline pa_status make_group_map(CUtensorMap* m, const void* cache, int Hkv, int num_blocks, CUtensorMapDataType dt,
                         const char* what) {
  const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(2) * Hkv, static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[4] = {256, 128, 2048, static_cast<cuuint64_t>(4096) * Hkv};
  const cuuint32_t box[5] = {64, 8, 2, 2, 1};
  return encode_map(m, dt, 5, cache, dims, strides, box, what);
}
// TMA map over q [T][Hq][D], `stride` elements between tokens, whose box is a 64-dim span of gp heads (a group,
// padded to a power of two) of as many nodes as make 32 rows.
inline pa_status make_q_map(CUtensorMap* m, const void* q, int D, int Hq, int T, int64_t stride, int gp,
                     CUtensorMapDataType dt, const char* what) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(gp), static_cast<cuuint32_t>(gp < 32 ? 32 / gp : 1)};
  return encode_map(m, dt, 3, q, dims, strides, box, what);
}

}  // namespace
}  // namespace pa
