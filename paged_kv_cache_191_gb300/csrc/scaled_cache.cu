// New rows into a block-scaled cache (E4M3 codes, one power-of-two scale per
// (block, kv head)), for sm_103a.
//
// For the rows x that a (block, head) gets: 2^e the smallest power of two with
// max |x| <= 448 2^e, scale = max(2^e, the scale of the rows that stay), code =
// E4M3(x / scale).  A power of two leaves E4M3's relative precision as it is (it
// is a floating-point code), makes the division a product, and makes rounding
// the staying rows' codes to a grown scale a shift of their exponents: exact but
// for those that become subnormal, where a scale of amax / 448 would round every
// code again with every growth.
//
// One warp owns a (block, head): its tile of K and that of V, 16 rows of 128 values
// each, 8 values a lane and row, so that all rows of a tile (16-bit input: of both) are
// in flight at once and a maximum is one reduction over the warp; nothing is read
// twice.  Tiles are found from q_start alone: sequence b may touch at most n_b / 16 + 2
// blocks, so its tiles are grid columns q_start[b] / 16 + 2 b .., and a warp finds its
// sequence by a search 32 ways at a time.  No column is longer than the batch is,
// however uneven the sequences are.  The chain of loads before the rows (q_start,
// length, table) is what both tiles share.  Nine chunks of up to 2043 tokens, 32 heads,
// f16: 39 us, 86 % of the copy rate (47 us with a warp per tile); float32, whose K and V
// tiles do not fit a warp's registers together, 80 us, 70 %; one token 2.8 us, 64
// of 8 heads 3.4 us: the launch.
#include "cache_rows.cuh"
#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

__device__ uint32_t g_scaled_err;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 8, kDim = 128;

struct AppendArgs {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  const int32_t* q_start;
  const int32_t* block_tables;
  const int32_t* context_lens;
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int32_t T, B, Hkv, max_blocks, num_blocks;
};

__device__ __forceinline__ int column_of(const AppendArgs& a, int b) { return a.q_start[b] / PA_BLOCK_SIZE + 2 * b; }

// First new row and length of sequence b; the length is 0, and the bits say why,
// where they are out of range.
__device__ __forceinline__ uint32_t rows_of(const AppendArgs& a, int b, int& qs, int& n, int& L) {
  qs = a.q_start[b];
  const int end = a.q_start[b + 1];
  L = a.context_lens[b];
  uint32_t err = 0;
  if (qs < 0 || end < qs || end > a.T) err |= PA_DEVERR_QUERY_RANGE;
  n = err ? 0 : end - qs;
  if (L < 0 || n > L || L > static_cast<int64_t>(a.max_blocks) * PA_BLOCK_SIZE) err |= PA_DEVERR_CONTEXT_LEN;
  if (err) n = 0;
  return err;
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e] * inv, x[2 * e + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// A lane's values of a tile as they came: 8 of each of 8 rows.
template <int IN>
struct Rows {
  uint4 w[8];
  __device__ __forceinline__ void load(int i, const void* src, size_t at, bool live) {
    w[i] = live ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + at) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(int i, float (&y)[8]) const {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = IN == PA_DTYPE_F16 ? dev::unpack2<__half>(u[e]) : dev::unpack2<__nv_bfloat16>(u[e]);
      y[2 * e] = f.x;
      y[2 * e + 1] = f.y;
    }
  }
  // The largest size over the warp's values (finite: of those that are), as a float32's
  // bits; sizes order like their bits, infinities and NaN above all.
  __device__ __forceinline__ uint32_t largest(bool finite) const {
    constexpr uint32_t INF = IN == PA_DTYPE_F16 ? 0x7C00u : 0x7F80u;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t size = u[e] & 0x7FFF7FFFu;
        if (finite) size &= ~__vcmpgeu2(size, INF * 0x10001u);
        top = __vmaxu2(top, size);
      }
    }
    top = __reduce_max_sync(FULL, max(top & 0xFFFFu, top >> 16));
    const float2 f = IN == PA_DTYPE_F16 ? dev::unpack2<__half>(top) : dev::unpack2<__nv_bfloat16>(top);
    return __float_as_uint(f.x) & 0x7FFFFFFFu;
  }
};
template <>
struct Rows<PA_DTYPE_F32> {
  float x[8][8];
  __device__ __forceinline__ void load(int i, const void* src, size_t at, bool live) {
    if (live) {
      dev::load8<PA_DTYPE_F32>(src, at, x[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    }
  }
  __device__ __forceinline__ void get(int i, float (&y)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[i][e];
  }
  __device__ __forceinline__ uint32_t largest(bool finite) const {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __float_as_uint(x[i][e]) & 0x7FFFFFFFu;
        if (!finite || u < 0x7F800000u) top = max(top, u);
      }
    return __reduce_max_sync(FULL, top);
  }
};

template <int IN>
__global__ void __launch_bounds__(32 * kWarps) scaled_append(const __grid_constant__ AppendArgs a) {
  const int lane = static_cast<int>(threadIdx.x & 31), col = static_cast<int>(blockIdx.x);
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  if (col == 0 && blockIdx.y == 0) {  // every sequence is checked once
    uint32_t bits = 0;
    for (int b = static_cast<int>(threadIdx.x); b < a.B; b += 32 * kWarps) {
      int qs, n, L;
      bits |= rows_of(a, b, qs, n, L);
    }
    if (bits) atomicOr(&g_scaled_err, bits);
  }
  const int g = static_cast<int>(blockIdx.y) * kWarps + static_cast<int>(threadIdx.x >> 5);
  if (g >= a.Hkv) return;
  // the last sequence whose columns start at or before this one
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const unsigned m = __ballot_sync(FULL, b < hi && column_of(a, b) <= col);
    // (q_start out of order.  A tile may then have another sequence's column, or none: it is not
    // stored, and the sequence that is out of order is flagged.  No tile has two.)
    if (m == 0) return;
    lo += (31 - __clz(m)) * step;
    hi = min(lo + step, hi);
  }
  int qs, n, L;
  rows_of(a, lo, qs, n, L);
  const int first = L - n, j = first / PA_BLOCK_SIZE + col - column_of(a, lo);
  if (n == 0 || j < first / PA_BLOCK_SIZE || j > (L - 1) / PA_BLOCK_SIZE) return;
  const int64_t blk = a.block_tables[static_cast<size_t>(lo) * a.max_blocks + j];
  if (blk < 0 || blk >= a.num_blocks) {
    if (lane == 0) atomicOr(&g_scaled_err, PA_DEVERR_BLOCK_RANGE);
    return;
  }
  const size_t tile = blk * a.Hkv + g;
  // rows r0 .. r1 - 1 of the block are new; a half warp takes every other one
  const int r0 = max(0, first - j * PA_BLOCK_SIZE), r1 = min(PA_BLOCK_SIZE, L - j * PA_BLOCK_SIZE);
  const int half = lane >> 4, c = 8 * (lane & 15);
  const float old[2] = {r0 > 0 ? a.ks[tile] : 0.f, r0 > 0 ? a.vs[tile] : 0.f};
  Rows<IN> x[2];
  auto load = [&](int v) {
    const int64_t stride = v ? a.v_stride : a.k_stride;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 2 * i + half;
      const size_t t = static_cast<size_t>(qs) + (j * PA_BLOCK_SIZE + r - first);
      x[v].load(i, v ? a.v : a.k, t * stride + static_cast<size_t>(g) * kDim + c, r >= r0 && r < r1);
    }
  };
  load(0);
  if constexpr (IN != PA_DTYPE_F32) load(1);
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    if constexpr (IN == PA_DTYPE_F32) {
      if (v == 1) load(1);
    }
    uint32_t top = x[v].largest(false);
    if (top >= 0x7F800000u) top = x[v].largest(true);  // of the finite ones
    // 448 = 1.75 x 2^8: the exponent less 8, one more for fractions above 1.75
    float want = 0.f;
    if (top > 0) {
      const int e = max(-126, static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0));
      want = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    }
    float s = fmaxf(want, old[v]);  // (a NaN that stands there counts as none)
    if (!(s > 0.f)) s = 1.f;
    const float inv = 1.f / s;
    uint8_t* dst = (v ? a.vc : a.kc) + tile * (PA_BLOCK_SIZE * kDim) + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 2 * i + half;
      float y[8];
      x[v].get(i, y);
      if (r >= r0 && r < r1) *reinterpret_cast<uint2*>(dst + r * kDim) = encode8(y, inv);
    }
    if (r0 > 0 && s > old[v]) {  // the rows that stay, under a larger scale
#pragma unroll 1
      for (int r = half; r < r0; r += 2) {
        uint2* at = reinterpret_cast<uint2*>(dst + r * kDim);
        const uint2 w = *at;
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = dev::unpack2<__half>(
              dev::e4m3x2_to<__half>(static_cast<uint16_t>((e < 2 ? w.x : w.y) >> (16 * (e & 1)))));
          y[2 * e] = f.x;
          y[2 * e + 1] = f.y;
        }
        *at = encode8(y, old[v] * inv);
      }
    }
    if (lane == 0) (v ? a.vs : a.ks)[tile] = s;
  }
}

}  // namespace

pa_status launch_scaled_append(const ScaledAppendLaunch& l, const pa_cache_desc* d, void* stream) {
  AppendArgs a;
  a.k = l.k;
  a.v = l.v;
  a.k_stride = l.k_stride;
  a.v_stride = l.v_stride;
  a.q_start = l.q_start;
  a.block_tables = l.block_tables;
  a.context_lens = l.context_lens;
  a.kc = static_cast<uint8_t*>(l.k_cache);
  a.vc = static_cast<uint8_t*>(l.v_cache);
  a.ks = l.k_scale;
  a.vs = l.v_scale;
  a.T = l.T;
  a.B = l.B;
  a.Hkv = d->num_kv_heads;
  a.max_blocks = l.max_blocks;
  a.num_blocks = d->num_blocks;
  const auto kernel = l.in_dtype == PA_DTYPE_F16    ? scaled_append<PA_DTYPE_F16>
                      : l.in_dtype == PA_DTYPE_BF16 ? scaled_append<PA_DTYPE_BF16>
                                                    : scaled_append<PA_DTYPE_F32>;
  const dim3 grid(static_cast<unsigned>(l.T / PA_BLOCK_SIZE + 2 * l.B), static_cast<unsigned>((a.Hkv + kWarps - 1) / kWarps));
  cudaError_t e = launch_dependent(kernel, grid, dim3(32 * kWarps), 0, static_cast<cudaStream_t>(stream), a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_block_scaled_append launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

pa_status read_errors_scaled_cache(uint32_t* flags, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_scaled_err, sizeof(v));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_scaled_err, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_device_errors: %s", cudaGetErrorString(e));
  *flags = v;
  return PA_OK;
}

}  // namespace pa
