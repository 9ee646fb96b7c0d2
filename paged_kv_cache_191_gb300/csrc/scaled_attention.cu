// Attention over a block-scaled cache: one CTA per (token, kv head), its warps
// taking every eighth key, merged at the end.
#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

__device__ uint32_t g_sa_err;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 8, kDim = 128, kHeads = 8;

struct Args {
  const void* q;
  int64_t q_stride;
  const int32_t* q_start;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* out;
  int32_t B, T, Hq, Hkv, G, max_blocks, num_blocks, max_context_len, max_q_len, q_bf16, out_f32;
  float scale_log2;
};

__device__ __forceinline__ float4 codes4(uint32_t w) {
  uint32_t lo, hi;
  dev::e4m3x4_to_f16(w, lo, hi);
  const float2 a = dev::unpack2<__half>(lo), b = dev::unpack2<__half>(hi);
  return make_float4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(32 * kWarps) scaled_attention_simple(const __grid_constant__ Args a) {
  __shared__ float part[kWarps][kHeads][kDim + 2];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = blockIdx.y;
  dev::grid_dependency_wait();
  // the sequence of row blockIdx.x
  int b = 0;
  const int t = blockIdx.x;
  while (b < a.B && !(t >= a.q_start[b] && t < a.q_start[b + 1])) ++b;
  if (b == a.B) return;
  const int n = a.q_start[b + 1] - a.q_start[b], cap = min(a.max_context_len, a.max_blocks * 16);
  int L = a.context_lens[b];
  uint32_t err = 0;
  if (n > a.max_q_len || a.q_start[b] < 0 || a.q_start[b + 1] > a.T) err |= PA_DEVERR_QUERY_RANGE;
  if (L < 0 || L > cap || n > L) err |= PA_DEVERR_CONTEXT_LEN;
  if (err && threadIdx.x == 0) atomicOr(&g_sa_err, err);
  if (err & PA_DEVERR_QUERY_RANGE) return;
  L = max(0, min(L, cap));
  const int keys = L - n + (t - a.q_start[b]) + 1;
  for (int h0 = 0; h0 < a.G; h0 += kHeads) {
    const int nh = min(kHeads, a.G - h0);
    float4 q[kHeads], o[kHeads];
    float m[kHeads], l[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
      q[h] = o[h];
      m[h] = -INFINITY;
      l[h] = 0.f;
      if (h < nh) {
        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + t * a.q_stride +
                                                        static_cast<size_t>(g * a.G + h0 + h) * kDim + 4 * lane);
        const float2 u = a.q_bf16 ? dev::unpack2<__nv_bfloat16>(x.x) : dev::unpack2<__half>(x.x);
        const float2 v = a.q_bf16 ? dev::unpack2<__nv_bfloat16>(x.y) : dev::unpack2<__half>(x.y);
        q[h] = make_float4(u.x, u.y, v.x, v.y);
      }
    }
    for (int k = w; k < keys; k += kWarps) {
      int blk = a.block_tables[static_cast<size_t>(b) * a.max_blocks + k / 16];
      if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0) atomicOr(&g_sa_err, PA_DEVERR_BLOCK_RANGE);
        blk = 0;
      }
      const size_t tile = static_cast<size_t>(blk) * a.Hkv + g, at = (tile * 16 + k % 16) * kDim + 4 * lane;
      const float4 K = codes4(*reinterpret_cast<const uint32_t*>(a.kc + at));
      const float4 V = codes4(*reinterpret_cast<const uint32_t*>(a.vc + at));
      const float ks = a.ks[tile] * a.scale_log2, vs = a.vs[tile];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        float s = q[h].x * K.x + q[h].y * K.y + q[h].z * K.z + q[h].w * K.w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(FULL, s, off);
        s *= ks;
        const float mm = fmaxf(m[h], s), f = m[h] == mm ? 1.f : exp2f(m[h] - mm);
        const float p = s == -INFINITY ? 0.f : exp2f(s - mm), y = p * vs;
        m[h] = mm;
        l[h] = l[h] * f + p;
        o[h] = make_float4(o[h].x * f + y * V.x, o[h].y * f + y * V.y, o[h].z * f + y * V.z, o[h].w * f + y * V.w);
      }
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      *reinterpret_cast<float2*>(&part[w][h][4 * lane]) = make_float2(o[h].x, o[h].y);
      *reinterpret_cast<float2*>(&part[w][h][4 * lane + 2]) = make_float2(o[h].z, o[h].w);
      if (lane == 0) {
        part[w][h][kDim] = m[h];
        part[w][h][kDim + 1] = l[h];
      }
    }
    __syncthreads();
    for (int h = w; h < nh; h += kWarps) {
      float M = -INFINITY, sum = 0.f;
      for (int i = 0; i < kWarps; ++i) M = fmaxf(M, part[i][h][kDim]);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < kWarps; ++i) {
        const float mi = part[i][h][kDim];
        if (mi == -INFINITY && part[i][h][kDim + 1] == 0.f) continue;  // (a NaN score leaves NaN in l)
        const float f = mi == M ? 1.f : exp2f(mi - M);
        sum += f * part[i][h][kDim + 1];
        for (int e = 0; e < 4; ++e) acc[e] += f * part[i][h][4 * lane + e];
      }
      const size_t at = (static_cast<size_t>(t) * a.Hq + g * a.G + h0 + h) * kDim + 4 * lane;
      const float inv = keys > 0 ? 1.f / sum : 0.f;
      for (int e = 0; e < 4; ++e) {
        const float y = keys > 0 ? acc[e] * inv : 0.f;
        if (a.out_f32)
          static_cast<float*>(a.out)[at + e] = y;
        else if (a.q_bf16)
          static_cast<__nv_bfloat16*>(a.out)[at + e] = __float2bfloat16(y);
        else
          static_cast<__half*>(a.out)[at + e] = __float2half(y);
      }
    }
    __syncthreads();
  }
}

}  // namespace

pa_status launch_scaled_attention(const ScaledAttentionLaunch& l, void* stream) {
  Args a;
  a.q = l.q;
  a.q_stride = l.q_stride;
  a.q_start = l.q_start;
  a.kc = static_cast<const uint8_t*>(l.k_cache);
  a.vc = static_cast<const uint8_t*>(l.v_cache);
  a.ks = l.k_scale;
  a.vs = l.v_scale;
  a.block_tables = l.block_tables;
  a.context_lens = l.context_lens;
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
  a.q_bf16 = l.q_dtype == PA_DTYPE_BF16;
  a.out_f32 = l.out_dtype == PA_DTYPE_F32;
  a.scale_log2 = l.scale * 1.4426950408889634f;
  cudaError_t e = launch_dependent(scaled_attention_simple, dim3(static_cast<unsigned>(a.T), static_cast<unsigned>(a.Hkv)),
                                   dim3(32 * kWarps), 0, static_cast<cudaStream_t>(stream), a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_block_scaled_attention launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

pa_status read_errors_scaled_attention(uint32_t* flags, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_sa_err, sizeof(v));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_sa_err, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_device_errors: %s", cudaGetErrorString(e));
  *flags = v;
  return PA_OK;
}

}  // namespace pa
