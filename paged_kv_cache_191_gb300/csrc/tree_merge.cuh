// Merge of the partial rows that attention items spanning CTAs leave, shared by
// the tree attention and the attention over block-scaled caches.
#pragma once

#include "tree_common.cuh"

namespace pa {
namespace {

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

}  // namespace
}  // namespace pa
