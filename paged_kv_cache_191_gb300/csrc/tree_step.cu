// The steps around tree attention for sm_103a: rotary positions with the
// cache write, acceptance of a drafted tree, and the move of the accepted
// rows.
//
// Rotary cache write.  A head's first rot dims are rotated in pairs by the
// angle position * inv_freq:  (x1, x2) -> (x1 c - x2 s, x1 s + x2 c) with
// c, s = factor * cos, factor * sin; the pairs are dims (i, i + rot / 2) or
// (2 i, 2 i + 1).  Queries go to q_out, rotated keys and the values to their
// slots ("LLM推理引擎深度实战：从PagedAttention到分布式推理部署", 2.2).  It is a byte
// mover, bound by HBM for prompts and by latency for a tree: each value is
// read once and written once, 16 bytes at a time, and the angles are formed
// once per token and CTA.  An angle is kept as a 64-bit fraction of a turn:
// position times the frequency's fraction, modulo one turn, is one integer
// product, exact for every position, where float32 radians at position 2^20
// would be off by 2^-4.
//
// Acceptance ([same] 6.1).  Node 0 is accepted; after an accepted node comes
// its lowest child whose drafted token is the token the model picked there.
// One CTA per sequence: every node finds in parallel whether it agrees and
// claims its parent (atomicMin in shared memory: the lowest wins, whatever the
// order), then one thread follows the claims.
//
// Commit.  Path element i's K/V row moves from the position of node path[i]
// to the i-th position of the tree.  path[i] >= i, so a copy in ascending
// order never reads a row it has overwritten; a thread owns one 16-byte
// column of the row and runs eight loads ahead of its stores.
#include "cache_rows.cuh"
#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

__device__ uint32_t g_step_err;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 64;  // rot_dim / 2

struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int64_t* positions;
  const double* inv_freq;
  const int64_t* slots;
  void* q_out;
  void* kc;
  void* vc;
  float* ks;
  float* vs;
  int32_t Hq, Hkv, D, rot, num_blocks;
  int32_t q_f32, q_bf16;                     // type of q_out for float32 inputs
  float factor;
};

// cos and sin (times factor) of pair i's angle at `pos`.  The frequency in
// turns, modulo one, as a 64-bit fraction: two 64-bit float operations per
// pair; pos * fraction wraps modulo one turn.
__device__ __forceinline__ float2 rotation(int64_t pos, double inv_freq, float factor) {
  double turns = inv_freq * 0.15915494309189535;  // 1 / (2 pi)
  turns -= floor(turns);
  const uint64_t frac = static_cast<uint64_t>(turns * 18446744073709551616.0);  // 2^64; saturates
  const int64_t ang = static_cast<int64_t>(static_cast<uint64_t>(pos) * frac);
  // [-1, 1].  (An infinite or NaN frequency, whose turns are NaN, has no angle; a
  // select in place of the product with 0 took 69 us for 65 in the 8192-token prompt.)
  const float half_turns = fmaf(static_cast<float>(turns), 0.f, static_cast<float>(ang) * 0x1p-63f);
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * factor, s * factor);
}

// 8 floats -> a 16-byte vector of 16-bit values.
template <int OUT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (OUT == PA_DTYPE_F16)
      w[e] = dev::pack2<__half>(x[2 * e], x[2 * e + 1]);
    else
      w[e] = dev::pack2<__nv_bfloat16>(x[2 * e], x[2 * e + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A unit is 16 dims of one head, two vectors of 8: in the rotated part dims
// 8 u .. and rot / 2 + 8 u .. (whichever pairing: both vectors' partners are
// in the unit), behind it 16 consecutive dims.  u counts within the head.
__device__ __forceinline__ void unit_dims(int u, int rot, int& d0, int& d1) {
  const int n = rot >> 4;
  d0 = u < n ? 8 * u : 16 * u;
  d1 = u < n ? (rot >> 1) + 8 * u : 16 * u + 8;
}
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[8], float (&y)[8], int u, int rot, const float2* cs) {
  if (u >= (rot >> 4)) return;
  if constexpr (INTER) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = cs[4 * u + e], g = cs[(rot >> 2) + 4 * u + e];
      const float a = x[2 * e], b = x[2 * e + 1], c = y[2 * e], d = y[2 * e + 1];
      x[2 * e] = a * f.x - b * f.y;
      x[2 * e + 1] = a * f.y + b * f.x;
      y[2 * e] = c * g.x - d * g.y;
      y[2 * e + 1] = c * g.y + d * g.x;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = cs[8 * u + e];
      const float a = x[e], b = y[e];
      x[e] = a * f.x - b * f.y;
      y[e] = a * f.y + b * f.x;
    }
  }
}

template <int IN>
__device__ __forceinline__ void unpack8(const uint4* raw, float (&x)[8]) {
  if constexpr (IN == PA_DTYPE_F32) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      x[4 * v] = __uint_as_float(raw[v].x);
      x[4 * v + 1] = __uint_as_float(raw[v].y);
      x[4 * v + 2] = __uint_as_float(raw[v].z);
      x[4 * v + 3] = __uint_as_float(raw[v].w);
    }
  } else {
    const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (IN == PA_DTYPE_F16)
        f = dev::unpack2<__half>(w[i]);
      else
        f = dev::unpack2<__nv_bfloat16>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <int IN>
__device__ __forceinline__ void store_q(const RopeArgs& a, size_t at, const float (&x)[8]) {
  if constexpr (IN == PA_DTYPE_F32) {
    if (a.q_f32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + at);
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + at) =
          a.q_bf16 ? pack8<PA_DTYPE_BF16>(x) : pack8<PA_DTYPE_F16>(x);
    }
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + at) = pack8<IN>(x);
  }
}

// U: units a thread takes.  KV: F16 / BF16: the CTA's units are the token's q, k and v units in order.
// FP8 / INT8: CTA row 0 quantises the token's K and V rows (amax over the
// token's heads and dims, after the rotation, in float32), the others take q.
template <int IN, int KV, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_write(const RopeArgs a) {
  constexpr bool Q8 = KV == PA_DTYPE_FP8_E4M3 || KV == PA_DTYPE_INT8;
  __shared__ float2 cs[kMaxPairs];
  __shared__ float red[33];
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();  // a dependent kernel waits for our completion itself
  const int t = static_cast<int>(blockIdx.x);
  const int upr = a.D >> 4, nq = a.Hq * upr, nk = a.Hkv * upr;
  const int64_t slot = a.slots[t];
  const int64_t pos = a.positions[t];
  const double freq = threadIdx.x < (a.rot >> 1) ? a.inv_freq[threadIdx.x] : 0.;
  auto angles = [&]() {
    if (threadIdx.x < (a.rot >> 1)) cs[threadIdx.x] = rotation(pos, freq, a.factor);
    __syncthreads();
  };
  const bool keep = slot >= 0 && slot < static_cast<int64_t>(a.num_blocks) * PA_BLOCK_SIZE;
  if (blockIdx.y == 0 && threadIdx.x == 0 && slot >= static_cast<int64_t>(a.num_blocks) * PA_BLOCK_SIZE)
    atomicOr(&g_step_err, PA_DEVERR_SLOT_RANGE);
  const int64_t blk = keep ? slot / PA_BLOCK_SIZE : 0, off = keep ? slot % PA_BLOCK_SIZE : 0;
  if constexpr (Q8) {
    if (blockIdx.y == 0) {
      angles();
      if (!keep) return;
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        const void* src = which ? a.v : a.k;
        const size_t row = static_cast<size_t>(t) * (which ? a.v_stride : a.k_stride);
        uint8_t* cache = static_cast<uint8_t*>(which ? a.vc : a.kc);
        auto values = [&](int i, float (&x)[8], float (&y)[8], int& h, int& d0, int& d1) {
          h = i / upr;
          const int u = i - h * upr;
          unit_dims(u, a.rot, d0, d1);
          dev::load8<IN>(src, row + static_cast<size_t>(h) * a.D + d0, x);
          dev::load8<IN>(src, row + static_cast<size_t>(h) * a.D + d1, y);
          if (!which) rotate<INTER>(x, y, u, a.rot, cs);
        };
        float x[8], y[8], amax = 0.f;
        int h, d0, d1;
        for (int i = threadIdx.x; i < nk; i += kRopeThreads) {
          values(i, x, y, h, d0, d1);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e]), fabsf(y[e])));
        }
        amax = dev::block_max(amax, red);
        constexpr bool I8 = KV == PA_DTYPE_INT8;
        const float scale = amax > 0.f ? __fdiv_rn(amax, I8 ? 127.0f : 448.0f) : 1.0f;
        for (int i = threadIdx.x; i < nk; i += kRopeThreads) {
          if (nk > kRopeThreads) values(i, x, y, h, d0, d1);  // else still in registers
          auto codes = [&](const float (&z)[8]) {
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e >> 2] |= dev::encode_q8<I8>(__fdiv_rn(z[e], scale)) << (8 * (e & 3));
            return make_uint2(w[0], w[1]);
          };
          const size_t dst = ((static_cast<size_t>(blk) * a.Hkv + h) * PA_BLOCK_SIZE + off) * a.D;
          *reinterpret_cast<uint2*>(cache + dst + d0) = codes(x);
          *reinterpret_cast<uint2*>(cache + dst + d1) = codes(y);
        }
        if (threadIdx.x == 0) (which ? a.vs : a.ks)[slot] = scale;
        __syncthreads();  // `red` is reused by the next tensor
      }
      return;
    }
  }
  // Every unit's loads are in flight before the angles are formed, and before
  // the slot is known (rows without one are read too, and dropped).
  constexpr int NV = IN == PA_DTYPE_F32 ? 2 : 1;  // 16-byte vectors per 8 values
  const int first = (static_cast<int>(blockIdx.y) - (Q8 ? 1 : 0)) * (U * kRopeThreads) + static_cast<int>(threadIdx.x);
  const int total = nq + (Q8 ? 0 : 2 * nk);
  uint4 raw[U][2][NV];
#pragma unroll
  for (int w = 0; w < U; ++w) {
    const int i = first + w * kRopeThreads;
    if (i >= total) continue;
    const int kind = i < nq ? 0 : i < nq + nk ? 1 : 2;  // q, k, v
    const int j = i - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk), h = j / upr;
    int d0, d1;
    unit_dims(j - h * upr, a.rot, d0, d1);
    const size_t row = static_cast<size_t>(t) * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                       static_cast<size_t>(h) * a.D;
    const uint8_t* src = static_cast<const uint8_t*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
#pragma unroll
    for (int x = 0; x < NV; ++x) {
      raw[w][0][x] = reinterpret_cast<const uint4*>(src + (row + d0) * (2 * NV))[x];
      raw[w][1][x] = reinterpret_cast<const uint4*>(src + (row + d1) * (2 * NV))[x];
    }
  }
  angles();
#pragma unroll
  for (int w = 0; w < U; ++w) {
    const int i = first + w * kRopeThreads;
    if (i >= total || (i >= nq && !keep)) continue;
    const int kind = i < nq ? 0 : i < nq + nk ? 1 : 2;
    const int j = i - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk), h = j / upr, u = j - h * upr;
    int d0, d1;
    unit_dims(u, a.rot, d0, d1);
    uint16_t* dst = nullptr;
    if constexpr (!Q8)
      dst = static_cast<uint16_t*>(kind == 1 ? a.kc : a.vc) +
            ((static_cast<size_t>(blk) * a.Hkv + h) * PA_BLOCK_SIZE + off) * a.D;
    if constexpr (IN == KV) {
      if (kind == 2) {  // V rows are copied bit for bit
        *reinterpret_cast<uint4*>(dst + d0) = raw[w][0][0];
        *reinterpret_cast<uint4*>(dst + d1) = raw[w][1][0];
        continue;
      }
    }
    float x[8], y[8];
    unpack8<IN>(raw[w][0], x);
    unpack8<IN>(raw[w][1], y);
    if (kind < 2) rotate<INTER>(x, y, u, a.rot, cs);
    if (kind == 0) {
      const size_t at = static_cast<size_t>(t) * a.q_out_stride + static_cast<size_t>(h) * a.D;
      store_q<IN>(a, at + d0, x);
      store_q<IN>(a, at + d1, y);
    } else if constexpr (!Q8) {
      *reinterpret_cast<uint4*>(dst + d0) = pack8<KV>(x);
      *reinterpret_cast<uint4*>(dst + d1) = pack8<KV>(y);
    }
  }
}

// ---- acceptance ------------------------------------------------------------
constexpr int kAcceptThreads = 128;
constexpr int kClaims = 2048;  // nodes whose claims fit in shared memory

__global__ void __launch_bounds__(kAcceptThreads)
    tree_accept(const int64_t* __restrict__ draft, const int64_t* __restrict__ target,
                const int32_t* __restrict__ parents, const int32_t* __restrict__ q_start, int T, int max_path,
                int32_t* __restrict__ path, int32_t* __restrict__ path_len, int64_t* __restrict__ next_token) {
  __shared__ int claim[kClaims];
  __shared__ int len_s;
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  const int b = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  int qs = q_start[b], n = q_start[b + 1] - qs;
  if (qs < 0 || n < 0 || qs > T - n) {
    if (tid == 0) atomicOr(&g_step_err, PA_DEVERR_QUERY_RANGE);
    qs = n = 0;
  }
  int32_t* out = path + static_cast<size_t>(b) * max_path;
  draft += qs;
  target += qs;
  parents += qs;
  // node i agrees with its parent's pick; -1: no parent
  auto parent_of = [&](int i) {
    const int p = parents[i];
    if (p < -1 || p >= i) {
      atomicOr(&g_step_err, PA_DEVERR_TREE);
      return -1;
    }
    return p;
  };
  int len = 0;
  if (n > 0 && n <= kClaims) {
    for (int i = tid; i < n; i += kAcceptThreads) claim[i] = INT32_MAX;
    __syncthreads();
    for (int i = tid; i < n; i += kAcceptThreads) {
      if (i == 0) continue;
      const int p = parent_of(i);
      if (p >= 0 && draft[i] == target[p]) atomicMin(&claim[p], i);
    }
    __syncthreads();
    if (tid == 0) {
      int cur = 0;
      for (;;) {
        out[len++] = cur;
        const int nx = claim[cur];
        if (nx == INT32_MAX || len >= max_path) break;
        cur = nx;
      }
      path_len[b] = len;
      next_token[b] = target[cur];
      len_s = len;
    }
  } else if (n > 0) {  // a wide tree: every step scans the nodes behind the current one
    int cur = 0;
    for (;;) {
      if (tid == 0) {
        out[len] = cur;
        claim[0] = INT32_MAX;
      }
      ++len;
      __syncthreads();
      const int64_t want = target[cur];
      for (int i = cur + 1 + tid; i < n; i += kAcceptThreads)
        if (parents[i] == cur && draft[i] == want) {
          atomicMin(&claim[0], i);
          break;
        }
      __syncthreads();
      const int nx = claim[0];
      __syncthreads();
      if (nx == INT32_MAX || len >= max_path) break;
      cur = nx;
    }
    for (int i = 1 + tid; i < n; i += kAcceptThreads) parent_of(i);  // flags what is malformed
    if (tid == 0) {
      path_len[b] = len;
      next_token[b] = target[cur];
      len_s = len;
    }
  } else if (tid == 0) {
    path_len[b] = 0;
    next_token[b] = -1;
    len_s = 0;
  }
  __syncthreads();
  for (int i = len_s + tid; i < max_path; i += kAcceptThreads) out[i] = -1;
}

// ---- commit ----------------------------------------------------------------
constexpr int kCommitThreads = 256;
constexpr int kMoves = 256;  // path elements staged at a time
constexpr int kAhead = 8;

struct CommitArgs {
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* q_start;
  const int32_t* path;
  const int32_t* path_len;
  int32_t* new_lens;
  int32_t max_blocks, num_blocks, max_path, Hkv, row_bytes;  // row_bytes: one head's row
};

__global__ void __launch_bounds__(kCommitThreads) tree_commit(const CommitArgs a) {
  __shared__ int2 at[kMoves];  // (source, destination) slot of a move; slots fit 32 bits (checked on the host)
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  const int b = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  const int L = a.context_lens[b], n = a.q_start[b + 1] - a.q_start[b], len = a.path_len[b];
  const int32_t* path = a.path + static_cast<size_t>(b) * a.max_path;
  const int32_t* table = a.block_tables + static_cast<size_t>(b) * a.max_blocks;
  uint32_t err = 0;
  if (n < 0)
    err = PA_DEVERR_QUERY_RANGE;
  else if (L < n || L > a.max_blocks * PA_BLOCK_SIZE)
    err = PA_DEVERR_CONTEXT_LEN;
  else if (len < 0 || len > n || len > a.max_path)
    err = PA_DEVERR_TREE;
  const int first = L - n;  // position of node 0
  auto block_of = [&](int pos) {
    const int id = table[pos / PA_BLOCK_SIZE];
    if (id < 0 || id >= a.num_blocks) {
      err |= PA_DEVERR_BLOCK_RANGE;
      return 0;
    }
    return id;
  };
  // the whole path is checked before anything moves: a bad one moves nothing
  auto stage = [&](int i0) {
    for (int i = i0 + tid; i < min(len, i0 + kMoves); i += kCommitThreads) {
      const int p = path[i], before = i ? path[i - 1] : -1;
      if (p < i || p >= n || p <= before) {
        err |= PA_DEVERR_TREE;
        continue;
      }
      const int s = first + p, d = first + i;
      at[i - i0] = make_int2(block_of(s) * PA_BLOCK_SIZE + s % PA_BLOCK_SIZE,
                             block_of(d) * PA_BLOCK_SIZE + d % PA_BLOCK_SIZE);
    }
  };
  if (!err)
    for (int i0 = 0; i0 < len; i0 += kMoves) stage(i0);
  if (__syncthreads_or(err != 0)) {
    if (err) atomicOr(&g_step_err, err);
    if (tid == 0 && blockIdx.y == 0 && a.new_lens) a.new_lens[b] = L;
    return;
  }
  if (tid == 0 && blockIdx.y == 0 && a.new_lens) a.new_lens[b] = first + len;
  const int cpr = a.row_bytes >> 4, cols = a.Hkv * cpr;  // 16-byte columns of one tensor's token row
  const int col = static_cast<int>(blockIdx.y) * kCommitThreads + tid;
  const bool isv = col >= cols;
  const int c = isv ? col - cols : col, h = c / cpr;
  uint8_t* cache = isv ? a.vc : a.kc;
  const size_t blk_bytes = static_cast<size_t>(a.Hkv) * PA_BLOCK_SIZE * a.row_bytes;
  const size_t in_blk = static_cast<size_t>(h) * PA_BLOCK_SIZE * a.row_bytes + static_cast<size_t>(c - h * cpr) * 16;
  auto addr = [&](int slot) {
    return reinterpret_cast<uint4*>(cache + static_cast<size_t>(slot / PA_BLOCK_SIZE) * blk_bytes + in_blk +
                                    static_cast<size_t>(slot % PA_BLOCK_SIZE) * a.row_bytes);
  };
  for (int i0 = 0; i0 < len; i0 += kMoves) {
    if (len > kMoves) {  // else the check staged them all
      __syncthreads();
      stage(i0);
      __syncthreads();
    }
    const int m = min(len - i0, kMoves);
    if (col < 2 * cols) {
      for (int i = 0; i < m; i += kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i + k < m && at[i + k].x != at[i + k].y) v[k] = *addr(at[i + k].x);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i + k < m && at[i + k].x != at[i + k].y) *addr(at[i + k].y) = v[k];
      }
    }
    if (a.ks && blockIdx.y == 0 && tid < 2) {  // one thread per scale array, in order
      float* s = tid ? a.vs : a.ks;
      for (int i = 0; i < m; ++i) s[at[i].y] = s[at[i].x];
    }
  }
}

// One unit a thread while the tokens alone do not fill the SMs; four (their
// loads in flight together, the angles formed once) when they do.
template <int IN, int KV>
cudaError_t launch_rope_t(const RopeArgs& a, bool inter, int64_t T, cudaStream_t st) {
  constexpr bool Q8 = KV == PA_DTYPE_FP8_E4M3 || KV == PA_DTYPE_INT8;
  const int units = (a.D >> 4) * (a.Hq + (Q8 ? 0 : 2 * a.Hkv));
  const bool wide = T >= 2 * sm_count();
  const int per = kRopeThreads * (wide ? 4 : 1);
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>((units + per - 1) / per + (Q8 ? 1 : 0)));
  auto kernel = wide ? (inter ? rope_write<IN, KV, true, 4> : rope_write<IN, KV, false, 4>)
                     : (inter ? rope_write<IN, KV, true, 1> : rope_write<IN, KV, false, 1>);
  return launch_dependent(kernel, grid, dim3(kRopeThreads), 0, st, a);
}

}  // namespace

pa_status launch_rope_write(const RopeLaunch& l, const pa_cache_desc* d, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  RopeArgs a;
  a.q = l.q;
  a.k = l.k;
  a.v = l.v;
  a.q_stride = l.q_stride;
  a.k_stride = l.k_stride;
  a.v_stride = l.v_stride;
  a.q_out_stride = l.q_out_stride;
  a.positions = l.positions;
  a.inv_freq = l.inv_freq;
  a.slots = l.slots;
  a.q_out = l.q_out;
  a.kc = l.k_cache;
  a.vc = l.v_cache;
  a.ks = l.k_scale;
  a.vs = l.v_scale;
  a.Hq = l.Hq;
  a.Hkv = d->num_kv_heads;
  a.D = d->head_dim;
  a.rot = l.rot_dim;
  a.num_blocks = d->num_blocks;
  a.q_f32 = l.q_out_dtype == PA_DTYPE_F32;
  a.q_bf16 = l.q_out_dtype == PA_DTYPE_BF16;
  a.factor = l.factor;
  cudaError_t e = cudaSuccess;
  const bool inter = l.interleaved != 0;
  switch (d->kv_dtype) {
    case PA_DTYPE_F16:
      if (l.in_dtype == PA_DTYPE_F16)
        e = launch_rope_t<PA_DTYPE_F16, PA_DTYPE_F16>(a, inter, l.T, st);
      else
        e = launch_rope_t<PA_DTYPE_F32, PA_DTYPE_F16>(a, inter, l.T, st);
      break;
    case PA_DTYPE_BF16:
      if (l.in_dtype == PA_DTYPE_BF16)
        e = launch_rope_t<PA_DTYPE_BF16, PA_DTYPE_BF16>(a, inter, l.T, st);
      else
        e = launch_rope_t<PA_DTYPE_F32, PA_DTYPE_BF16>(a, inter, l.T, st);
      break;
    case PA_DTYPE_FP8_E4M3:
      if (l.in_dtype == PA_DTYPE_F16)
        e = launch_rope_t<PA_DTYPE_F16, PA_DTYPE_FP8_E4M3>(a, inter, l.T, st);
      else if (l.in_dtype == PA_DTYPE_BF16)
        e = launch_rope_t<PA_DTYPE_BF16, PA_DTYPE_FP8_E4M3>(a, inter, l.T, st);
      else
        e = launch_rope_t<PA_DTYPE_F32, PA_DTYPE_FP8_E4M3>(a, inter, l.T, st);
      break;
    default:
      if (l.in_dtype == PA_DTYPE_F16)
        e = launch_rope_t<PA_DTYPE_F16, PA_DTYPE_INT8>(a, inter, l.T, st);
      else if (l.in_dtype == PA_DTYPE_BF16)
        e = launch_rope_t<PA_DTYPE_BF16, PA_DTYPE_INT8>(a, inter, l.T, st);
      else
        e = launch_rope_t<PA_DTYPE_F32, PA_DTYPE_INT8>(a, inter, l.T, st);
      break;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_rope_cache_write launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

pa_status launch_tree_accept(const int64_t* draft, const int64_t* target, const int32_t* parents,
                             const int32_t* q_start, int32_t T, int32_t B, int32_t max_path, int32_t* path,
                             int32_t* path_len, int64_t* next_token, void* stream) {
  cudaError_t e = launch_dependent(tree_accept, dim3(static_cast<unsigned>(B)), dim3(kAcceptThreads), 0,
                                   static_cast<cudaStream_t>(stream), draft, target, parents, q_start, T, max_path,
                                   path, path_len, next_token);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_tree_accept launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

pa_status launch_tree_commit(const CommitLaunch& l, const pa_cache_desc* d, void* stream) {
  CommitArgs a;
  a.kc = static_cast<uint8_t*>(l.k_cache);
  a.vc = static_cast<uint8_t*>(l.v_cache);
  a.ks = l.k_scale;
  a.vs = l.v_scale;
  a.block_tables = l.block_tables;
  a.context_lens = l.context_lens;
  a.q_start = l.q_start;
  a.path = l.path;
  a.path_len = l.path_len;
  a.new_lens = l.new_lens;
  a.max_blocks = l.max_blocks;
  a.num_blocks = d->num_blocks;
  a.max_path = l.max_path;
  a.Hkv = d->num_kv_heads;
  a.row_bytes = d->head_dim * dtype_bytes(d->kv_dtype);
  const int cols = 2 * a.Hkv * (a.row_bytes >> 4);
  const dim3 grid(static_cast<unsigned>(l.B), static_cast<unsigned>((cols + kCommitThreads - 1) / kCommitThreads));
  cudaError_t e = launch_dependent(tree_commit, grid, dim3(kCommitThreads), 0, static_cast<cudaStream_t>(stream), a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_tree_commit launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

pa_status read_errors_tree_step(uint32_t* flags, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_step_err, sizeof(v));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_step_err, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_device_errors: %s", cudaGetErrorString(e));
  *flags = v;
  return PA_OK;
}

}  // namespace pa
