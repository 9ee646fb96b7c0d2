// Verification of drafted tokens against the target's probabilities, from given
// random numbers, for sm_103a ("LLM推理引擎深度实战：从PagedAttention到分布式推理
// 部署", 6.1: the target model checks the draft's tokens in one pass).
//
// Node 0 is accepted.  A chain with the draft's distribution q accepts node i's
// child x when u q[x] < p[x], and draws from max(p - q, 0) behind the first
// refusal; without one, the children of an accepted node are tried in order, x
// accepted when u (1 - S) < p[x], S what the refused ones had, and the draw is
// from p without them.  Either way accepted and drawn tokens are distributed as p.
//
// A drawn token is the first whose cumulated weight passes u0 times the sum.
// Neighbouring sums of a large vocabulary differ by less than float32 sums are
// off, and a sum's order is the split's, so weights are taken as multiples of
// 2^-44 in 64-bit integers (p - q too, exactly): any order gives the same
// sum, and any split the same token.  A probability's integer comes out of four
// float32 additions, its upper and its lower 22 bits as the mantissas of x + 2 and of
// what that left + 1.5 x 2^-21 (ulps 2^-22 and 2^-44), so that a pair of values costs 13
// instructions; with shifts of 64-bit integers it was 40, 106 us in the batch of 256
// below, and float64 additions would take longer than the row.
//
// One cluster of CTAs per sequence, so that one row is read by several SMs and
// the sums meet in distributed shared memory, in one launch without a workspace.
// Every CTA finds the accepted path by itself (a few gathers, from L2 for all
// but the first), then sums its share of the row; after one cluster barrier
// each knows where the threshold lies, and the warp whose share holds it reads one
// batch of 256 values again, whose sum it had kept.  (A scan of its whole share took
// longer than the sums: 106 us for 55 in the batch below.)
// 256 chains over 128000 tokens, two tables: 53 us, 73 % of the copy rate; 48 trees of 9
// to 26 nodes over 65521: 13 us; one chain of 5 over 32000: 9 us, which are the launch
// of a cluster and the gathers, path, sums and scan one after another.
#include <cooperative_groups.h>

#include <algorithm>
#include <utility>

#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

namespace cg = cooperative_groups;

__device__ uint32_t g_verify_err;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;  // of a CTA at most
constexpr int kNodes = 1024;  // of a sequence at most
constexpr int kMaxCluster = 8;
constexpr int kAhead = 8;     // 32-value rows of a batch: on their way before the first is used
constexpr int kBatch = 32 * kAhead, kBatches = 32;  // of a warp's share at most

struct VerifyArgs {
  const int64_t* tokens;
  const float* target;
  const float* draft;
  int64_t target_stride, draft_stride;
  int32_t V;
  const float* uniform;
  const int32_t* parents;
  const int32_t* q_start;
  int32_t T, max_path;
  int32_t share;  // values of a warp, a multiple of 32
  int32_t* path;
  int32_t* path_len;
  int64_t* next_token;
};

// A probability, taken into 0 .. 1 (NaN as 0), in units of 2^-44, to nearest even:
// 2^22 (hi - kTwo) + lo - kSmall.
constexpr uint32_t kTwo = 0x40000000u, kSmall = 0x35400000u;  // 2, 1.5 x 2^-21
__device__ __forceinline__ void fixed44(float p, uint32_t& hi, uint32_t& lo) {
  const float t = __fadd_rn(p, 2.f);
  const float rest = __fadd_rn(p, -__fadd_rn(t, -2.f));  // exact
  hi = __float_as_uint(t);
  lo = __float_as_uint(__fadd_rn(rest, __uint_as_float(kSmall)));
}
// Sums of upper and lower parts as one.
__device__ __forceinline__ uint64_t join44(uint32_t up, uint32_t down) {
  return (static_cast<uint64_t>(up) << 22) + static_cast<uint64_t>(static_cast<int64_t>(static_cast<int32_t>(down)));
}
// A weight p - q, 0 where it is not above that.
__device__ __forceinline__ uint64_t weight44(float p, float q) {
  p = __saturatef(p);
  q = __saturatef(q);
  if (!(p > q)) return 0ull;
  uint32_t ph, pl, qh, ql;
  fixed44(p, ph, pl);
  fixed44(q, qh, ql);
  return join44(ph - qh, pl - ql);
}

// floor(u total) exactly, total - 1 at most, 0 for a u that is no number or not above 0:
// a whole sum is above u total where it is above that.  (A float64 product, 53 bits of the 24
// + 45 and more, can reach the next whole number.)  u = m 2^-s, s >= 24 as u < 1.
__device__ __forceinline__ uint64_t threshold(float u, uint64_t total) {
  if (!(u > 0.f)) return 0ull;
  if (u >= 1.f) return total - 1;
  const uint32_t bits = __float_as_uint(u), e = max(bits >> 23, 1u);
  const uint64_t m = (bits & 0x7FFFFFu) | (bits >> 23 ? 0x800000u : 0u);
  const int s = 150 - static_cast<int>(e);
  const uint64_t hi = __umul64hi(total, m), lo = total * m;  // (2^87 at most)
  if (s < 64) return hi << (64 - s) | lo >> s;
  return s < 128 ? hi >> (s - 64) : 0ull;
}

__global__ void __launch_bounds__(kThreads) draft_verify(const __grid_constant__ VerifyArgs a) {
  __shared__ float node_p[kNodes], node_u[kNodes];
  __shared__ int32_t node_parent[kNodes];
  __shared__ int32_t node_token[kNodes];  // -1: outside the vocabulary
  __shared__ uint8_t node_hit[kNodes];    // accepted if no sibling before it was tried
  __shared__ int32_t gone_token[kNodes];  // the refused tokens of the last node's children, each once
  __shared__ float gone_p[kNodes];
  __shared__ uint64_t batch_sum[kWarps][kBatches], warp_sum[kWarps], cta_sum[2][kMaxCluster];
  __shared__ int walk[4];  // last accepted node; refused one of its children; accepted nodes; tokens gone
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int b = static_cast<int>(blockIdx.x) / C, tid = static_cast<int>(threadIdx.x);
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5, lane = tid & 31, wid = tid >> 5;
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  const bool report = rank == 0;
  int qs = a.q_start[b], n = a.q_start[b + 1] - qs;
  if (qs < 0 || n < 0 || n > kNodes || qs > a.T - n) {
    if (report && tid == 0) atomicOr(&g_verify_err, PA_DEVERR_QUERY_RANGE);
    qs = n = 0;
  }
  int32_t* path = a.path + static_cast<size_t>(b) * a.max_path;
  if (n == 0) {  // (the same for the whole cluster)
    if (report) {
      for (int i = tid; i < a.max_path; i += threads) path[i] = -1;
      if (tid == 0) {
        a.path_len[b] = 0;
        a.next_token[b] = -1;
      }
    }
    return;
  }
  auto running = cluster.barrier_arrive();  // no CTA writes to one that has not begun
  // ---- the accepted path -----------------------------------------------------
  for (int i = tid; i < n; i += threads) {
    int parent = i - 1;
    int64_t x = -1;
    float p = 0.f, q = 0.f;
    if (i > 0) {
      uint32_t err = 0;
      if (a.parents) {
        parent = a.parents[qs + i];
        if (parent < -1 || parent >= i) {
          err = PA_DEVERR_TREE;
          parent = -1;
        }
      }
      x = a.tokens[qs + i];
      if (x < 0 || x >= a.V) {
        err = PA_DEVERR_TREE;
        x = -1;
      } else if (parent >= 0) {
        const size_t row = static_cast<size_t>(qs + parent);
        p = a.target[row * a.target_stride + x];
        if (a.draft) q = a.draft[row * a.draft_stride + x];
      }
      if (err && report) atomicOr(&g_verify_err, err);
    }
    node_parent[i] = parent;
    node_token[i] = static_cast<int32_t>(x);
    const float u = a.uniform[qs + i];
    p = __saturatef(p);
    node_p[i] = p;
    node_u[i] = u;
    node_hit[i] = x >= 0 && static_cast<double>(u) * (a.draft ? static_cast<double>(__saturatef(q)) : 1.0) < static_cast<double>(p);
  }
  __syncthreads();
  if (wid == 0) {
    int cur = 0, len = 1, gone = 0;
    bool refused = false;
    if (report && lane == 0) path[0] = 0;
#pragma unroll 1
    while (len < a.max_path) {
      // the children of cur, in order, up to the first accepted one
      double rest = 1.0;
      int next = -1;
      refused = false;
      gone = 0;
#pragma unroll 1
      for (int c0 = cur + 1; c0 < n && next < 0; c0 += 32) {
        if (!a.parents && c0 > cur + 1) break;  // a chain: one child
        const int c = c0 + lane;
        unsigned kids = __ballot_sync(FULL, c < n && node_parent[c] == cur);
#pragma unroll 1
        while (kids && next < 0) {
          const int k = c0 + __ffs(kids) - 1, x = node_token[k];
          kids &= kids - 1;
          // a token that was refused before
          bool twin = false;
          for (int s = lane; s < gone; s += 32) twin |= gone_token[s] == x;
          if (x >= 0 && !__any_sync(FULL, twin)) {
            const float p = node_p[k];
            if (gone == 0 ? node_hit[k] != 0 : static_cast<double>(node_u[k]) * rest < static_cast<double>(p)) {
              next = k;
            } else {
              if (a.parents) rest -= static_cast<double>(p);
              if (lane == 0) {
                gone_token[gone] = x;
                gone_p[gone] = p;
              }
              ++gone;
              __syncwarp();
            }
          }
          if (next < 0) refused = true;
        }
      }
      if (next < 0) break;
      cur = next;
      refused = false;
      gone = 0;
      if (report && lane == 0) path[len] = cur;
      ++len;
    }
    if (lane == 0) {
      walk[0] = cur;
      walk[1] = refused;
      walk[2] = len;
      walk[3] = gone;
    }
  }
  __syncthreads();
  const int last = walk[0], len = walk[2];
  if (report) {
    for (int i = len + tid; i < a.max_path; i += threads) path[i] = -1;
    if (tid == 0) a.path_len[b] = len;
  }
  // ---- the drawn token ---------------------------------------------------------
  const float* prow = a.target + static_cast<size_t>(qs + last) * a.target_stride;
  const float* qrow = walk[1] && a.draft ? a.draft + static_cast<size_t>(qs + last) * a.draft_stride : nullptr;
  int gone = a.draft ? 0 : walk[3];  // the refused children's tokens have no weight
  const int lo = (rank * warps + wid) * a.share, hi = min(lo + a.share, a.V);
  uint64_t total = 0, before = 0, t = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = 0;  // of the warp's share, as are the batches'
    auto add = [&](auto with_q) {
      auto batch = [&](int i0, auto whole) {
        float p[kAhead], q[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int v = lo + i0 * kBatch + 32 * i + lane;
          p[i] = whole || v < hi ? __ldg(prow + v) : 0.f;
          q[i] = with_q && (whole || v < hi) ? __ldg(qrow + v) : 0.f;
        }
        // (2^22 at most to a step, 2^30 to the warp's batch)
        uint32_t up = 0, down = 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float x = __saturatef(p[i]), y = with_q ? __saturatef(q[i]) : 0.f;
          uint32_t xh, xl, yh = kTwo, yl = kSmall;
          fixed44(x, xh, xl);
          if (with_q) fixed44(y, yh, yl);
          up += x > y ? xh - yh : 0u;
          down += x > y ? xl - yl : 0u;
        }
        const uint64_t all = join44(__reduce_add_sync(FULL, up), __reduce_add_sync(FULL, down));
        if (lane == 0) batch_sum[wid][i0] = all;
        sum += all;
      };
      int i0 = 0;
#pragma unroll 1
      for (; lo + (i0 + 1) * kBatch <= hi; ++i0) batch(i0, std::true_type{});
      if (lo + i0 * kBatch < hi) batch(i0, std::false_type{});
    };
    if (qrow)
      add(std::true_type{});
    else
      add(std::false_type{});
    __syncwarp();
    for (int k = 0; k < gone; ++k) {
      const int v = gone_token[k] - lo;
      if (v < 0 || v >= hi - lo) continue;
      const uint64_t w = weight44(gone_p[k], 0.f);
      if (lane == 0) batch_sum[wid][v / kBatch] -= w;
      sum -= w;
    }
    if (lane == 0) warp_sum[wid] = sum;
    __syncthreads();
    if (pass == 0) cluster.barrier_wait(std::move(running));
    if (tid < C) {
      uint64_t mine = 0;
      for (int w = 0; w < warps; ++w) mine += warp_sum[w];
      *cluster.map_shared_rank(&cta_sum[pass][rank], tid) = mine;
    }
    cluster.sync();  // (no CTA leaves before its last write from another is in)
    total = before = 0;
    for (int r = 0; r < C; ++r) {
      const uint64_t x = cta_sum[pass][r];
      if (r < rank) before += x;
      total += x;
    }
    if (total > 0 || !(qrow || gone > 0)) break;
    qrow = nullptr;  // nothing is left: the target's row as it is
    gone = 0;
  }
  if (total == 0) {
    if (report && tid == 0) {
      atomicOr(&g_verify_err, PA_DEVERR_TREE);
      a.next_token[b] = -1;
    }
    return;
  }
  t = threshold(node_u[0], total);
  for (int w = 0; w < wid; ++w) before += warp_sum[w];
  if (t < before || t - before >= warp_sum[wid]) return;
  // the warp that holds it: the batch, its row of 32, the value
  t -= before;
  auto scan = [&](uint64_t x) {  // of a value a lane: the first lane whose inclusive sum is above t, which loses what is before
    uint64_t inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint64_t y = __shfl_up_sync(FULL, inc, off);
      if (lane >= off) inc += y;
    }
    const int f = __ffs(__ballot_sync(FULL, inc > t)) - 1;
    t -= __shfl_sync(FULL, inc - x, f);
    return f;
  };
  const int v0 = lo + scan(lane * kBatch < hi - lo ? batch_sum[wid][lane] : 0ull) * kBatch;
  uint64_t w[kAhead], rows = 0;  // a lane's of each row; row `lane`
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int v = v0 + 32 * i + lane;
    w[i] = v < hi ? weight44(__ldg(prow + v), qrow ? __ldg(qrow + v) : 0.f) : 0ull;
    for (int k = 0; k < gone; ++k)
      if (gone_token[k] == v) w[i] = 0;
    uint64_t all = w[i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(FULL, all, off);
    if (lane == i) rows = all;
  }
  const int row = scan(rows);
  uint64_t mine = 0;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (row == i) mine = w[i];
  const int at = scan(mine);
  if (lane == 0) a.next_token[b] = v0 + 32 * row + at;
}

}  // namespace

pa_status launch_draft_verify(const VerifyLaunch& l, void* stream) {
  VerifyArgs a;
  a.tokens = l.tokens;
  a.target = l.target;
  a.draft = l.draft;
  a.target_stride = l.target_stride;
  a.draft_stride = l.draft_stride;
  a.V = l.V;
  a.uniform = l.uniform;
  a.parents = l.parents;
  a.q_start = l.q_start;
  a.T = l.T;
  a.max_path = l.max_path;
  a.path = l.path;
  a.path_len = l.path_len;
  a.next_token = l.next_token;
  // Warps of a row: 6144 in all fill the SMs (256 rows of 128000, two tables: 24 a row 54 us,
  // 64 57, 128 69; 64 rows: 96 18 us, 128 22), a batch or two each at least (200 rows of
  // 32003: 32 a row 13 us, 128 32) and 32 batches at most; in CTAs of up to 16.
  int warps = std::min({kMaxCluster * kWarps, 6144 / l.B, l.V / (2 * kBatch)});
  warps = std::max({warps, 8, (l.V + kBatches * kBatch - 1) / (kBatches * kBatch)});
  int cluster = 1;
  while (cluster * kWarps < warps) cluster *= 2;
  warps = (warps + cluster - 1) / cluster;
  a.share = (l.V + cluster * warps - 1) / (cluster * warps);
  a.share = (a.share + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(l.B) * cluster);
  cfg.blockDim = dim3(32 * warps);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, draft_verify, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_draft_verify launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

pa_status read_errors_verify(uint32_t* flags, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_verify_err, sizeof(v));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_verify_err, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_device_errors: %s", cudaGetErrorString(e));
  *flags = v;
  return PA_OK;
}

}  // namespace pa
