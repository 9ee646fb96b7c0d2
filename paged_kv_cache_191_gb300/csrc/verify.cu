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
// sum, and any split the same token.  Four integer operations per value are a
// third of what HBM leaves time for; float64 additions would take as long as the row.
//
// One cluster of CTAs per sequence, so that one row is read by several SMs and
// the sums meet in distributed shared memory, in one launch without a workspace.
// Every CTA finds the accepted path by itself (a few gathers, from L2 for all
// but the first), then sums its share of the row; after one cluster barrier
// each knows where the threshold lies, and the warp whose share holds it reads
// that share again, from L2.
#include <cooperative_groups.h>

#include <utility>

#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

namespace cg = cooperative_groups;

__device__ uint32_t g_verify_err;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kNodes = 1024;  // of a sequence at most
constexpr int kMaxCluster = 8;
constexpr int kAhead = 8;     // 32-value rows of a warp's share in flight

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

// A probability in units of 2^-44: into 0 .. 1, NaN as 0.
__device__ __forceinline__ uint64_t fixed44(float p) {
  p = fminf(fmaxf(p, 0.f), 1.f);  // (fmaxf drops a NaN)
  const uint32_t u = __float_as_uint(p);
  // mantissa x 2^(exponent - 127 - 23 + 44)
  const uint64_t m = (u & 0x7FFFFFu) | 0x800000u;
  const int sh = static_cast<int>(u >> 23) - 106;
  return sh >= 0 ? m << sh : sh > -25 ? m >> -sh : 0ull;
}

struct Node {
  float p, q, u;
  int32_t parent;
  int64_t token;
};

// The row that the next token is drawn from.
struct Row {
  const float* p;
  const float* q;  // null: nothing is taken off
  int last;        // its node, refused children of which have no weight (gone)
  bool gone;
};

__global__ void __launch_bounds__(kThreads) draft_verify(const __grid_constant__ VerifyArgs a) {
  __shared__ float node_p[kNodes], node_q[kNodes], node_u[kNodes];
  __shared__ int32_t node_parent[kNodes];
  __shared__ int32_t node_token[kNodes];  // -1: outside the vocabulary
  __shared__ uint64_t warp_sum[kWarps], cta_sum[2][kMaxCluster];
  __shared__ int walk[3];  // last accepted node; refused one of its children; accepted nodes
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int b = static_cast<int>(blockIdx.x) / C, tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 31, wid = tid >> 5;
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
      for (int i = tid; i < a.max_path; i += kThreads) path[i] = -1;
      if (tid == 0) {
        a.path_len[b] = 0;
        a.next_token[b] = -1;
      }
    }
    return;
  }
  auto running = cluster.barrier_arrive();  // no CTA writes to one that has not begun
  // ---- the accepted path -----------------------------------------------------
  for (int i = tid; i < n; i += kThreads) {
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
    node_p[i] = fminf(fmaxf(p, 0.f), 1.f);
    node_q[i] = fminf(fmaxf(q, 0.f), 1.f);
    node_u[i] = a.uniform[qs + i];
  }
  __syncthreads();
  if (wid == 0) {
    int cur = 0, len = 1;
    bool refused = false;
    if (report && lane == 0) path[0] = 0;
#pragma unroll 1
    while (len < a.max_path) {
      // the children of cur, in order, up to the first accepted one
      double rest = 1.0;
      int next = -1;
      refused = false;
#pragma unroll 1
      for (int c0 = cur + 1; c0 < n && next < 0; c0 += 32) {
        if (!a.parents && c0 > cur + 1) break;  // a chain: one child
        const int c = c0 + lane;
        unsigned kids = __ballot_sync(FULL, c < n && node_parent[c] == cur);
#pragma unroll 1
        while (kids && next < 0) {
          const int k = c0 + __ffs(kids) - 1, x = node_token[k];
          kids &= kids - 1;
          // a sibling before it with the same token
          bool twin = false;
          for (int s = cur + 1 + lane; s < k; s += 32) twin |= node_parent[s] == cur && node_token[s] == x;
          if (!__any_sync(FULL, twin) && x >= 0) {
            const double p = node_p[k], q = a.draft ? static_cast<double>(node_q[k]) : rest;
            if (static_cast<double>(node_u[k]) * q < p)
              next = k;
            else
              rest -= p;
          }
          if (next < 0) refused = true;
        }
      }
      if (next < 0) break;
      cur = next;
      refused = false;
      if (report && lane == 0) path[len] = cur;
      ++len;
    }
    if (lane == 0) {
      walk[0] = cur;
      walk[1] = refused;
      walk[2] = len;
    }
  }
  __syncthreads();
  const int last = walk[0], len = walk[2];
  if (report) {
    for (int i = len + tid; i < a.max_path; i += kThreads) path[i] = -1;
    if (tid == 0) a.path_len[b] = len;
  }
  // ---- the drawn token ---------------------------------------------------------
  const float* prow = a.target + static_cast<size_t>(qs + last) * a.target_stride;
  const float* qrow = walk[1] && a.draft ? a.draft + static_cast<size_t>(qs + last) * a.draft_stride : nullptr;
  bool gone = walk[1] && !a.draft;  // the refused children's tokens have no weight
  const int lo = (rank * kWarps + wid) * a.share, hi = min(lo + a.share, a.V);
  // whether v's weight is taken away: a child of `last` has the token
  auto taken = [&](int v) {
    for (int k = last + 1; k < n; ++k)
      if (node_parent[k] == last && node_token[k] == v) return true;
    return false;
  };
  uint64_t total = 0, before = 0, t = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = 0;
#pragma unroll 1
    for (int v0 = lo + lane; v0 < hi; v0 += 32 * kAhead) {
      float p[kAhead], q[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = v0 + 32 * i;
        p[i] = v < hi ? __ldcg(prow + v) : 0.f;
        q[i] = qrow && v < hi ? __ldcg(qrow + v) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint64_t x = fixed44(p[i]), y = qrow ? fixed44(q[i]) : 0ull;
        sum += x > y ? x - y : 0ull;
      }
    }
    if (gone) {  // each refused token once
      for (int k = last + 1 + lane; k < n; k += 32) {
        const int x = node_parent[k] == last ? node_token[k] : -1;
        if (x < lo || x >= hi) continue;
        bool twin = false;
        for (int s = last + 1; s < k; ++s) twin |= node_parent[s] == last && node_token[s] == x;
        if (!twin) sum -= fixed44(node_p[k]);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL, sum, off);
    if (lane == 0) warp_sum[wid] = sum;
    __syncthreads();
    if (pass == 0) cluster.barrier_wait(std::move(running));
    if (tid < C) {
      uint64_t mine = 0;
      for (int w = 0; w < kWarps; ++w) mine += warp_sum[w];
      *cluster.map_shared_rank(&cta_sum[pass][rank], tid) = mine;
    }
    cluster.sync();  // (no CTA leaves before its last write from another is in)
    total = before = 0;
    for (int r = 0; r < C; ++r) {
      const uint64_t x = cta_sum[pass][r];
      if (r < rank) before += x;
      total += x;
    }
    if (total > 0 || !(qrow || gone)) break;
    qrow = nullptr;  // nothing is left: the target's row as it is
    gone = false;
  }
  if (total == 0) {
    if (report && tid == 0) {
      atomicOr(&g_verify_err, PA_DEVERR_TREE);
      a.next_token[b] = -1;
    }
    return;
  }
  const float u0 = node_u[0];
  t = u0 > 0.f ? static_cast<uint64_t>(static_cast<double>(fminf(u0, 1.f)) * static_cast<double>(total)) : 0ull;
  if (t >= total) t = total - 1;
  for (int w = 0; w < wid; ++w) before += warp_sum[w];
  if (t < before || t - before >= warp_sum[wid]) return;
  // the warp that holds it: 32 values at a time
  uint64_t at = before;
#pragma unroll 1
  for (int v0 = lo; v0 < hi; v0 += 32 * kAhead) {
    uint64_t w[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = v0 + 32 * i + lane;
      const uint64_t x = v < hi ? fixed44(__ldcg(prow + v)) : 0ull, y = qrow && v < hi ? fixed44(__ldcg(qrow + v)) : 0ull;
      w[i] = x > y ? x - y : 0ull;
      if (gone && w[i] > 0 && taken(v)) w[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      uint64_t inc = w[i];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t y = __shfl_up_sync(FULL, inc, off);
        if (lane >= off) inc += y;
      }
      const unsigned over = __ballot_sync(FULL, at + inc > t);
      if (over) {
        if (lane == 0) a.next_token[b] = v0 + 32 * i + __ffs(over) - 1;
        return;
      }
      at += __shfl_sync(FULL, inc, 31);
    }
  }
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
  int cluster = kMaxCluster;
  a.share = (l.V + cluster * kWarps - 1) / (cluster * kWarps);
  a.share = (a.share + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(l.B) * cluster);
  cfg.blockDim = dim3(kThreads);
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
