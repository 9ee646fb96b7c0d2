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
// (node, head of the group); they all read the same K/V, so a CTA takes up to
// 128 x TILES of them at once and streams the context in chunks of 128 keys
// (8 blocks).  One unit of work is one chunk for one such item; the launch has
// one persistent CTA per SM, and CTA k takes units [k u, (k + 1) u) of the
// batch in order, u = ceil(units / CTAs): every CTA streams the same number of
// chunks whatever the lengths.  The lengths stay on the device: each CTA
// counts the units itself from context_lens and q_start.  An item that spans
// CTAs leaves partial rows (o, m, l), at most two sets per CTA, merged by
// tree_merge with log-sum-exp weights.
//
// Inside a CTA (one per SM; 512 TMEM columns S0 S1 O0 O1):
//   warp 0       producer: K and V chunks into a ring of slots by TMA (128-byte
//                swizzle, one box of 16 keys per block and half row);
//   warp 1       issues the MMAs from one thread: S = Q K^T (M 128, N 128) and
//                O += P V (M 128, N = head_dim, P read from TMEM);
//   warps 4-7,   two softmax warpgroups, one per tile; thread r owns row r =
//   8-11         TMEM lane r.  With more than 128 rows the tiles are the two
//                halves of the rows and share every chunk; with 128 or fewer
//                they are the same rows over the even and the odd chunks, and
//                their two results are joined from TMEM at the end.  Either way
//                one tile's products run while the other's exponentials do.
//   warps 12-15  1-byte caches only: convert a landed slot's codes in place to
//                the 16-bit K-major / MN-major layouts the MMAs read.
// P overwrites S as 16-bit values and is normalised by the sum of the rounded
// weights, so a row that rests on one key returns that key's value exactly.
// 16 bits for P because the product's operands share V's type; its rounding
// (half a step, independent over keys) adds as much as the rounding of the
// output itself.  m, l and O are float32.  m only moves when a chunk's maximum
// exceeds it by 2^8, so O is rescaled rarely.
//
// What bounds it: HBM while the rows per kv head stay below ~290 (4 D flops
// per key and row against 4 D bytes per key at 16 bits), the exponentials and
// the MMAs above that.
//
// Values in masked places: chunks that reach the tree or the context's end
// take masks; V rows past the end are zeroed in shared memory, and a node's V
// row that holds an infinity or NaN (a slot nothing was ever written to) is
// zeroed too and added by hand to the rows that do see it, so it reaches no
// other row.  K needs no such care: a masked score is replaced.
#include <cudaTypedefs.h>

#include <mutex>

#include "device_common.cuh"
#include "kv_map.h"
#include "pa_internal.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

__device__ uint32_t g_tree_err;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kMaxDevices = 64;
constexpr int kKeys = 128;    // keys per chunk
constexpr int kBlk = kKeys / 16;
constexpr float kMove = 8.f;  // log2 of how far the scores may outgrow m before it moves
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kLimit = 2000000000ull, kLimitExit = 100000000ull;

struct TreeArgs {
  const void* q;
  const int32_t* q_start;
  const uint64_t* mask;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* part_o;  // [2 * CTAs][rows of an item][D], then m and l [2 * CTAs][rows]
  float* part_m;
  float* part_l;
  int32_t B, T, Hq, Hkv, G, max_blocks, num_blocks, max_context_len, max_q_len, words;
  int32_t min_units;  // units a CTA takes at least
  int32_t n_cta;
  float scale_log2;   // |scale| log2 e
  uint32_t q_flip;    // 0x80008000 when scale < 0: the sign goes into Q
  int32_t out_f32;
};

// ---- the batch's work ------------------------------------------------------
struct Seq {
  int qs, n, L;   // first query row, nodes, context length
  int tiles, nch;  // row tiles per kv head, chunks
};
// Sequence b's view, clamped to what the launch can serve; violations are
// flagged by the one thread that reports.
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b, int rows, bool report) {
  Seq s;
  s.qs = a.q_start[b];
  s.n = a.q_start[b + 1] - s.qs;
  s.L = a.context_lens[b];
  if (s.qs < 0 || s.n < 0 || s.n > a.max_q_len || s.qs > a.T - s.n) {
    if (report) atomicOr(&g_tree_err, PA_DEVERR_QUERY_RANGE);
    s.qs = s.n = 0;
  }
  const int cap = min(a.max_context_len, a.max_blocks * 16);
  if (s.L < 0 || s.L > cap) {
    if (report) atomicOr(&g_tree_err, PA_DEVERR_CONTEXT_LEN);
    s.L = max(0, min(s.L, cap));
  }
  if (s.n > s.L && report) atomicOr(&g_tree_err, PA_DEVERR_CONTEXT_LEN);
  s.tiles = (s.n * a.G + rows - 1) / rows;
  s.nch = max(1, (s.L + kKeys - 1) / kKeys);  // a sequence without keys still owns its zero rows
  return s;
}
__device__ __forceinline__ int units_of(const TreeArgs& a, const Seq& s) { return s.tiles * a.Hkv * s.nch; }
__device__ __forceinline__ int units_per_cta(const TreeArgs& a, int total) {
  return max((total + a.n_cta - 1) / a.n_cta, a.min_units);
}
__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL, v, off);
  return v;
}

// One item's run of chunks [c0, c1) for a CTA.
struct Piece {
  int b, g, qt, c0, c1, slot;  // slot: its set of partial rows (-1: the whole item)
  Seq s;
};
// Walks a CTA's units in order; every role of the CTA walks the same pieces.
struct Walk {
  int u, end, start, b, ub;
  template <int ROWS>
  __device__ __forceinline__ bool next(const TreeArgs& a, Piece& p) {
    if (u >= end) return false;
    Seq s = seq_of(a, b, ROWS, false);
    int w = units_of(a, s);
    while (u >= ub + w) {
      ub += w;
      ++b;
      s = seq_of(a, b, ROWS, false);
      w = units_of(a, s);
    }
    const int at = u - ub, item = at / s.nch;
    p.b = b;
    p.s = s;
    p.g = item / s.tiles;
    p.qt = item - p.g * s.tiles;
    p.c0 = at - item * s.nch;
    p.c1 = min(s.nch, p.c0 + end - u);
    const bool whole = p.c0 == 0 && p.c1 == s.nch;
    p.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (u == start ? 0 : 1);
    u += p.c1 - p.c0;
    return true;
  }
};

// ---- shared memory -----------------------------------------------------------
template <typename KT, int D, int TILES>
struct Lay {
  static constexpr bool Q8 = sizeof(KT) == 1;
  static constexpr int SPANS = D / 64;               // 128-byte spans of a 16-bit row
  static constexpr int QTILE = 128 * D * 2;
  static constexpr int SLOT = kKeys * D * 2;         // one K or V chunk, 16-bit
  static constexpr int NS = (D == 64 ? 2 : 1) * (TILES == 2 ? (Q8 ? 4 : 5) : (Q8 ? 5 : 6));
  static constexpr int RING = TILES * QTILE;
  static constexpr int SCALES = RING + NS * SLOT;    // 1-byte codes: [8 chunks][K 128, V 128] float
  static constexpr int BAR = SCALES + (Q8 ? 8 * 1024 : 0);
  static constexpr int NBAR = 3 * NS + 8;
  static constexpr int MISC = (BAR + NBAR * 8 + 15) & ~15;  // tmem address, work; at 64: bad keys
  static constexpr int BYTES = MISC + 128 + 1024;
  static constexpr int THREADS = Q8 ? 512 : 384;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// A bounded wait whose outcome is the same in every lane (lane 0's), so the
// warp-collective instructions that follow stay converged.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
  const bool ok = dev::mbar_wait_bounded(bar, parity, kLimit);
  return __shfl_sync(FULL, ok ? 1 : 0, 0) != 0;
}
// Tensor-memory loads that have arrived when they return (load and wait in one
// statement, so no use of the registers can be scheduled between them).
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r)
               : "r"(taddr)
               : "memory");
  return r;
}
__device__ __forceinline__ float2 tmem_ld2(uint32_t taddr) {
  uint32_t x, y;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(x), "=r"(y)
               : "r"(taddr)
               : "memory");
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ void tmem_st2(uint32_t taddr, float x, float y) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(taddr),
               "r"(__float_as_uint(x)), "r"(__float_as_uint(y))
               : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
template <typename T>
__device__ __forceinline__ bool bad16(uint32_t w) {  // a pair holds an infinity or NaN
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  return (w & E) == E || ((w >> 16) & E) == E;
}
// Bits of nodes off .. off + 31 in a mask row of `words` 64-bit words; nodes
// below 0 are context (set), nodes from n on do not exist (clear).
__device__ __forceinline__ uint32_t mask32(const uint64_t* row, int words, int off, int n) {
  if (off <= -32) return FULL;
  uint32_t v = 0;
  if (off < 0) {
    const uint32_t w0 = n > 0 ? static_cast<uint32_t>(row[0]) : 0u;
    const int live = min(n, 32 + off);  // node bits that fit
    const uint32_t keep = live <= 0 ? 0u : live >= 32 ? FULL : (1u << live) - 1u;
    return ((1u << -off) - 1u) | ((w0 & keep) << -off);
  }
  if (off >= n) return 0;
  const int wi = off >> 6, sh = off & 63;
  uint64_t x = row[wi] >> sh;
  if (sh > 32 && wi + 1 < words) x |= row[wi + 1] << (64 - sh);
  v = static_cast<uint32_t>(x);
  const int live = n - off;
  return live >= 32 ? v : v & ((1u << live) - 1u);
}

template <typename T>
__device__ __forceinline__ void store8(const TreeArgs& a, size_t idx, const float (&x)[8]) {
  if (a.out_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + idx);
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + idx) =
        make_uint4(dev::pack2<T>(x[0], x[1]), dev::pack2<T>(x[2], x[3]), dev::pack2<T>(x[4], x[5]),
                   dev::pack2<T>(x[6], x[7]));
  }
}

template <typename KT, typename T, int D, int TILES>
__global__ void __launch_bounds__(Lay<KT, D, TILES>::THREADS, 1)
    tree_main(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const TreeArgs a) {
  using namespace tcg;
  using L = Lay<KT, D, TILES>;
  constexpr bool Q8 = L::Q8;
  constexpr int NS = L::NS, ROWS = 128 * TILES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (base - raw);
  const int wid = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);

  const uint32_t bars = base + L::BAR;
  auto full = [&](int s) { return bars + 8 * s; };             // slot s landed
  auto conv = [&](int s) { return bars + 8 * (NS + s); };      // 1-byte codes: slot s converted
  auto empty = [&](int s) { return bars + 8 * (2 * NS + s); };  // slot s read by its last product
  auto sfull = [&](int t) { return bars + 8 * (3 * NS + t); };      // tile t: S in TMEM
  auto pfull = [&](int t) { return bars + 8 * (3 * NS + 2 + t); };  // tile t: P in TMEM
  auto pdone = [&](int t) { return bars + 8 * (3 * NS + 4 + t); };  // tile t: O += P V complete
  const uint32_t qfull = bars + 8 * (3 * NS + 6);                   // Q in shared memory, O of the piece before read
  const uint32_t mdone = bars + 8 * (3 * NS + 7);                   // after a timeout: every product has ended
  int* work = reinterpret_cast<int*>(gb + L::MISC + 16);  // start unit, end, sequence, units before it
  auto ready = [&](int s) { return Q8 ? conv(s) : full(s); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      dev::mbar_init(full(s), 1);
      dev::mbar_init(conv(s), 4);
      dev::mbar_init(empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      dev::mbar_init(sfull(t), 1);
      dev::mbar_init(pfull(t), 4);
      dev::mbar_init(pdone(t), 1);
    }
    dev::mbar_init(qfull, 8);
    dev::mbar_init(mdone, 1);
    dev::fence_barrier_init();
    dev::prefetch_tensormap(&tmK);
    dev::prefetch_tensormap(&tmV);
  }
  if (wid == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + L::MISC),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  dev::grid_dependency_wait();  // the cache write before this kernel is visible
  if (wid == 0) {
    // this CTA's units, counted 32 sequences at a time
    const bool report = blockIdx.x == 0;
    int total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32)
      total += b0 + lane < a.B ? units_of(a, seq_of(a, b0 + lane, ROWS, report)) : 0;
    total = warp_sum(total);
    const int upc = units_per_cta(a, total);
    const int start = min(static_cast<int>(blockIdx.x) * upc, total), end = min(start + upc, total);
    int run = 0, fb = 0, fu = 0;
    for (int b0 = 0; start < end && b0 < a.B; b0 += 32) {
      const int w = b0 + lane < a.B ? units_of(a, seq_of(a, b0 + lane, ROWS, false)) : 0;
      int inc = w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(FULL, inc, off);
        if (lane >= off) inc += y;
      }
      const unsigned over = __ballot_sync(FULL, run + inc > start);
      if (over) {
        const int f = __ffs(over) - 1;
        fb = b0 + f;
        fu = run + __shfl_sync(FULL, inc - w, f);
        break;
      }
      run += __shfl_sync(FULL, inc, 31);
    }
    if (lane == 0) {
      work[0] = start;
      work[1] = end;
      work[2] = fb;
      work[3] = fu;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gb + L::MISC);
  Walk walk;
  walk.start = walk.u = work[0];
  walk.end = work[1];
  walk.b = work[2];
  walk.ub = work[3];
  Piece p;
  bool ok = true;
  int it = 0;  // ring items before this piece: K(c), V(c) of each chunk in order

  if (wid == 0) {
    // ---- producer: lane i < 8 issues block i of a chunk --------------------------
    int issued = 0;
    while (walk.next<ROWS>(a, p)) {
      const int nblk = (p.s.L + 15) / 16;
      const int32_t* row = a.block_tables + static_cast<size_t>(p.b) * a.max_blocks;
      auto fetch = [&](int c) {
        const int j = c * kBlk + lane;
        int v = lane < kBlk && j < nblk ? row[j] : 0;
        if (v < 0 || v >= a.num_blocks) {
          atomicOr(&g_tree_err, PA_DEVERR_BLOCK_RANGE);  // block 0 is read instead; flagged
          v = 0;
        }
        return v;
      };
      int nxt = fetch(p.c0);
      for (int c = p.c0; c < p.c1; ++c) {
        const int id = nxt;
        if (c + 1 < p.c1) nxt = fetch(c + 1);
        const int live = max(0, min(kBlk, nblk - c * kBlk));  // blocks of this chunk that exist
#pragma unroll 1
        for (int v = 0; v < 2; ++v, ++it) {
          const int s = it % NS;
          if (ok && it >= NS) {
            ok = wait_warp(empty(s), ((it / NS) - 1) & 1);
            if (!ok && lane == 0) atomicOr(&g_tree_err, PA_DEVERR_TIMEOUT);
          }
          if (!ok) continue;
          issued = it + 1;
          dev::fence_proxy_async_smem();  // the softmax's and converters' accesses precede the refill
          const uint32_t dst = base + L::RING + s * L::SLOT, bar = full(s);
          if constexpr (Q8) {
            // codes land in the upper half of the slot; 16 scales a block
            if (lane == 0) dev::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live * (16 * D + 64)));
            __syncwarp();
            if (lane < live) {
              dev::tma_load_3d(dst + L::SLOT / 2 + lane * 2048, v ? &tmV : &tmK, bar, 0, p.g * 16, id);
              dev::bulk_load(base + L::SCALES + ((it >> 1) & 7) * 1024 + v * 512 + lane * 64,
                             (v ? a.v_scale : a.k_scale) + static_cast<size_t>(id) * 16, 64, bar);
            }
          } else {
            if (lane == 0) dev::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live * 16 * D * 2));
            __syncwarp();
            if (lane < live) {
              if constexpr (D == 64) {
                dev::tma_load_3d(dst + lane * 2048, v ? &tmV : &tmK, bar, 0, p.g * 16, id);
              } else if (v) {  // [block][span][16][128 B]
                dev::tma_load_5d(dst + lane * 4096, &tmV, bar, 0, 0, 0, p.g, id);
              } else {         // [span][128 keys][128 B]
                dev::tma_load_3d(dst + lane * 2048, &tmK, bar, 0, p.g * 16, id);
                dev::tma_load_3d(dst + 16384 + lane * 2048, &tmK, bar, 64, p.g * 16, id);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    // no copy may still be landing when the CTA exits
    for (int i = max(0, issued - NS); i < issued; ++i) dev::mbar_wait_bounded(full(i % NS), (i / NS) & 1, kLimitExit);
    __syncwarp();
  } else if (wid == 1) {
    // ---- MMA issuer: one thread ---------------------------------------------------
    if (lane == 0) {
      const uint32_t id_s = idesc<T>(kKeys, false), id_o = idesc<T>(D, true);
      int ns[2] = {0, 0}, np[2] = {0, 0};  // S and PV products issued per tile, all pieces
      int piece = 0;
      while (walk.next<ROWS>(a, p)) {
        const bool pair = TILES == 2 && (p.s.n * a.G - p.qt * ROWS) > 128;  // two row tiles share the chunks
        const int nc = p.c1 - p.c0;
        const int todo[2] = {pair ? nc : (nc + 1) / 2, pair ? nc : nc / 2};
        int cs[2] = {0, 0}, cp[2] = {0, 0};  // this piece's products, per tile
        int kfree = 0, vfree = 0;
        if (ok) ok = dev::mbar_wait_bounded(qfull, piece & 1, kLimit);
        uint64_t t0 = dev::global_timer_ns();
        int spin = 0;
        while (ok && (cp[0] < todo[0] || cp[1] < todo[1])) {
          bool moved = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            // O_t += P_t V once P_t is written and V has landed
            if (cp[t] < cs[t]) {
              const int c = pair ? cp[t] : 2 * cp[t] + t, i = it + 2 * c + 1, s = i % NS;
              if (dev::mbar_test(pfull(t), np[t] & 1) && dev::mbar_test(ready(s), (i / NS) & 1)) {
                fence_after();
                const uint32_t vd = base + L::RING + s * L::SLOT, pt = tmem + 128 * t, od = tmem + 256 + 128 * t;
#pragma unroll
                for (int kk = 0; kk < kBlk; ++kk)
                  mma_ts(od, pt + 8 * kk, sdesc(vd + kk * (2048 * L::SPANS), 2048, 1024), id_o,
                         cp[t] > 0 || kk > 0 ? 1u : 0u);
                commit(pdone(t));
                ++cp[t];
                ++np[t];
                if (pair) {
                  for (; vfree < min(cp[0], cp[1]); ++vfree) commit(empty((it + 2 * vfree + 1) % NS));
                } else {
                  commit(empty(s));
                }
                moved = true;
              }
            }
            // S_t = Q_t K^T once K has landed and O_t += P_t V released the buffer
            if (cs[t] < todo[t] && cs[t] == cp[t]) {
              const int c = pair ? cs[t] : 2 * cs[t] + t, i = it + 2 * c, s = i % NS;
              if (dev::mbar_test(ready(s), (i / NS) & 1) &&
                  (ns[t] == 0 || dev::mbar_test(pdone(t), (ns[t] - 1) & 1))) {
                fence_after();
                const uint32_t kd = base + L::RING + s * L::SLOT, qd = base + (pair ? t : 0) * L::QTILE;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  mma_ss(tmem + 128 * t, sdesc(qd + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                         sdesc(kd + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024), id_s, kk > 0 ? 1u : 0u);
                commit(sfull(t));
                ++cs[t];
                ++ns[t];
                if (pair) {
                  for (; kfree < min(cs[0], cs[1]); ++kfree) commit(empty((it + 2 * kfree) % NS));
                } else {
                  commit(empty(s));
                }
                moved = true;
              }
            }
          }
          if (moved) {
            spin = 0;
          } else if ((++spin & 63) == 0) {
            const uint64_t t1 = dev::global_timer_ns();
            if (spin == 64) t0 = t1;
            if (t1 - t0 > kLimit) ok = false;
          }
        }
        it += 2 * nc;
        ++piece;
      }
      if (!ok) {
        atomicOr(&g_tree_err, PA_DEVERR_TIMEOUT);
        commit(mdone);  // products in flight complete before their tensor memory is released
        dev::mbar_wait_bounded(mdone, 0, kLimitExit);
      }
    }
    __syncwarp();
  } else if (wid >= 4 && wid < 12) {
    // ---- softmax warpgroups -----------------------------------------------------------
    const int t = (wid - 4) >> 2;        // tile
    const int w4 = wid & 3;              // TMEM lane quadrant
    const int r = 32 * w4 + lane;        // row of the tile = TMEM lane
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * w4) << 16);
    const uint32_t ts = tl + 128 * t, to = tl + 256 + 128 * t;
    volatile uint32_t* badw = reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 64);  // [2 parities][2 tiles][4]
    const float sl2 = a.scale_log2;
    int n_s = 0;  // chunks of this tile so far, all pieces
    bool first = true;
    while (walk.next<ROWS>(a, p)) {
      const int nrows = p.s.n * a.G, R0 = p.qt * ROWS;
      const bool pair = TILES == 2 && nrows - R0 > 128;
      const int rr = R0 + (pair ? 128 * t : 0) + r;
      const bool has = rr < nrows;
      const bool live = R0 + (pair ? 128 * t : 0) + 32 * w4 < nrows;  // the warp has a row
      const int node = has ? rr / a.G : 0;
      const size_t head = has ? static_cast<size_t>(p.s.qs + node) * a.Hq + p.g * a.G + (rr - node * a.G) : 0;
      const uint64_t* mrow = a.mask + static_cast<size_t>(p.s.qs + node) * a.words;
      const int shift = p.s.L - p.s.n;  // key of node 0
      const int nc = p.c1 - p.c0;
      if (!first) named_bar(1, 256);  // both tiles have seen their last S: Q may be rewritten
      first = false;
      {  // Q rows -> shared memory, K-major, 128-byte swizzle; zeros for rows that do not exist
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + head * D);
        uint8_t* dst = gb + (pair ? t : 0) * L::QTILE + r * 128;
        const int c_lo = pair ? 0 : t * (D / 16), c_hi = pair ? D / 8 : c_lo + D / 16;
#pragma unroll 4
        for (int ch = c_lo; ch < c_hi; ++ch) {
          uint4 v = has ? src[ch] : make_uint4(0, 0, 0, 0);
          v.x ^= a.q_flip;
          v.y ^= a.q_flip;
          v.z ^= a.q_flip;
          v.w ^= a.q_flip;
          *reinterpret_cast<uint4*>(dst + (ch >> 3) * 16384 + (((ch & 7) ^ (r & 7)) << 4)) = v;
        }
        dev::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull);
      }
      float ref = -INFINITY, l = 0.f;
      bool has_extra = false;
      float extra[D];  // V rows with infinities or NaN, added by hand
      for (int c = pair ? 0 : t; c < nc; c += pair ? 1 : 2) {
        if (ok) ok = wait_warp(sfull(t), n_s & 1);
        ++n_s;
        fence_after();
        const int key0 = (p.c0 + c) * kKeys;
        const bool masked = key0 + kKeys > shift;
        const float* ksc = reinterpret_cast<const float*>(gb + L::SCALES + (((it >> 1) + c) & 7) * 1024);
        const float* vsc = ksc + 128;
        uint32_t mk[4] = {FULL, FULL, FULL, FULL};
        if (masked) {
#pragma unroll
          for (int w = 0; w < 4; ++w) mk[w] = has ? mask32(mrow, a.words, key0 + 32 * w - shift, p.s.n) : 0u;
        }
        // scores of keys 32 w .. 32 w + 31: K scale applied, masked keys -inf
        auto scores = [&](int w, float (&x)[32]) {
          uint32_t u[32];
          tmem_ld32(ts + 32 * w, u);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            x[j] = __uint_as_float(u[j]);
            if constexpr (Q8) x[j] *= ksc[32 * w + j];
          }
          if (masked) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = (mk[w] >> j) & 1u ? x[j] : -INFINITY;
          }
        };
        if (live) {
          float cmax = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            float x[32];
            scores(w, x);
            float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], x[j]);
            cmax = fmaxf(cmax, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
          }
          cmax *= sl2;
          const bool move = cmax > ref + kMove;
          const bool scale_o = move && ref != -INFINITY;
          if (__any_sync(FULL, scale_o)) {
            // (S was issued after the tile's last product had completed, so O is at rest)
            const float al = scale_o ? dev::ex2(ref - cmax) : 1.f;
#pragma unroll 1
            for (int qd = 0; qd < D / 32; ++qd) {
              uint32_t u[32];
              tmem_ld32(to + 32 * qd, u);
#pragma unroll
              for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * al);
              st32(to + 32 * qd, u);
            }
            wait_st();
            l *= al;
            if (has_extra)
#pragma unroll 1
              for (int d = 0; d < D; ++d) extra[d] *= al;
          }
          if (move) ref = cmax;
        }
        const float nref = ref == -INFINITY ? 0.f : -ref;
        if (masked) {
          // V rows that must not reach a product: past the context's end, or a
          // node's with an infinity or NaN.  Thread r checks key r.
          const int vi = it + 2 * c + 1, vs = vi % NS;
          if (ok) ok = wait_warp(ready(vs), (vi / NS) & 1);
          uint8_t* vrow = gb + L::RING + vs * L::SLOT + (r >> 4) * (2048 * L::SPANS) + (r & 15) * 128;
          volatile uint32_t* bw = badw + ((p.c0 + c) & 1) * 8 + (pair ? 0 : 4 * t);
          const bool scan = !pair || t == 0;
          const int bar_id = pair ? 1 : 2 + t, bar_n = pair ? 256 : 128;
          if (scan) {
            bool bad = false;
            if (key0 + r >= p.s.L) {
#pragma unroll
              for (int sp = 0; sp < L::SPANS; ++sp)
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                  *reinterpret_cast<uint4*>(vrow + sp * 2048 + ch * 16) = make_uint4(0, 0, 0, 0);
            } else if (key0 + r >= shift) {
#pragma unroll
              for (int sp = 0; sp < L::SPANS; ++sp)
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                  const uint4 v = *reinterpret_cast<const uint4*>(vrow + sp * 2048 + ((ch ^ (r & 7)) << 4));
                  bad |= bad16<T>(v.x) | bad16<T>(v.y) | bad16<T>(v.z) | bad16<T>(v.w);
                }
            }
            const uint32_t word = __ballot_sync(FULL, bad);
            if (lane == 0) bw[w4] = word;
            dev::fence_proxy_async_smem();
          }
          named_bar(bar_id, bar_n);
          if (bw[0] | bw[1] | bw[2] | bw[3]) {
#pragma unroll 1
            for (int j = 0; j < kKeys; ++j) {
              if (!((bw[j >> 5] >> (j & 31)) & 1u)) continue;
              float x = __uint_as_float(tmem_ld1(ts + j));
              const uint32_t mw = j < 32 ? mk[0] : j < 64 ? mk[1] : j < 96 ? mk[2] : mk[3];
              if ((mw >> (j & 31)) & 1u) {
                if constexpr (Q8) x *= ksc[j];
                float pj = dev::ex2(fmaf(x, sl2, nref));
                if constexpr (Q8) pj *= vsc[j];
                if (!has_extra) {
                  has_extra = true;
#pragma unroll 1
                  for (int d = 0; d < D; ++d) extra[d] = 0.f;
                }
                const uint8_t* vb = gb + L::RING + vs * L::SLOT + (j >> 4) * (2048 * L::SPANS) + (j & 15) * 128;
#pragma unroll 1
                for (int d = 0; d < D; d += 2) {
                  const uint32_t pr = *reinterpret_cast<const uint32_t*>(
                      vb + (d >> 6) * 2048 + ((((d & 63) >> 3) ^ (j & 7)) << 4) + (d & 7) * 2);
                  const float2 f = dev::unpack2<T>(pr);
                  extra[d] += pj * f.x;
                  extra[d + 1] += pj * f.y;
                }
              }
              __syncwarp();
            }
            named_bar(bar_id, bar_n);  // every reader is done with the rows
            if (scan && ((bw[w4] >> lane) & 1u)) {
#pragma unroll
              for (int sp = 0; sp < L::SPANS; ++sp)
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                  *reinterpret_cast<uint4*>(vrow + sp * 2048 + ch * 16) = make_uint4(0, 0, 0, 0);
            }
            dev::fence_proxy_async_smem();
            named_bar(bar_id, bar_n);
          }
        }
        if (live) {
          // P over S, 16-bit pairs: p = 2^(s |scale| log2 e - ref)
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[32];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            float x[32];
            scores(w, x);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float p0 = dev::ex2(fmaf(x[j], sl2, nref)), p1 = dev::ex2(fmaf(x[j + 1], sl2, nref));
              uint32_t& pr = pk[(w & 1) * 16 + (j >> 1)];
              if constexpr (Q8) {
                // V's scale rides on p; a masked key has p = 0 and perhaps a stale scale
                const float v0 = vsc[32 * w + j], v1 = vsc[32 * w + j + 1];
                pr = dev::pack2<T>(p0 == 0.f ? 0.f : p0 * v0, p1 == 0.f ? 0.f : p1 * v1);
                ls[(j >> 1) & 3] += p0 + p1;
              } else {
                pr = dev::pack2<T>(p0, p1);
                const float2 h = dev::unpack2<T>(pr);
                ls[(j >> 1) & 3] += h.x + h.y;
              }
            }
            if (w & 1) {
              // columns 0..31 (keys 0..63) overwrite scores already read; the
              // second half of the scores sits in columns 64..127
              st32(ts + 16 * (w - 1), pk);
            }
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(t));
      }
      // ---- the rows out -----------------------------------------------------------------
      if (walk.u >= walk.end) dev::grid_launch_dependents();
      const int mine = pair ? nc : (t ? nc / 2 : (nc + 1) / 2);
      if (ok && mine > 0) ok = wait_warp(pdone(t), (n_s - 1) & 1);
      fence_after();
      if (__any_sync(FULL, has_extra)) {
#pragma unroll 1
        for (int qd = 0; qd < D / 32; ++qd) {
          uint32_t u[32];
          tmem_ld32(to + 32 * qd, u);
          if (has_extra)
#pragma unroll 1
            for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) + extra[32 * qd + j]);
          st32(to + 32 * qd, u);
        }
        wait_st();
      }
      float m = ref, w0 = 1.f, w1 = 0.f;  // weights of tile 0's and tile 1's O (this tile's own with pairs)
      if (!pair) {  // join the even and the odd chunks
        tmem_st2(ts + 64, ref, l);  // the tile's S buffer is at rest; P took its columns 0..63
        fence_before();
        named_bar(1, 256);
        fence_after();
        const float2 x0 = tmem_ld2(tl + 64), x1 = tmem_ld2(tl + 128 + 64);
        m = fmaxf(x0.x, x1.x);
        const float mz = m == -INFINITY ? 0.f : m;
        w0 = dev::ex2(x0.x - mz);
        w1 = nc > 1 ? dev::ex2(x1.x - mz) : 0.f;
        l = x0.y * w0 + (nc > 1 ? x1.y * w1 : 0.f);
      }
      if (live) {
        const bool direct = p.slot < 0;
        const float inv = direct ? (m == -INFINITY ? 0.f : 1.f / l) : 1.f;
        const bool none = m == -INFINITY;
        const int d_lo = pair ? 0 : t * (D / 2), d_hi = pair ? D : d_lo + D / 2;
        const size_t prow = direct ? 0 : static_cast<size_t>(p.slot) * ROWS + (rr - R0);
#pragma unroll 1
        for (int d = d_lo; d < d_hi; d += 32) {
          uint32_t u[32];
          float o[32];
          tmem_ld32((pair ? to : tl + 256) + d, u);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(u[j]) * w0;
          if (!pair && nc > 1) {
            tmem_ld32(tl + 384 + d, u);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] += __uint_as_float(u[j]) * w1;
          }
          if (has) {
            if (direct) {
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = none ? 0.f : o[j + e] * inv;
                store8<T>(a, head * D + d + j, y);
              }
            } else {
              float4* po = reinterpret_cast<float4*>(a.part_o + prow * D + d);
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                po[j >> 2] = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
          }
        }
        if (has && !direct && (pair || t == 0)) {
          a.part_m[prow] = m;
          a.part_l[prow] = l;
        }
      }
      fence_before();  // O is read: the next piece's products may follow once Q is in place
      it += 2 * nc;
    }
    if (!ok && lane == 0) atomicOr(&g_tree_err, PA_DEVERR_TIMEOUT);
  } else if (Q8 && wid >= 12) {
    // ---- converters: codes of a landed slot -> 16-bit, in place -----------------------
    const int i0 = static_cast<int>(threadIdx.x) - 384;
    while (walk.next<ROWS>(a, p)) {
      const int nc = p.c1 - p.c0;
      for (int k = 0; k < 2 * nc; ++k, ++it) {
        const int s = it % NS;
        if (ok) ok = wait_warp(full(s), (it / NS) & 1);
        uint8_t* st = gb + L::RING + s * L::SLOT;
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // 16 codes: chunk c16 of row i / 8
          const int i = i0 + 128 * j, key = i >> 3, c16 = i & 7;
          w[j] = *reinterpret_cast<const uint4*>(st + L::SLOT / 2 + key * 128 + ((c16 ^ (key & 7)) << 4));
        }
        named_bar(4, 128);  // every code is in registers before the slot is rewritten
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + 128 * j, key = i >> 3, c16 = i & 7, cc = 2 * (c16 & 3), sp = c16 >> 2;
          uint32_t f[8];
          dev::code8x4_to<KT, T>(w[j].x, f[0], f[1]);
          dev::code8x4_to<KT, T>(w[j].y, f[2], f[3]);
          dev::code8x4_to<KT, T>(w[j].z, f[4], f[5]);
          dev::code8x4_to<KT, T>(w[j].w, f[6], f[7]);
          uint8_t* row = (k & 1) ? st + (key >> 4) * 4096 + sp * 2048 + (key & 15) * 128  // V
                                 : st + sp * 16384 + key * 128;                          // K
          *reinterpret_cast<uint4*>(row + ((cc ^ (key & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<uint4*>(row + (((cc + 1) ^ (key & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
        }
        dev::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(conv(s));
      }
    }
    if (!ok && lane == 0) atomicOr(&g_tree_err, PA_DEVERR_TIMEOUT);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (wid == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Merge of the items that span CTAs: one warp per (node, query head) row,
// kMergeRows rows per CTA.  A row finds its sequence by binary search over
// q_start and the CTAs of its item from the same unit count as tree_main.
constexpr int kMergeRows = 8;

template <typename T, int D, int TILES>
__global__ void __launch_bounds__(32 * kMergeRows) tree_merge(const TreeArgs a) {
  constexpr int V = D / 32, ROWS = 128 * TILES;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 5);
  dev::grid_dependency_wait();
  if (row >= static_cast<int64_t>(a.T) * a.Hq) return;
  const int tok = static_cast<int>(row / a.Hq), h = static_cast<int>(row - static_cast<int64_t>(tok) * a.Hq);
  if (a.q_start[0] > tok) return;
  int lo = 0, hi = a.B;  // the last sequence that starts at or before tok
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= tok) lo = mid; else hi = mid;
  }
  const int b = lo;
  const Seq s = seq_of(a, b, ROWS, false);
  const int i = tok - s.qs;
  if (i < 0 || i >= s.n || s.nch < 2) return;  // outside every sequence, or one chunk
  int total = 0, before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int w = b0 + lane < a.B ? units_of(a, seq_of(a, b0 + lane, ROWS, false)) : 0;
    total += w;
    before += b0 + lane < b ? w : 0;
  }
  total = warp_sum(total);
  before = warp_sum(before);
  const int upc = units_per_cta(a, total);
  const int g = h / a.G, rr = i * a.G + (h - g * a.G), qt = rr / ROWS;
  const int u0 = before + (g * s.tiles + qt) * s.nch, u1 = u0 + s.nch;
  const int k0 = u0 / upc, k1 = (u1 - 1) / upc;
  if (k0 == k1) return;  // written by tree_main
  auto slot_row = [&](int k) {
    return (static_cast<size_t>(2 * k + (u0 <= k * upc ? 0 : 1))) * ROWS + (rr - qt * ROWS);
  };
  float M = -INFINITY, ls = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int c0 = k0; c0 <= k1; c0 += 32) {
    const int n = min(32, k1 + 1 - c0);
    const float mv = lane < n ? a.part_m[slot_row(c0 + lane)] : -INFINITY;
    const float lv = lane < n ? a.part_l[slot_row(c0 + lane)] : 0.f;
    float cm = mv;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) cm = fmaxf(cm, __shfl_xor_sync(FULL, cm, off));
    const float nm = fmaxf(M, cm);
    if (nm == -INFINITY) continue;  // no key in any of them
    const float again = dev::ex2(M - nm);
    M = nm;
    const float w = lane < n ? dev::ex2(mv - nm) : 0.f;
    float wl = w * lv;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) wl += __shfl_xor_sync(FULL, wl, off);
    ls = ls * again + wl;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= again;
    for (int k = 0; k < n; ++k) {
      const float wk = __shfl_sync(FULL, w, k);
      const float* src = a.part_o + slot_row(c0 + k) * D + lane * V;
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const float2 f = *reinterpret_cast<const float2*>(src + v);
        acc[v] += wk * f.x;
        acc[v + 1] += wk * f.y;
      }
    }
  }
  const float inv = M == -INFINITY ? 0.f : 1.f / ls;
  const size_t at = (static_cast<size_t>(tok) * a.Hq + h) * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    if (a.out_f32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + v) = make_float2(acc[v] * inv, acc[v + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + at + v) = dev::pack2<T>(acc[v] * inv, acc[v + 1] * inv);
  }
}

template <typename KT, typename T, int D, int TILES>
pa_status launch_tiles(const TreeLaunch& l, TreeArgs a, CUtensorMapDataType dt, cudaStream_t stream) {
  using Y = Lay<KT, D, TILES>;
  constexpr int EB = static_cast<int>(sizeof(KT));
  CUtensorMap tmK, tmV;
  pa_status st = make_kv_map(&tmK, l.k_cache, l.Hkv, l.num_blocks, D * EB, EB, dt, "pa_tree_attention", false);
  if (st != PA_OK) return st;
  st = make_kv_map(&tmV, l.v_cache, l.Hkv, l.num_blocks, D * EB, EB, dt, "pa_tree_attention", true);
  if (st != PA_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices)
    return fail(PA_ERR_CUDA, "pa_tree_attention: no CUDA device");
  static std::once_flag once[kMaxDevices];
  static cudaError_t setup[kMaxDevices];
  std::call_once(once[dev], [dev] {
    setup[dev] =
        cudaFuncSetAttribute(tree_main<KT, T, D, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, Y::BYTES);
  });
  if (setup[dev] != cudaSuccess)
    return fail(PA_ERR_CUDA, "pa_tree_attention: %s", cudaGetErrorString(setup[dev]));
  const size_t rows = static_cast<size_t>(2) * a.n_cta * 128 * TILES;
  a.part_o = static_cast<float*>(l.workspace);
  a.part_m = a.part_o + rows * D;
  a.part_l = a.part_m + rows;
  cudaError_t e = launch_dependent(tree_main<KT, T, D, TILES>, dim3(static_cast<unsigned>(a.n_cta)),
                                   dim3(Y::THREADS), Y::BYTES, stream, tmK, tmV, a);
  if (e == cudaSuccess && l.max_context_len > kKeys)
    e = launch_dependent(tree_merge<T, D, TILES>,
                         dim3(static_cast<unsigned>((static_cast<int64_t>(l.T) * l.Hq + kMergeRows - 1) / kMergeRows)),
                         dim3(32 * kMergeRows), 0, stream, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_tree_attention launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

template <typename KT, typename T, int D>
pa_status launch_t(const TreeLaunch& l, CUtensorMapDataType dt, cudaStream_t stream) {
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
  const float mag = l.scale < 0.f ? -l.scale : l.scale;
  // a scale of 0 stays 0 for every finite score and leaves masked ones at -inf
  a.scale_log2 = mag * 1.4426950408889634f > 1e-30f ? mag * 1.4426950408889634f : 1e-30f;
  a.q_flip = l.scale < 0.f ? 0x80008000u : 0u;
  a.out_f32 = l.out_dtype == PA_DTYPE_F32;
  a.min_units = l.tiles == 2 ? 4 : 2;
  return l.tiles == 2 ? launch_tiles<KT, T, D, 2>(l, a, dt, stream) : launch_tiles<KT, T, D, 1>(l, a, dt, stream);
}

}  // namespace

pa_status launch_tree(const TreeLaunch& l, void* stream_ptr) {
  cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
  if (l.kv_dtype == PA_DTYPE_F16)
    return l.D == 64 ? launch_t<__half, __half, 64>(l, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, st)
                     : launch_t<__half, __half, 128>(l, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, st);
  if (l.kv_dtype == PA_DTYPE_BF16)
    return l.D == 64 ? launch_t<__nv_bfloat16, __nv_bfloat16, 64>(l, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, st)
                     : launch_t<__nv_bfloat16, __nv_bfloat16, 128>(l, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, st);
  const bool f16 = l.q_dtype == PA_DTYPE_F16;  // 1-byte codes, head_dim 128 (checked by the caller)
  if (l.kv_dtype == PA_DTYPE_INT8)
    return f16 ? launch_t<int8_t, __half, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st)
               : launch_t<int8_t, __nv_bfloat16, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st);
  return f16 ? launch_t<uint8_t, __half, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st)
             : launch_t<uint8_t, __nv_bfloat16, 128>(l, CU_TENSOR_MAP_DATA_TYPE_UINT8, st);
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
