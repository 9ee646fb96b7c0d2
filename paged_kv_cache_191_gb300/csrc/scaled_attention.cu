// Attention of new tokens over a block-scaled cache, on tcgen05 (sm_103a).
//
// What it computes: token i of the last n of an L-token context sees the keys
// 0 .. L - n + i,
//     out_i = sum_t p_it V_t / sum_t p_it,   p_it = exp(scale q_i . K_t),
// K and V one scale per (block, kv head) times E4M3 codes ("LLM推理引擎深度实战：
// 从PagedAttention到分布式推理部署", 5.3 and 2.3).
//
// The codes are never converted: they go from HBM by TMA to shared memory and from
// there into tcgen05.mma kind::f8f6f4 as they are.  What meets them, queries and
// weights, has more bits than an 8-bit type, so each is a sum of three E5M2 terms,
// which hold an f16 value exactly (scaled_common.cuh), and the terms are three times the
// columns of one product rather than three products: K and V, the larger operand, are
// read from shared memory once.  (Converting them to f16 there, as the calls over
// per-token scales do, moves a code's byte in, and out again as two, before the product
// reads those: at 8 rows that kernel's shape is bound by shared memory at half of HBM's
// rate.)  Above 40 rows per (sequence, kv head) the terms' columns outgrow tensor memory,
// and another kernel takes over (scaled_rows.cuh).
//
// The products are transposed as in the tree attention: S^T = K Q^T (M = the
// chunk's 128 keys, N = 3 terms x rows) and O^T += V^T P^T (M = 128 dims), a
// softmax thread owning a key, whose scales are its own registers: a block's scale
// multiplies the score after the product and the weight before it.  An item is 8, 16,
// 32 or 40 rows (tokens x heads of one kv head, the heads up to a power of two) and
// streams its context in chunks of 128 keys; of a prompt's items each only the chunks
// that its tokens see.  One persistent CTA per SM takes an equal run of the batch's
// chunks, planned on the device from the lengths; the parts of an item that spans CTAs
// are joined by whichever CTA writes the last one, in the order of the parts.
//
// Inside a CTA: warp 0 loads K and the scales, warp 2 V, warp 1 issues the products,
// warp 3 plans the pieces; warps 4-7 and 8-11 are two softmax warpgroups on alternate
// chunks, each with its scores, accumulators and references; warps 12-15 split the
// queries of the pieces to come into terms and write the rows of those that are over.
//
// What bounds it: HBM while a kv head has few rows, and what a CTA does besides.  8
// sequences of 8 kv heads, 4 rows, contexts to 32768: 70 us, 85 % of the copy rate; the
// chunks go by at 96 % of it, and the start (launch, lengths, block ids, scales, first
// chunk: 5 us) and the last joined rows (3 us) are the rest.  64 sequences of 8 kv heads,
// 8 rows, mean context 2064: 54 us, 74 %.  32 sequences of 32 kv heads, one row, mean
// context 1024: 56 us, 71 %: items of 8 chunks, whose first needs new references (700
// clocks) and a barrier.  The same 64 with chains of 2 tokens (16 rows) 57 us, 71 %, of
// 4 (32 rows) 80 us, 51 %, of 2 to 5 (40 rows) 91 us, 45 %: the
// softmax warpgroups, 2200 clocks a chunk where HBM takes 1420; a chunk's exponents take
// a warp 1000 clocks at 40 rows, the terms of its weights 900, one after the other.
// Code that runs once per piece is kept small where it costs no latency: a planner of
// many copies, 136 KB in all, took 78 us where 78 KB took 65 (the instruction caches; 32
// kv heads).  Not kept, since no faster: 8 rows at a time skipped that a short chain has
// not (114 us for 100: it cuts the straight line of exponents); scores of one row's three
// terms side by side along K, so that the product sums them (105 for 100); a fixed order
// of products in the middle of a piece (106 for 100).
//
// Values in masked places: a masked exponent is replaced; V rows that no row sees
// are zeroed in shared memory, and a NaN code in a row that only some see is
// zeroed and remembered for (dim, row), which end as NaN.  A NaN score or query comes
// out by the row's sum.
#include <atomic>
#include <mutex>

#include "pa_internal.h"
#include "scaled_rows.cuh"
#include "tree_maps.h"

namespace pa {
namespace {

constexpr int kMaxDevices = 64;

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc));
}
// kind::f8f6f4, f32 accumulate, M = 128, A E4M3, B E5M2; both K-major, or both not.
__device__ __forceinline__ constexpr uint32_t idesc_f8(int N, bool mn_major) {
  return (1u << 4) | (1u << 10) | (mn_major ? 3u << 15 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | ((128u >> 4) << 24);
}

// The MMA warp: S^T of a chunk once K has landed and the score buffer is read, O^T +=
// V^T P^T once P^T is written and V has landed.
template <typename L>
__device__ __forceinline__ void multiply_scaled(uint8_t* gb, Sync<L> sy, uint32_t tmem) {
  using namespace tcg;
  constexpr int NS = L::NS;
  bool ok = true;
  Units<L> s, o;  // (a unit a chunk)
  s.start(sy, gb, ok);
  o.start(sy, gb, ok);
  int spin = 0;
  int ns0 = 0, ns1 = 0, no0 = 0, no1 = 0;  // S^T and O^T issued per tile
  int pieces_over = 0;                     // pieces whose accumulators are read
  uint64_t t0 = 0;
  auto test = [&](uint32_t bar, int parity) { return __all_sync(FULL, dev::mbar_test(bar, parity & 1)) != 0; };
  auto landed = [&](int i) { return test(sy.full(i % NS), i / NS); };
#pragma unroll 1
  while (o.k.live) {
    bool moved = false;
    if (ns0 + ns1 > no0 + no1) {
      const int t = o.tile, i = o.k.it0 + 2 * o.k.c + 1;
      // (a piece's first products wait for the piece that had its accumulators)
      const bool fresh = o.k.c < 2;
      const int over = fresh ? o.k.i - (L::OPAR - 1) : 0;
      if (pieces_over < over && test(out_free(sy, pieces_over), pieces_over >> 1)) ++pieces_over;
      if (pieces_over >= over && test(sy.pfull(t), t ? no1 : no0) && landed(i)) {
        fence_after();
        const uint32_t id = idesc_f8(L::COLS, true);
        const uint64_t vd = sdesc(sy.base + L::RING + (i % NS) * L::SLOT, 16, 1024);
        const uint64_t pd = sdesc(sy.base + L::P0 + t * 16384, 16, 1024);
        const uint32_t od = tmem + L::COL_O + ((o.k.i & (L::OPAR - 1)) * 2 + t) * L::COLS;
        const uint32_t acc = fresh ? 0u : 1u;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f8(od, vd + ((kk * 4096) >> 4), pd + ((kk * 4096) >> 4), id, kk > 0 ? 1u : acc);
          commit(sy.pdone(t));
          commit(sy.empty(i % NS));
          if (o.k.c + 1 == o.k.nc) commit(out_full(sy, o.k.i));
        }
        __syncwarp();
        ++(t ? no1 : no0);
        o.next(sy, gb, ok);
        moved = true;
      }
    }
    // (Scores two pieces ahead of the products at most: the next piece's plan, which
    // s.next waits for, may wait for the last but three to be over.)
    if (s.k.live && s.k.i - o.k.i <= 2) {
      const int t = s.tile, i = s.k.it0 + 2 * s.k.c, qb = s.k.i & 1, n = t ? ns1 : ns0;
      if ((n == 0 || test(sy.sfree(t), n - 1)) &&
          (s.k.c > 0 || test(sy.qfull(qb), s.k.i >> 1)) && landed(i)) {
        fence_after();
        const uint32_t id = idesc_f8(L::COLS, false);
        const uint64_t kd = sdesc(sy.base + L::RING + (i % NS) * L::SLOT, 16, 1024);
        const uint64_t qd = sdesc(sy.base + qb * L::QTILE, 16, 1024);
        const uint32_t sd = tmem + L::COLS * t;
        const bool over = s.k.c + 1 == s.k.nc;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f8(sd, kd + ((kk * 32) >> 4), qd + ((kk * 32) >> 4), id, kk > 0 ? 1u : 0u);
          commit(sy.sfull(t));
          commit(sy.empty(i % NS));
          if (over) commit(sy.qfree(qb));
        }
        __syncwarp();
        ++(t ? ns1 : ns0);
        s.next(sy, gb, ok);
        moved = true;
      }
    }
    if (moved) {
      spin = 0;
    } else if ((++spin & 63) == 0) {
      const uint64_t t1 = dev::global_timer_ns();
      if (spin == 64) t0 = t1;
      if (uniform(t1 - t0 > kLimit)) {
        ok = false;
        break;
      }
    }
  }
  ok = __all_sync(FULL, ok);
  if (!ok && elect_one()) {
    flag(PA_DEVERR_TIMEOUT);
    commit(sy.mdone());  // products in flight complete before their tensor memory is released
    wait_thread(sy.mdone(), 0);
  }
  __syncwarp();
}

// The terms' columns of 8 rows: on their way, arrived (no use of the registers moves
// above the wait), summed (the small ones first).
struct Terms8 {
  uint32_t a[8], b[8], c[8];
};
__device__ __forceinline__ void terms_load(uint32_t at, int step, Terms8& x) {
#define PA_X8(c, r) c(r[0]), c(r[1]), c(r[2]), c(r[3]), c(r[4]), c(r[5]), c(r[6]), c(r[7])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];"
      : PA_X8("=r", x.a), PA_X8("=r", x.b), PA_X8("=r", x.c)
      : "r"(at), "r"(at + step), "r"(at + 2 * step));
}
__device__ __forceinline__ void terms_wait(Terms8& x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : PA_X8("+r", x.a), PA_X8("+r", x.b), PA_X8("+r", x.c));
#undef PA_X8
}
__device__ __forceinline__ void terms_sum(const Terms8& x, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    auto two = [&](const uint32_t(&r)[8]) { return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])); };
    const float2 s = add2(add2(two(x.c), two(x.b)), two(x.a));
    f[i] = s.x;
    f[i + 1] = s.y;
  }
}
// Of N rows 8 W at a time, the next ones on their way while f sees these: f(row, sums of 8).
template <int N, typename F>
__device__ __forceinline__ void terms_each(uint32_t at, int step, F f) {
  // (16 rows at a time: 32 rows 64 us for 66, 40 rows, which have no registers for the next
  // ones too, 92 for 93)
  constexpr int W = N < 32 ? 1 : 2;
  constexpr bool AHEAD = N <= 32;
  Terms8 x[AHEAD ? 2 : 1][W];
  auto load = [&](int j, Terms8(&y)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (j + 8 * i < N) terms_load(at + j + 8 * i, step, y[i]);
  };
  load(0, x[0]);
#pragma unroll
  for (int j = 0; j < N; j += 8 * W) {
    Terms8(&now)[W] = x[AHEAD ? (j / (8 * W)) & 1 : 0];
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (j + 8 * i < N) terms_wait(now[i]);
    if (AHEAD && j + 8 * W < N) load(j + 8 * W, x[((j / (8 * W)) & 1) ^ 1]);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (j + 8 * i >= N) continue;
      float v[8];
      terms_sum(now[i], v);
      f(j + 8 * i, v);
    }
    if (!AHEAD && j + 8 * W < N) load(j + 8 * W, x[0]);
  }
}

// Sum over the warp's lanes of N values a lane, N a power of two: lane j * (32 / N) gets
// value j's.
template <int N>
__device__ __forceinline__ float lane_sums(float (&v)[N], int lane) {
  int bit = 16;
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int j = 0; j < h; ++j) {
      const float give = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
      v[j] = keep + __shfl_xor_sync(FULL, give, bit);
    }
  }
  float x = v[0];
#pragma unroll
  for (; bit > 0; bit >>= 1) x += __shfl_xor_sync(FULL, x, bit);
  return x;
}

// New references where a row has none yet or an exponent outgrew it; O^T and the
// exponents e move with them.  alpha: what the rows' l are to be multiplied by, in
// scratch[5 R ..], if the result's bit 0 is set.  Bit 1: some row still has no reference.
// (rest: waits until O^T is at rest.)
template <typename L, typename F>
__device__ __forceinline__ int settle_scaled(const KeyLane& x, float (&e)[L::R], float* refs, float lv, uint32_t oc,
                                             bool exists, bool& seen, float& ref, F rest) {
  constexpr int R = L::R;
  const int bar = 2 + x.t;
  float best = -INFINITY;  // of row `lane`
#pragma unroll
  for (int j = 0; j < R; ++j) {
    e[j] -= refs[j];  // (back to the scores; a first chunk's are: its references are 0)
    const float m = warp_max(e[j] + lv);
    if (x.lane == (j & 31)) best = m;
    if (j == 31 && R > 32) x.scratch[R * x.w4 + x.lane] = best;
  }
  if (x.lane < (R > 32 ? R - 32 : R)) x.scratch[R * x.w4 + (R > 32 ? 32 : 0) + x.lane] = best;
  named_bar(bar, 128);
  bool rescale = false;
  if (x.r < R) {
    const float cm = fmaxf(fmaxf(x.scratch[x.r], x.scratch[R + x.r]), fmaxf(x.scratch[2 * R + x.r], x.scratch[3 * R + x.r]));
    float alpha = 1.f;
    if (exists && (seen ? cm > ref + L::MOVE : cm > -INFINITY)) {
      rescale = seen;
      if (seen) alpha = dev::ex2(ref - (cm - L::LIFT));
      ref = cm - L::LIFT;
      seen = true;
    }
    if (exists) refs[x.r] = -ref;
    x.scratch[5 * R + x.r] = alpha;
  }
  const bool unset = bar_or(bar, 128, x.r < R && !seen);
  rescale = bar_or(bar, 128, rescale);
#pragma unroll
  for (int j = 0; j < R; ++j) e[j] += refs[j];
  if (rescale) {
    rest();
#pragma unroll 1
    for (int j = 0; j < kParts * R; j += 8) {
      uint32_t o[8];
      tmem_ld8(oc + j, o);
      const float* by = x.scratch + 5 * R + j % R;
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * by[q]);
      tmem_st8(oc + j, o);
    }
    tcg::wait_st();
  }
  return (rescale ? 1 : 0) | (unset ? 2 : 0);
}

// V rows that not every row sees: those that none does are zeroed, NaN codes in the
// others too, and noted as the first row that sees one.  Thread r has key r's; the rows
// from `from` on see it.
template <typename L>
__device__ __forceinline__ void guard_scaled(const KeyLane& x, uint8_t* vslot, int* poison, int from) {
  uint8_t* row = vslot + x.r * 128;
  if (from <= 0) return;
#pragma unroll 1
  for (int ch = 0; ch < 8; ++ch) {  // (in the order that the lanes' banks differ)
    uint4* at = reinterpret_cast<uint4*>(row + ((ch ^ x.r) & 7) * 16);
    if (from >= L::R) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint32_t w[4] = {at->x, at->y, at->z, at->w}, bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (bad == 0u) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll 1
      for (int sh = 0; sh < 32; sh += 8) {
        if (((w[i] >> sh) & 0x7Fu) != 0x7Fu) continue;
        w[i] &= ~(0xFFu << sh);
        atomicMin(poison + 16 * ch + 4 * i + sh / 8, from);  // (chunk ch of the row is at ch ^ its number)
      }
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The outputs' warpgroup: each piece's queries two pieces ahead, and its rows out once
// both tiles' products have ended: O^T of both times the rows' weights, a thread a dim.
// (The softmax warpgroups go on with the next piece meanwhile: what they did at a
// piece's end themselves took as long as four chunks of 8 rows.)  Of an item that other
// CTAs have parts of, the last to be written is joined with the others by its
// warpgroup, a warp a row, in the order of the parts.
template <typename L>
__device__ __forceinline__ void outputs(const ScaledArgs& sa, uint8_t* gb, Sync<L> sy, uint32_t tmem) {
  constexpr int R = L::R, D = L::D;
  const TreeArgs& a = sa.t;
  const int lane = static_cast<int>(threadIdx.x & 31), w4 = static_cast<int>(threadIdx.x >> 5) & 3, r = 32 * w4 + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * w4) << 16);
  float4* rows = reinterpret_cast<float4*>(gb + L::OUT);  // the weights of a row's two tiles, and where it goes
  bool ok = true;
  Piece p, next[2];  // of this step; and the two whose queries are loaded
  // (sy.piece tells a lane; the warpgroup goes on, or leaves, as a whole)
  auto open = [&](int i, Piece& x) {
    const bool live = sy.piece(gb, i, x, ok);
    ok = !bar_or(4, 128, !ok);
    return ok && live;
  };
  auto bits16 = [&](float o) {
    return sa.q_bf16 ? __bfloat16_as_ushort(__float2bfloat16(o)) : __half_as_ushort(__float2half(o));
  };
  // A piece of an item that has more: its rows are written; the item's are joined, if all are.
  // A part's word holds the launch's stamp once its rows are written.  Who then finds all
  // of the item's words stamped joins the parts: the last to write does, and where
  // another does too, both write the same.  Words are cleared behind it, for a graph that
  // runs the launch again.  (No counter: 150 CTAs that count one up took 70 us.)
  auto join = [&](const Piece& p, int2 part) {
    auto slot_of = [&](int q) { return q == 0 ? 2 * part.x + 1 : 2 * (part.x + q); };
    volatile uint64_t* words = sa.written;
    int* all_written = reinterpret_cast<int*>(rows);
    named_bar(4, 128);
    if (w4 == 0) {
      if (lane == 0) {
        __threadfence();  // (of the whole warpgroup's rows)
        words[p.slot] = sa.stamp;
      }
      __syncwarp();
      asm volatile("fence.sc.gpu;" ::: "memory");  // own word before the others'
      bool all = true;
      for (int q = lane; q < part.y; q += 32) all &= words[slot_of(q)] == sa.stamp;
      all = __all_sync(FULL, all);
      if (all) __threadfence();
      if (lane == 0) *all_written = all;
    }
    named_bar(4, 128);
    const bool last = *all_written != 0;
    named_bar(4, 128);  // (the rows' weights take its place)
    if (!last) return;
    // a warp takes every fourth row, NB of them at a time, two parts of each on their way
    // (3 and 4 rows need more registers than the warps have: 90 and 96 us for 91 in chains, 56 and 58 for 55 elsewhere)
    constexpr int NB = 2;
#pragma unroll 1
    for (int j0 = w4; j0 < p.rows; j0 += 4 * NB) {
      auto row_of = [&](int q, int e) { return static_cast<size_t>(slot_of(q)) * R + min(j0 + 4 * e, p.rows - 1); };
      float M[NB], ls[NB], w[NB];
      float4 acc[NB];
#pragma unroll
      for (int e = 0; e < NB; ++e) {
        M[e] = -INFINITY;
        ls[e] = 0.f;
        acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll 1
      for (int q0 = 0; q0 < part.y; q0 += 32) {  // lane i has part q0 + i's maximum and sum
        const int n = min(32, part.y - q0);
        float4 o[NB][2];
        auto load = [&](int q) {
#pragma unroll
          for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              o[e][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + row_of(q0 + min(q + k, n - 1), e) * D) + lane);
        };
        float m[NB], l[NB];
#pragma unroll
        for (int e = 0; e < NB; ++e) {
          m[e] = lane < n ? __ldcg(a.part_m + row_of(q0 + lane, e)) : -INFINITY;
          l[e] = lane < n ? __ldcg(a.part_l + row_of(q0 + lane, e)) : 0.f;
        }
        load(0);
#pragma unroll
        for (int e = 0; e < NB; ++e) {
          const float top = fmaxf(M[e], warp_max(m[e])), mz = top == -INFINITY ? 0.f : top, again = dev::ex2(M[e] - mz);
          // (a part without a key has no row that counts, but NaN sums have 0 for a maximum)
          w[e] = dev::ex2(m[e] - mz);
          float wl = w[e] * l[e];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) wl += __shfl_xor_sync(FULL, wl, off);
          M[e] = top;
          ls[e] = ls[e] * again + wl;
          acc[e] = make_float4(acc[e].x * again, acc[e].y * again, acc[e].z * again, acc[e].w * again);
        }
#pragma unroll 1
        for (int q = 0;;) {
#pragma unroll
          for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float we = __shfl_sync(FULL, w[e], min(q + k, 31));
              if (q + k >= n) continue;
              acc[e] = make_float4(fmaf(we, o[e][k].x, acc[e].x), fmaf(we, o[e][k].y, acc[e].y),
                                   fmaf(we, o[e][k].z, acc[e].z), fmaf(we, o[e][k].w, acc[e].w));
            }
          q += 2;
          if (q >= n) break;
          load(q);
        }
      }
#pragma unroll
      for (int e = 0; e < NB; ++e) {
        const int j = j0 + 4 * e, head = j & ((1 << a.gl) - 1);
        if (j >= p.rows || head >= a.G) continue;
        const float inv = M[e] == -INFINITY ? 0.f : 1.f / ls[e];
        const size_t at = (static_cast<size_t>((p.qs + ((p.row0 + j) >> a.gl)) * a.Hq + p.g * a.G + head) * D) / 4 + lane;
        const float4 y = make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
        if (a.out_f32)
          static_cast<float4*>(a.out)[at] = y;
        else
          static_cast<uint2*>(a.out)[at] = make_uint2(bits16(y.x) | static_cast<uint32_t>(bits16(y.y)) << 16,
                                                      bits16(y.z) | static_cast<uint32_t>(bits16(y.w)) << 16);
      }
    }
    named_bar(4, 128);
    for (int q = r; q < part.y; q += 128) words[slot_of(q)] = 0ull;
  };
  int loaded = 0;  // pieces whose queries are
  bool more = true, pending = false;  // pending: the piece before has to be joined
  int2 part = make_int2(0, 0);
#pragma unroll 1
  for (int i = 0;; ++i) {
#pragma unroll 1
    for (; more && loaded < i + 2; ++loaded) {
      Piece x;
      more = open(loaded, x);
      if (!more) break;
      load_queries<L>(sa, gb, sy, x, loaded, ok);
      next[0] = next[1];
      next[1] = x;
    }
    // (Not before the next queries are on their way: rows take a while to arrive where others
    // see them, up to 12000 clocks while the ring fills.)
    if (pending) join(p, part);
    if (i >= loaded) break;
    p = loaded == i + 2 ? next[0] : next[1];
    const int pp = i & 1;
    part = reinterpret_cast<const int2*>(gb + L::PARTS)[i & 3];
    if (ok) ok = wait_warp(sums_full(sy, i, 0), (i >> 1) & 1) && wait_warp(sums_full(sy, i, 1), (i >> 1) & 1);
    if (ok) ok = wait_warp(out_full(sy, i), (i >> 1) & 1);
    ok = !bar_or(4, 128, !ok);
    if (!ok) break;
    tcg::fence_after();
    const bool direct = p.slot < 0;
    const int h = r & ((1 << a.gl) - 1);
    if (r < R) {
      const float* top = reinterpret_cast<const float*>(gb + L::TOP) + 2 * R * pp + r;
      const float* sums = reinterpret_cast<const float*>(gb + L::SUM) + 8 * R * pp + r;
      const float l0 = (sums[0] + sums[R]) + (sums[2 * R] + sums[3 * R]);
      const float l1 = (sums[4 * R] + sums[5 * R]) + (sums[6 * R] + sums[7 * R]);
      // (a row that saw only NaN scores has no reference and a sum of NaN)
      const float m0 = top[0] == -INFINITY && l0 != l0 ? 0.f : top[0], m1 = top[R] == -INFINITY && l1 != l1 ? 0.f : top[R];
      const float m = fmaxf(m0, m1), mz = m == -INFINITY ? 0.f : m;
      const float w0 = dev::ex2(m0 - mz), w1 = dev::ex2(m1 - mz), sum = w0 * l0 + w1 * l1;
      const float inv = direct && m != -INFINITY ? 1.f / sum : 1.f;
      // where the row goes, in rows of out or of the partials
      const bool exists = r < p.rows && h < a.G;
      const int at = p.row0 + r;
      const int place = !exists ? -1 : direct ? (p.qs + (at >> a.gl)) * a.Hq + p.g * a.G + h : p.slot * R + r;
      rows[r] = make_float4(w0 * inv, w1 * inv, __int_as_float(place), 0.f);
      if (!direct && exists) {
        a.part_m[place] = m;
        a.part_l[place] = sum;
      }
    }
    int* poison = reinterpret_cast<int*>(gb + L::POISON) + 256 * pp;
    const int nan_from = min(poison[r], poison[128 + r]);
    poison[r] = poison[128 + r] = R;
    named_bar(4, 128);
    const uint32_t oa = tl + L::COL_O + (i & (L::OPAR - 1)) * 2 * L::COLS;
    float* f32 = !direct ? a.part_o : a.out_f32 ? static_cast<float*>(a.out) : nullptr;
#pragma unroll 1
    for (int j0 = 0; j0 < p.rows; j0 += 8) {
      Terms8 tu, tv;
      float u[8], v[8];
      terms_load(oa + j0, R, tu);
      terms_load(oa + L::COLS + j0, R, tv);
      terms_wait(tu);
      terms_wait(tv);
      terms_sum(tu, u);
      terms_sum(tv, v);
      int at[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 row = rows[j0 + e];
        float o = row.x == 0.f ? 0.f : u[e] * row.x;
        if (row.y != 0.f) o = fmaf(v[e], row.y, o);
        u[e] = j0 + e >= nan_from ? NAN : o;
        at[e] = __float_as_int(row.z);
      }
      if (f32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at[e] >= 0) f32[static_cast<size_t>(at[e]) * D + r] = u[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at[e] >= 0) static_cast<uint16_t*>(a.out)[static_cast<size_t>(at[e]) * D + r] = bits16(u[e]);
      }
    }
    tcg::fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(out_free(sy, i));
      mbar_arrive(piece_over(sy, i));
    }
    pending = !direct;
  }
  if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
}

template <int R_>
__global__ void __launch_bounds__(ScaledLay<R_>::THREADS, 1)
    scaled_keys(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ ScaledArgs sa) {
  using namespace tcg;
  using L = ScaledLay<R_>;
  constexpr int R = L::R, NS = L::NS;
  extern __shared__ __align__(1024) uint8_t gb[];
  const TreeArgs& a = sa.t;
  const Sync<L> sy{dev::smem_addr(gb)};
  if (sy.base & 1023u) {  // the swizzled tiles need it; a launch without static shared memory has it
    if (threadIdx.x == 0) flag(PA_DEVERR_TIMEOUT);
    return;
  }
  const int wid = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  if (threadIdx.x == 64) {
    for (int i = 0; i < 8; ++i) dev::mbar_init(scales_full(sy, i), 1);
    for (int i = 0; i < 4; ++i) {
      dev::mbar_init(piece_over(sy, i), 4);
      dev::mbar_init(factors_full(sy, i), 1);
      dev::mbar_init(sums_full(sy, i >> 1, i & 1), 4);
    }
    for (int i = 0; i < 2; ++i) {
      dev::mbar_init(out_full(sy, i), 1);
      dev::mbar_init(out_free(sy, i), 4);
    }
    dev::fence_barrier_init();  // (the products' commits arrive on out_full)
  }
  for (int i = static_cast<int>(threadIdx.x); i < 512; i += L::THREADS) reinterpret_cast<int*>(gb + L::POISON)[i] = R;
  const uint32_t tmem = setup<L>(gb, sy, wid, &tmK, &tmV, &tmK);

  if (wid == 0) {
    fewer_registers<L>();
    produce_scaled<L, false>(a, &tmK, gb, sy);
  } else if (wid == 1) {
    fewer_registers<L>();
    multiply_scaled<L>(gb, sy, static_cast<uint32_t>(uniform(static_cast<int>(tmem))));
  } else if (wid == 2) {
    fewer_registers<L>();
    produce_scaled<L, true>(a, &tmV, gb, sy);
  } else if (wid >= 12) {  // (ahead of the planner: chains of 40 rows 91 us, behind it 93)
    fewer_registers<L>();
    outputs<L>(sa, gb, sy, tmem);
  } else if (wid == 3) {
    fewer_registers<L>();
    plan_scaled<L>(a, gb, sy);
  } else {
    // ---- softmax warpgroups: thread r owns key r of a chunk -----------------------------
    more_registers<L>();
    KeyLane x;
    x.t = (wid - 4) >> 2;
    x.w4 = wid & 3;
    x.lane = lane;
    x.r = 32 * x.w4 + lane;
    x.tl = tmem + (static_cast<uint32_t>(32 * x.w4) << 16);
    uint8_t* pbuf = gb + L::P0 + x.t * 16384;
    x.scratch = reinterpret_cast<float*>(gb + L::SCRATCH) + 6 * R * x.t;
    const int t = x.t, r = x.r, bar = 2 + t;
    uint8_t* prow = pbuf + r * 128;  // the key's row of P^T, swizzled by r & 7
    const uint32_t sc = x.tl + L::COLS * t;
    bool ok = true;
    int n = 0;  // chunks of this tile so far
    Cursor<L> k;
    k.i = k.it0 = k.ph = 0;
#pragma unroll 1
    for (;; k.close()) {
      k.open(sy, gb, ok);
      const Piece& p = k.p;
      const bool exists = r < p.rows && (r & ((1 << a.gl) - 1)) < a.G;  // row r (r < R)
      const int pp = k.i & 1;
      float* refs = reinterpret_cast<float*>(gb + L::REF) + (2 * pp + t) * R;
      if (r < R) refs[r] = exists ? 0.f : -INFINITY;  // (a row that does not exist gets weight 0)
      // The barriers inside a piece have no limit, so where one warp has given up a
      // wait the whole warpgroup leaves, here.
      ok = !bar_or(bar, 128, !ok);
      if (!ok || !__all_sync(FULL, k.live)) break;
      const int shift = p.L - p.n, i0 = p.row0 >> a.gl;  // the item's first token
      const uint32_t oc = x.tl + L::COL_O + ((k.i & (L::OPAR - 1)) * 2 + t) * L::COLS;
      const float* fac = reinterpret_cast<const float*>(gb + L::FAC) + (k.i & 3) * R;
      int* poison = reinterpret_cast<int*>(gb + L::POISON) + 256 * pp;
      bool seen = !exists, unset = true;  // row r has a reference (or does not exist); some row may have none
      float ref = 0.f, l[R];
#pragma unroll
      for (int j = 0; j < R; ++j) l[j] = 0.f;
      const int c_first = (t ^ k.ph) & 1;
      if (ok) ok = wait_warp(factors_full(sy, k.i), (k.i >> 2) & 1);
      // (what the piece notes for the outputs' warpgroup takes the place of the last but one's)
      if (ok && k.i >= 2) ok = wait_warp(out_free(sy, k.i), ((k.i - 2) >> 1) & 1);
#pragma unroll 1
      for (int c = c_first; c < k.nc; c += 2, ++n) {
        const int chunk = (k.it0 >> 1) + c, key = (p.c0 + c) * kKeys + r;
        const bool masked = (p.c0 + c + 1) * kKeys > shift + i0 + 1;
        if (ok) ok = wait_warp(sy.sfull(t), n & 1);
        if (ok) ok = wait_warp(scales_full(sy, chunk), (chunk >> 3) & 1);
        fence_after();
        const float* scales = reinterpret_cast<const float*>(gb + L::SC) + (chunk & 7) * 16;
        const float ks = scales[r >> 4], vsc = scales[8 + (r >> 4)], lv = log2_scale(vsc);
        // the first row that sees the key: those of the first token at or behind it
        const int from = !masked ? 0 : key >= p.L ? R : max(0, min(R, (key - shift - i0) << a.gl));
        float e[R];
        float top = -INFINITY;  // of the exponents, scores less the references
        {
          terms_each<R>(sc, R, [&](int j, const float(&f)[8]) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
              const float4 fa = *reinterpret_cast<const float4*>(fac + j + i);
              const float4 rf = *reinterpret_cast<const float4*>(refs + j + i);
              // (the factors first: a large row's sum times its own is beyond float32 before a small
              // scale takes it back)
              const float2 y = fma2(make_float2(f[i], f[i + 1]), mul2(make_float2(fa.x, fa.y), make_float2(ks, ks)),
                                    make_float2(rf.x, rf.y));
              const float2 z = fma2(make_float2(f[i + 2], f[i + 3]), mul2(make_float2(fa.z, fa.w), make_float2(ks, ks)),
                                    make_float2(rf.z, rf.w));
              e[j + i] = y.x;
              e[j + i + 1] = y.y;
              e[j + i + 2] = z.x;
              e[j + i + 3] = z.y;
            }
          });
          if (masked) {  // whatever the key's score and scale are
#pragma unroll
            for (int j = 0; j < R; ++j) e[j] = j >= from ? e[j] : -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < R; j += 2) top = max3(top, e[j], e[j + 1]);
        }
        if (unset || bar_or(bar, 128, top > L::MOVE - lv)) {
          const int what = settle_scaled<L>(x, e, refs, lv, oc, exists, seen, ref, [&] {
            if (ok && n > 0) ok = wait_warp(sy.pdone(t), (n - 1) & 1);
            fence_after();
          });
          unset = what & 2;
          if (what & 1) {
#pragma unroll
            for (int j = 0; j < R; ++j) l[j] *= x.scratch[5 * R + j];
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.sfree(t));  // the scores and scales are read
        // weights, their sum, and the terms of weight x V scale
        uint32_t out[kParts][R / 4];
#pragma unroll
        for (int j = 0; j < R; j += 4) {
          uint32_t p0[kParts], p1[kParts];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = j + 2 * h;
            const float2 w = make_float2(dev::ex2(e[i]), dev::ex2(e[i + 1]));
            const float2 ll = add2(make_float2(l[i], l[i + 1]), w), y = mul2(w, make_float2(vsc, vsc));
            l[i] = ll.x;
            l[i + 1] = ll.y;
            terms(dev::pack2<__half>(y.x, y.y), h ? p1 : p0);
          }
#pragma unroll
          for (int q = 0; q < kParts; ++q) out[q][j / 4] = upper(p0[q], p1[q]);
        }
        if (ok && n > 0) ok = wait_warp(sy.pdone(t), (n - 1) & 1);  // P^T's buffer is free
        const uint32_t* flat = &out[0][0];
        constexpr int WORDS = kParts * R / 4;
#pragma unroll
        for (int ch = 0; 4 * ch < WORDS; ++ch) {
          uint8_t* to = prow + ((ch ^ (r & 7)) << 4);
          if (4 * ch + 4 <= WORDS)
            *reinterpret_cast<uint4*>(to) = make_uint4(flat[4 * ch], flat[4 * ch + 1], flat[4 * ch + 2], flat[4 * ch + 3]);
          else
            *reinterpret_cast<uint2*>(to) = make_uint2(flat[4 * ch], flat[4 * ch + 1]);
        }
        if (masked) {
          const int vi = k.it0 + 2 * c + 1, vs = vi % NS;
          if (ok) ok = __all_sync(FULL, wait_issued(sy.issued(), chunk)) && wait_warp(sy.full(vs), (vi / NS) & 1);
          guard_scaled<L>(x, gb + L::RING + vs * L::SLOT, poison + 128 * t, from);
        }
        dev::fence_proxy_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.pfull(t));
      }
      // ---- the piece's end --------------------------------------------------------------
      if (p.last) dev::grid_launch_dependents();
      // l over the 128 keys' lanes, and the references, for the outputs' warpgroup
      float* sums = reinterpret_cast<float*>(gb + L::SUM) + ((2 * pp + t) * 4 + x.w4) * R;
      constexpr int R0 = R > 32 ? 32 : R;
      float v[R0];
#pragma unroll
      for (int j = 0; j < R0; ++j) v[j] = l[j];
      const float sum = lane_sums<R0>(v, lane);
      if (lane % (32 / R0) == 0) sums[lane / (32 / R0)] = sum;
      if constexpr (R > 32) {
        float v2[R - 32];
#pragma unroll
        for (int j = 0; j < R - 32; ++j) v2[j] = l[32 + j];
        const float sum2 = lane_sums<R - 32>(v2, lane);
        if (lane % (32 / (R - 32)) == 0) sums[32 + lane / (32 / (R - 32))] = sum2;
      }
      if (r < R) reinterpret_cast<float*>(gb + L::TOP)[(2 * pp + t) * R + r] = exists && seen ? ref : -INFINITY;
      __syncwarp();
      if (lane == 0) mbar_arrive(sums_full(sy, k.i, t));
    }
    if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  }
  teardown(wid, tmem);
}

std::atomic<uint64_t> g_launches{0};  // of every kernel and device: workspaces may go from one to another

// L: a kernel's layout; kernel: with a thread per key it has no map of q.
template <typename L, typename K>
pa_status launch_kernel(const ScaledAttentionLaunch& l, K kernel, cudaStream_t stream) {
  const char* fn = "pa_block_scaled_attention";
  ScaledArgs sa = {};
  TreeArgs& a = sa.t;
  a.q = l.q;
  a.q_start = l.q_start;
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
  a.n_cta = l.n_cta;
  while ((1 << a.gl) < a.G) ++a.gl;
  a.scale_log2 = l.scale * 1.4426950408889634f;
  if (L::ROWS && l.scale < 0.f) {  // the products negate Q
    a.scale_log2 = -a.scale_log2;
    a.negate = 1;
  }
  a.out_f32 = l.out_dtype == PA_DTYPE_F32;
  a.min_units = 6 * L::CHUNK;
  a.item_rows = a.slot_rows = l.item_rows;
  sa.q_stride = l.q_stride;
  sa.q_bf16 = l.q_dtype == PA_DTYPE_BF16;
  const size_t rows = static_cast<size_t>(2) * a.n_cta * a.slot_rows;
  a.part_o = static_cast<float*>(l.workspace);
  a.part_m = a.part_o + rows * L::D;
  a.part_l = a.part_m + rows;
  a.split = reinterpret_cast<int4*>(a.part_l + rows);
  sa.written = reinterpret_cast<uint64_t*>(a.part_l + rows);
  sa.stamp = 0x9E3779B97F4A7C15ull * ++g_launches;  // (odd multiples: no two alike, none 0, no number that memory is full of)

  CUtensorMap tm[3];
  for (int v = 0; v < 2; ++v) {
    const pa_status st = make_kv_map(&tm[v], v ? l.v_cache : l.k_cache, l.Hkv, l.num_blocks, L::D, 1,
                                     CU_TENSOR_MAP_DATA_TYPE_UINT8, fn);
    if (st != PA_OK) return st;
  }
  if constexpr (L::ROWS) {
    const pa_status st = make_q_map(&tm[2], l.q, L::D, l.Hq, l.T, l.q_stride, 1 << a.gl,
                                    sa.q_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, fn);
    if (st != PA_OK) return st;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return fail(PA_ERR_CUDA, "%s: no CUDA device", fn);
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
  if (setup[dev] != cudaSuccess) return fail(PA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(setup[dev]));
  const dim3 grid(static_cast<unsigned>(a.n_cta)), block(L::THREADS);
  cudaError_t e;
  if constexpr (L::ROWS)
    e = launch_dependent(kernel, grid, block, L::BYTES, stream, tm[0], tm[1], tm[2], sa);
  else
    e = launch_dependent(kernel, grid, block, L::BYTES, stream, tm[0], tm[1], sa);
  if constexpr (L::ROWS) {
    if (e == cudaSuccess && l.max_context_len > kKeys) {  // (no item of one chunk is cut)
      const dim3 mgrid(static_cast<unsigned>(a.n_cta), a.slot_rows / kMergeRows), mblock(32 * kMergeRows);
      e = sa.q_bf16 ? launch_dependent(tree_merge<__nv_bfloat16, L::D>, mgrid, mblock, 0, stream, a)
                    : launch_dependent(tree_merge<__half, L::D>, mgrid, mblock, 0, stream, a);
    }
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return PA_OK;
}

}  // namespace

// A thread per key while one kv head's rows fit in 128 columns of three terms, then a
// thread per row.
pa_status launch_scaled_attention(const ScaledAttentionLaunch& l, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (l.item_rows) {
    case 8: return launch_kernel<ScaledLay<8>>(l, scaled_keys<8>, st);
    case 16: return launch_kernel<ScaledLay<16>>(l, scaled_keys<16>, st);
    case 32: return launch_kernel<ScaledLay<32>>(l, scaled_keys<32>, st);
    case 40: return launch_kernel<ScaledLay<40>>(l, scaled_keys<40>, st);
    default:
      return l.q_dtype == PA_DTYPE_BF16 ? launch_kernel<ScaledRowsLay<__nv_bfloat16>>(l, scaled_rows<__nv_bfloat16>, st)
                                        : launch_kernel<ScaledRowsLay<__half>>(l, scaled_rows<__half>, st);
  }
}

pa_status read_errors_scaled_attention(uint32_t* flags, bool clear) {
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
