// The tree-attention kernel with a thread per row: items of up to 256 rows.
//
// S = Q K^T (M = 128 rows, N = the chunk's keys) and O += P V, P in tensor memory
// in the place of the scores it came from (bf16 weights' low halves in columns 64 ..,
// and another product with V).  Two tiles of 128 rows take turns,
// one in its products while the other is in its softmax: an item of up to 128
// rows gives each tile every other chunk (own accumulator, own references,
// joined at the item's end), a larger one gives each tile half of its rows and
// every chunk.  A thread holds its row's 128 scores in registers: its maximum,
// reference and sum need no other lane, and O moves with the reference inside
// the warp.  1-byte caches have scales per key: there a thread holds 2 columns of
// 8 of 2 rows at a time (the MMA fragment), so that 4 scales serve 8 rows of a
// read, and their items are up to 128 rows (the stages of codes take the room).
//
// A tile's cycle is softmax (~1500 clocks a chunk), P V and the next scores (~600
// each) and the waits between them (~1000); two tiles in turns keep the tensor pipe
// busy 57 % of it (512 rows, by its counter).  P V in two halves, the first issued before the second
// half's weights exist, was slower (357 us for 334 then), and so were two softmax
// warpgroups per tile (345 us for 334, and 130 for 110): 104 registers a thread spill.
//   64 sequences of 8 kv heads, 128 rows, bf16, mean context 2064: 120 us, 4.8
//   TB/s, 71 % of the copy rate: HBM, the launch and merge (10 us), and V's slot of the
//   ring, which both halves of the weights hold longer (6 us their softmax, 4 us their
//   product).
//   8 sequences of 8 kv heads, 512 rows, f16, contexts to 32768: 323 us, 1.27
//   PFLOP/s, 66 % of the library product's burst rate: the cycle above.  Repeated for
//   seconds 345 us, 61 % (68 % of the sustained rate): the board's power limit (1370 W,
//   1.94 GHz of 2.07).
//   8 sequences of 8 kv heads, 96 .. 128 rows, E4M3, contexts to 32768: 131 us,
//   3.1 TB/s, 46 % of the copy rate: shared memory, ~83 % of whose cycles are taken
//   by codes in (32 KB a chunk, read again), their conversion out (64 KB), the
//   MMAs' operands (96 KB) and the scales (64 KB).
#pragma once

#include "tree_common.cuh"

namespace pa {
namespace {

// tensor memory columns: scores [tile] x 128, O [tile] x 128
constexpr uint32_t kRowS = 0, kRowO = 256;

// A walk over the units of all pieces, in order: the chunks, or two (one per
// tile) of each chunk.  Units alternate between the tiles.
template <typename L>
struct Units {
  Cursor<L> k;
  int j, tile;  // unit of the chunk
  __device__ __forceinline__ void settle() {
    k.live = uniform(k.live);
    k.nc = uniform(k.nc);
    k.p.rows = uniform(k.p.rows);
    k.both = k.p.rows > L::HQ;
  }
  __device__ __forceinline__ void start(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    k.start(sy, gb, ok);
    j = tile = 0;
    settle();
  }
  __device__ __forceinline__ bool ends_chunk() const { return !k.both || j == 1; }
  __device__ __forceinline__ bool ends_piece() const { return ends_chunk() && k.c + 1 == k.nc; }
  __device__ __forceinline__ void next(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    tile ^= 1;
    if (!ends_chunk()) {
      j = 1;
      return;
    }
    j = 0;
    if (k.next(sy, gb, ok)) settle();
  }
};

// The MMA warp: a unit's scores once K has landed and its tile's last product is
// issued (products complete in order), O += P V once P is written and V has
// landed.  The same arrangement as with a thread per key: one warp that waits on
// all barriers in order, converged, on uniform values, one elected lane issuing.
template <typename T, typename L>
__device__ __forceinline__ void multiply_rows(const TreeArgs& a, uint8_t* gb, Sync<L> sy, uint32_t tmem) {
  using namespace tcg;
  constexpr int NS = L::NS, D = L::D;
  volatile uint32_t* force = reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 32);
  bool ok = true;
  Units<L> s, o;
  s.start(sy, gb, ok);
  o.start(sy, gb, ok);
  int ahead = 0, spin = 0;     // units whose scores are issued and O not
  int no0 = 0, no1 = 0;        // O issued per tile
  int pieces_over = 0;         // pieces that both warpgroups are done with
  uint64_t t0 = 0;
  auto test = [&](uint32_t bar, int parity) { return __all_sync(FULL, dev::mbar_test(bar, parity & 1)) != 0; };
  const uint32_t id_s = idesc<T>(kKeys, false) | (a.negate << 13), id_o = idesc<T>(D, true);
  // The ring items of the next scores and the next O: slot, and parity of its fill.
  int ks = 0, kf = 0, vs = 1, vf = 0;
  auto advance = [](int& slot, int& fill) {
    slot += 2;
    if (slot >= NS) {
      slot -= NS;
      fill ^= 1;
    }
  };
  auto scores = [&](int slot, int tile, int place, bool last) {  // by one thread
    const uint64_t kd = sdesc(sy.base + L::RING + slot * L::SLOT, 16, L::GRP);
    const uint64_t qd = sdesc(sy.base + place * L::QTILE, 16, 1024);
    const uint32_t sd = tmem + kRowS + 128 * tile;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      mma_ss(sd, qd + (((kk >> 2) * (L::HQ * 128) + (kk & 3) * 32) >> 4),
             kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_s, kk > 0 ? 1u : 0u);
    commit(sy.sfull(tile));
    if (last) commit(sy.empty(slot));
  };
  auto product = [&](int slot, int tile, uint32_t acc, bool last) {
    const uint64_t vd = sdesc(sy.base + L::RING + slot * L::SLOT, D == 128 ? 1024 : 0, L::GRP);
    const uint32_t od = tmem + kRowO + 128 * tile, pd = tmem + kRowS + 128 * tile;
#pragma unroll
    for (int kk = 0; kk < kBlk; ++kk)
      mma_ts(od, pd + 8 * kk, vd + ((kk * 2 * L::GRP) >> 4), id_o, kk > 0 ? 1u : acc);
    if constexpr (L::SPLIT) {
#pragma unroll
      for (int kk = 0; kk < kBlk; ++kk) mma_ts(od, pd + 64 + 8 * kk, vd + ((kk * 2 * L::GRP) >> 4), id_o, 1u);
    }
    commit(sy.pdone(tile));
    if (last) commit(sy.empty(slot));
  };
  bool k_ok = false, v_ok = false;  // all but its turn is there for the next scores, O
#pragma unroll 1
  while (o.k.live) {
    bool moved = false;
    // 1-byte caches: the middle of a piece in a fixed order and in little code, a
    // tile's product, then its next scores.  (What the general steps below do
    // between two groups of MMAs takes 300 to 400 clocks.  8 sequences of 8 kv heads,
    // 128 rows, E4M3: 132 us for 138.  16-bit caches, closer to the copy rate, lose by
    // waiting for K before the other tile's product: 335 us for 328 at 512 rows.)
    // (Their pieces have one unit per chunk.)
    if (L::Q8 && ahead == 2 && s.k.i == o.k.i && o.k.c >= 2 && s.k.c + 1 < s.k.nc) {
      const int count = s.k.nc - 1 - s.k.c;
      int t = uniform(o.tile), n = uniform(t ? no1 : no0), n_other = uniform(t ? no0 : no1);
#pragma unroll 1
      for (int u = 0; u < count; ++u) {
        ok = wait_warp(sy.pfull(t), n & 1) && wait_warp(sy.ready(vs), vf);
        if (!ok) break;
        fence_after();
        if (elect_one()) product(vs, t, 1u, true);
        __syncwarp();
        advance(vs, vf);
        ok = wait_warp(sy.ready(ks), kf);
        if (!ok) break;
        fence_after();
        if (elect_one()) scores(ks, t, s.k.i % L::QP, true);
        __syncwarp();
        advance(ks, kf);
        t ^= 1;
        const int x = n + 1;
        n = n_other;
        n_other = x;
      }
      if (!ok) break;
      no0 = t ? n_other : n;
      no1 = t ? n : n_other;
      o.tile = s.tile = t;
      o.k.c += count;
      s.k.c += count;
      k_ok = v_ok = false;
      continue;
    }
    // Scores first: a tile's follow its product without a look at the other tile.
    // What a step needs besides its turn is tested ahead of it, while idle.
    auto q_ready = [&](int i) {
      if constexpr (L::QREADY > 0)
        return test(sy.at(L::QREADY + (i & 3)), i >> 2);
      else
        return test(sy.qfull(i & 1), i >> 1);
    };
    if (s.k.live && !k_ok) k_ok = s.j > 0 || ((s.k.c > 0 || q_ready(s.k.i)) && test(sy.ready(ks), kf));
    if (k_ok && ahead < 2) {
      fence_after();
      const bool last = s.ends_chunk(), over = s.ends_piece();
      if (elect_one()) {
        scores(ks, s.tile, s.k.both ? s.tile : s.k.i % L::QP, last);
        if (over) commit(sy.qfree(s.k.i & 1));
      }
      __syncwarp();
      ++ahead;
      if (last) advance(ks, kf);
      s.next(sy, gb, ok);
      k_ok = false;
      moved = true;
    }
    if (ahead > 0) {
      const int t = o.tile;
      if (!v_ok) {
        // a tile's first product of a piece overwrites the O of the piece before
        if (o.k.c < 2 && pieces_over < o.k.i && test(sy.ofree(pieces_over & 1), pieces_over >> 1)) ++pieces_over;
        v_ok = (o.k.c >= 2 || pieces_over >= o.k.i) && (o.j > 0 || test(sy.ready(vs), vf));
      }
      if (v_ok && test(sy.pfull(t), t ? no1 : no0)) {
        fence_after();
        uint32_t acc = 1;
        if (o.k.c < (o.k.both ? 1 : 2)) {  // the tile's first chunk: O starts, unless rows were added by hand
          acc = uniform(force[t]);
          if (acc && elect_one()) force[t] = 0;
        }
        const bool last = o.ends_chunk();
        if (elect_one()) product(vs, t, acc, last);
        __syncwarp();
        ++(t ? no1 : no0);
        --ahead;
        if (last) advance(vs, vf);
        o.next(sy, gb, ok);
        v_ok = false;
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

// A thread's row of a piece.
struct Row {
  int t, w4, lane, r;  // tile, warp of the tile, lane, tensor memory lane
  uint32_t s, o;       // tensor memory: its scores, its O
  bool live, exists;   // the warp has a row; the thread has one
  int node;            // of the sequence
  const uint64_t* mask;  // its mask row
  uint64_t m0, m1;     // the row's words 0 and 1
};
// Visibility of the 32 keys from node j0 on (the context's before 0, none from n on).
__device__ __forceinline__ uint32_t sees(const TreeArgs& a, const Row& x, int j0, int n) {
  if (j0 <= -32) return FULL;
  if (j0 >= n) return 0u;
  auto word = [&](int w) -> uint64_t { return w == 0 ? x.m0 : w == 1 ? x.m1 : w < a.words ? x.mask[w] : 0ull; };
  if (j0 < 0) {
    uint32_t m = static_cast<uint32_t>(x.m0 << -j0);
    if (n - j0 < 32) m &= (1u << (n - j0)) - 1u;
    return m | ((1u << -j0) - 1u);
  }
  const int w = j0 >> 6, sh = j0 & 63;
  uint64_t m = word(w) >> sh;
  if (sh > 32) m |= word(w + 1) << (64 - sh);
  return static_cast<uint32_t>(m) & (n - j0 < 32 ? (1u << (n - j0)) - 1u : FULL);
}

// V rows that must not reach the product: past the context's end, or a node's
// with an infinity or NaN.  Thread r checks key r (jn: its node).  Such a node is
// added to O by hand, where its weight, in tensor memory, is not 0.
template <typename T, typename L>
__device__ __forceinline__ void guard_rows(const Row& x, uint8_t* gb, uint8_t* vslot, int parity, bool both, int jn,
                                           int n, bool fresh) {
  volatile uint32_t* force = reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 32);
  volatile uint32_t* bw =
      reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 64) + parity * 8 + (both ? 0 : 4 * x.t);
  const bool scan = !both || x.t == 0;
  const int bar = both ? 1 : 2 + x.t, bar_n = both ? 256 : 128;
  uint8_t* vrow = vslot + (x.r >> 3) * L::GRP + (x.r & 7) * 128;
  auto clear = [&]() {  // (in the order that the lanes' banks differ)
#pragma unroll 4
    for (int ch = 0; ch < 8 * L::SPANS; ++ch)
      *reinterpret_cast<uint4*>(vrow + (ch >> 3) * 1024 + ((ch ^ x.r) & 7) * 16) = make_uint4(0, 0, 0, 0);
  };
  if (scan) {
    bool bad = false;
    if (jn >= n) {
      clear();
    } else if (jn >= 0) {
#pragma unroll 4
      for (int ch = 0; ch < 8 * L::SPANS; ++ch) {
        const uint4 v = *reinterpret_cast<const uint4*>(vrow + (ch >> 3) * 1024 + ((ch ^ x.r) & 7) * 16);
        bad |= bad16<T>(v.x) | bad16<T>(v.y) | bad16<T>(v.z) | bad16<T>(v.w);
      }
    }
    const uint32_t word = __ballot_sync(FULL, bad);
    if (x.lane == 0) bw[x.w4] = word;
    dev::fence_proxy_async_smem();
  }
  named_bar(bar, bar_n);
  if (!(bw[0] | bw[1] | bw[2] | bw[3])) return;
  const bool first = fresh;
#pragma unroll 1
  for (int key = 0; key < kKeys; ++key) {
    if (!((bw[key >> 5] >> (key & 31)) & 1u)) continue;
    auto weight = [&](uint32_t column) {
      uint32_t p;
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                   : "=r"(p)
                   : "r"(x.s + column)
                   : "memory");
      const float2 pp = dev::unpack2<T>(p);
      return key & 1 ? pp.y : pp.x;
    };
    float w = weight(key >> 1);
    if constexpr (L::SPLIT) w += weight(64 + (key >> 1));
    const uint8_t* vk = vslot + (key >> 3) * L::GRP + (key & 7) * 128;
#pragma unroll 1
    for (int d = 0; d < L::D; d += 8) {
      uint32_t u[8];
      tmem_ld8(x.o + d, u);
      const uint4 q = *reinterpret_cast<const uint4*>(vk + (d >> 6) * 1024 + ((((d & 63) >> 3) ^ (key & 7)) << 4));
      const uint32_t v2[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = e & 1 ? dev::unpack2<T>(v2[e >> 1]).y : dev::unpack2<T>(v2[e >> 1]).x;
        const float o0 = fresh ? 0.f : __uint_as_float(u[e]);
        u[e] = __float_as_uint(w == 0.f ? o0 : o0 + w * v);
      }
      tmem_st8(x.o + d, u);
    }
    tcg::wait_st();
    fresh = false;
  }
  if (first && x.r == 0) force[x.t] = 1;  // the product adds to O
  named_bar(bar, bar_n);                  // every reader is done with the rows
  if (scan && ((bw[x.w4] >> x.lane) & 1u)) clear();
  dev::fence_proxy_async_smem();
  named_bar(bar, bar_n);
}

// O of the warp's rows times alpha, a row per lane.
template <typename L>
__device__ __forceinline__ void rescale(const Row& x, float alpha) {
#pragma unroll 1
  for (int d = 0; d < L::D; d += 8) {
    uint32_t u[8];
    tmem_ld8(x.o + d, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
    tmem_st8(x.o + d, u);
  }
}
// Two rows of a quad of lanes (1-byte caches: thread 4 a + b has columns 8 i + 2 b
// and + 1 of rows a and a + 8, so that a key's scales are read once for many rows).
struct Pair {
  float ref0, ref1;   // references
  float l0, l1;       // sums over the thread's columns
  bool seen0, seen1;  // the row has a reference
  bool has0, has1;    // the row exists
};
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(FULL, v, 1));
  return fmaxf(v, __shfl_xor_sync(FULL, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(FULL, v, 1);
  return v + __shfl_xor_sync(FULL, v, 2);
}
// Of four rows a quad (a, a + 8, a + 16, a + 24), the value of row `lane`.
__device__ __forceinline__ float to_lane(int lane, float v0, float v1, float v2, float v3) {
  const int from = 4 * (lane & 7);
  const float a = __shfl_sync(FULL, v0, from), b = __shfl_sync(FULL, v1, from);
  const float c = __shfl_sync(FULL, v2, from), d = __shfl_sync(FULL, v3, from);
  return lane < 16 ? (lane < 8 ? a : b) : (lane < 24 ? c : d);
}

// Dims [d0, d1) of the thread's row out: O of one tile, or of both, times their
// weights.
template <typename T, typename L>
__device__ __forceinline__ void write_row(const TreeArgs& a, const Row& x, const Piece& p, int row, float w,
                                          float w_other, uint32_t o_other, bool other, int d0, int d1) {
  const bool direct = p.slot < 0, narrow = direct && !a.out_f32;
  const int h = (p.row0 + row) & ((1 << a.gl) - 1);
  const size_t at = direct ? static_cast<size_t>(p.qs + x.node) * a.Hq + p.g * a.G + h
                           : static_cast<size_t>(p.slot) * a.slot_rows + row;
  float* to32 = (direct ? static_cast<float*>(a.out) : a.part_o) + at * L::D;
  T* to16 = static_cast<T*>(a.out) + at * L::D;
#pragma unroll 1
  for (int d = d0; d < d1; d += 8) {
    uint32_t u[8], v[8];
    tmem_ld8(x.o + d, u);
    if (other) tmem_ld8(o_other + d, v);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = w == 0.f ? 0.f : __uint_as_float(u[e]) * w;
      if (other && w_other != 0.f) f[e] = fmaf(__uint_as_float(v[e]), w_other, f[e]);
    }
    if (!x.exists) continue;
    if (narrow) {
      *reinterpret_cast<uint4*>(to16 + d) = make_uint4(dev::pack2<T>(f[0], f[1]), dev::pack2<T>(f[2], f[3]),
                                                       dev::pack2<T>(f[4], f[5]), dev::pack2<T>(f[6], f[7]));
    } else {
      *reinterpret_cast<float4*>(to32 + d) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(to32 + d + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
  __syncwarp();
}

// The weights of a chunk over a 1-byte cache: 16 rows at a time, as fragments.
// K's scales go on the scores and V's, once l has summed the weights, on them;
// only that product is rounded.  References go by its maximum: it is taken against
// them as they are, and again where it turns out to have outgrown one.
template <typename T, typename L>
__device__ __forceinline__ void soften(const TreeArgs& a, const Row& x, const uint8_t* gb, const Piece& p, int piece,
                                       Pair& ra, Pair& rb, const uint8_t* scales, bool masked, int j0, int tile_row,
                                       float sl2) {
  constexpr float kMost = static_cast<float>(1 << static_cast<int>(L::MOVE)), kHuge = 0x1p101f;
  const int b2 = 2 * (x.lane & 3);
  const float2* ks = reinterpret_cast<const float2*>(scales + b2 * 4);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const uint32_t sc = x.s + (static_cast<uint32_t>(16 * h) << 16);
    float2 ls0, ls1;
    uint32_t pk[32], low[L::SPLIT ? 32 : 1];
    bool settle = __any_sync(FULL, (ra.has0 && !ra.seen0) || (ra.has1 && !ra.seen1));
#pragma unroll 1
    for (;; settle = true) {
      uint32_t u[64];
      tmem_ld_frag(sc, u);
      float2 f[32];  // [i][row]
#pragma unroll
      for (int i = 0; i < 32; ++i)
        f[i] = mul2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), ks[4 * (i >> 1)]);
      if (masked) {  // whatever the key's score is
#pragma unroll 1
        for (int y = 0; y < 2; ++y) {
          const int r = tile_row + 32 * x.w4 + 16 * h + 8 * y + (x.lane >> 2);
          const bool has = y ? ra.has1 : ra.has0;
          Row z;
          z.node = (p.row0 + r) >> a.gl;
          z.mask = a.mask + static_cast<size_t>(p.qs + z.node) * a.words;
          const uint64_t* words = reinterpret_cast<const uint64_t*>(gb + L::MASK) + (piece & 1) * 64;
          z.m0 = !has ? 0ull : p.n <= 64 ? words[z.node] : z.mask[0];
          z.m1 = !has || p.n <= 64 ? 0ull : z.mask[1];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            // bits 8 i and 8 i + 1: the row sees the thread's two keys of group i
            const uint32_t m = (has ? sees(a, z, j0 + 32 * w, p.n) : 0u) >> b2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool s0 = (m >> (8 * i)) & 1u, s1 = (m >> (8 * i + 1)) & 1u;
              float2 &g0 = f[2 * (4 * w + i)], &g1 = f[2 * (4 * w + i) + 1];
              if (y == 0) g0 = make_float2(s0 ? g0.x : -INFINITY, s1 ? g0.y : -INFINITY);
              if (y == 1) g1 = make_float2(s0 ? g1.x : -INFINITY, s1 ? g1.y : -INFINITY);
            }
          }
        }
      }
      if (settle) {  // references from the maxima of score + log2 V scale; O and l follow
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 v = ks[64 + 2 * i], lg = make_float2(log2_scale(v.x), log2_scale(v.y));
          const float2 z0 = fma2(f[i], make_float2(sl2, sl2), lg), z1 = fma2(f[i + 1], make_float2(sl2, sl2), lg);
          t0 = max3(t0, z0.x, z0.y);
          t1 = max3(t1, z1.x, z1.y);
        }
        t0 = quad_max(t0);
        t1 = quad_max(t1);
        const bool move0 = ra.has0 && (ra.seen0 ? t0 > ra.ref0 + L::MOVE : t0 > -INFINITY);
        const bool move1 = ra.has1 && (ra.seen1 ? t1 > ra.ref1 + L::MOVE : t1 > -INFINITY);
        if (__any_sync(FULL, (move0 && ra.seen0) || (move1 && ra.seen1))) {
          const float a0 = move0 && ra.seen0 ? dev::ex2(ra.ref0 - (t0 - L::LIFT)) : 1.f;
          const float a1 = move1 && ra.seen1 ? dev::ex2(ra.ref1 - (t1 - L::LIFT)) : 1.f;
          ra.l0 *= a0;
          ra.l1 *= a1;
          rescale<L>(x, h ? to_lane(x.lane, 1.f, 1.f, a0, a1) : to_lane(x.lane, a0, a1, 1.f, 1.f));
        }
        ra.ref0 = move0 ? t0 - L::LIFT : ra.ref0;
        ra.ref1 = move1 ? t1 - L::LIFT : ra.ref1;
        ra.seen0 |= move0;
        ra.seen1 |= move1;
      }
      const float2 n0 = make_float2(-ra.ref0, -ra.ref0), n1 = make_float2(-ra.ref1, -ra.ref1);
      float t0 = 0.f, t1 = 0.f;
      ls0 = ls1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 e = fma2(f[i], make_float2(sl2, sl2), i & 1 ? n1 : n0);
        const float2 w = make_float2(dev::ex2(e.x), dev::ex2(e.y));
        const float2 y = mul2(w, ks[64 + 4 * (i >> 1)]);
        if (i & 1) {
          ls1 = add2(ls1, w);
          t1 = max3(t1, fabsf(y.x), fabsf(y.y));
        } else {
          ls0 = add2(ls0, w);
          t0 = max3(t0, fabsf(y.x), fabsf(y.y));
        }
        pk[i] = dev::pack2<T>(y.x, y.y);
        if constexpr (L::SPLIT) low[i] = low_half(y, pk[i]);
      }
      // (Beside a V scale of 0 a weight may outgrow float32 unseen by its product.)
      if (settle || !__any_sync(FULL, (ra.has0 && !(t0 <= kMost && ls0.x + ls0.y <= kHuge)) ||
                                          (ra.has1 && !(t1 <= kMost && ls1.x + ls1.y <= kHuge))))
        break;
    }
    ra.l0 += ls0.x + ls0.y;
    ra.l1 += ls1.x + ls1.y;
    tmem_st_frag(sc, pk);
    if constexpr (L::SPLIT) tmem_st_frag(sc + 64, low);
    const Pair other = rb;  // the other 16 rows' turn (and back)
    rb = ra;
    ra = other;
  }
  tcg::wait_st();
}

template <typename KT, typename T, int D>
__global__ void __launch_bounds__(Lay<KT, T, D, true>::THREADS, 1)
    tree_rows(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TreeArgs a) {
  using namespace tcg;
  using L = Lay<KT, T, D, true>;
  constexpr bool Q8 = L::Q8;
  constexpr int NS = L::NS;
  extern __shared__ __align__(1024) uint8_t gb[];
  const Sync<L> sy{dev::smem_addr(gb)};
  if (sy.base & 1023u) {  // the swizzled tiles need it; a launch without static shared memory has it
    if (threadIdx.x == 0) flag(PA_DEVERR_TIMEOUT);
    return;
  }
  const int wid = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const uint32_t tmem = setup<L>(gb, sy, wid, &tmK, &tmV, &tmQ);

  if (wid == 0) {
    fewer_registers<L>();
    produce<KT, L>(a, &tmK, &tmV, &tmQ, gb, sy, 0);
  } else if (wid == 1) {
    fewer_registers<L>();
    multiply_rows<T, L>(a, gb, sy, static_cast<uint32_t>(uniform(static_cast<int>(tmem))));
  } else if (wid == 2) {
    fewer_registers<L>();
    if constexpr (L::PRODUCERS == 2) produce<KT, L>(a, &tmK, &tmV, &tmQ, gb, sy, 1);
  } else if (wid == 3) {
    fewer_registers<L>();
    plan<L>(a, gb, sy);
  } else if (wid < 12) {
    // ---- softmax warpgroups: thread r owns row r of its tile -----------------------------
    more_registers<L>();
    Row x;
    x.t = (wid - 4) >> 2;
    x.w4 = wid & 3;
    x.lane = lane;
    x.r = 32 * x.w4 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * x.w4) << 16);
    x.s = tl + kRowS + 128 * x.t;
    x.o = tl + kRowO + 128 * x.t;
    const int t = x.t, r = x.r;
    float2* pubs = reinterpret_cast<float2*>(gb + L::PUB);
    const float sl2 = a.scale_log2;
    bool ok = true;
    int n = 0;  // units of this tile so far
    Cursor<L> k;
    k.i = k.it0 = k.ph = 0;
#pragma unroll 1
    for (;; k.close()) {
      k.open(sy, gb, ok);
      // The barriers inside a piece, of one or both warpgroups, have no limit: where a
      // warp has given up a wait, both warpgroups leave, here.
      ok = !bar_or(1, 256, !ok);
      if (!ok || !__all_sync(FULL, k.live)) break;
      const Piece& p = k.p;
      const int row = (k.both ? 128 * t : 0) + r, pp = k.i & 1, shift = p.L - p.n;
      x.live = row - lane < p.rows;
      x.exists = row < p.rows && ((p.row0 + row) & ((1 << a.gl) - 1)) < a.G;
      x.node = (p.row0 + row) >> a.gl;
      x.mask = a.mask + static_cast<size_t>(p.qs + x.node) * a.words;
      const bool tree = !Q8 && x.exists && p.c1 * kKeys > shift;  // (else every key of the piece is the context's)
      x.m0 = tree ? x.mask[0] : 0ull;
      x.m1 = tree && a.words > 1 ? x.mask[1] : 0ull;
      float ref = 0.f, l = 0.f;
      bool seen = false;  // the row has a reference
      Pair ra, rb;        // 1-byte caches: of rows a, a + 8 of the warp and a + 16, a + 24
      if constexpr (Q8) {
        ra = Pair{0.f, 0.f, 0.f, 0.f, false, false, false, false};
        rb = ra;
        const unsigned has = __ballot_sync(FULL, x.exists);
        ra.has0 = (has >> (lane >> 2)) & 1u;
        ra.has1 = (has >> ((lane >> 2) + 8)) & 1u;
        rb.has0 = (has >> ((lane >> 2) + 16)) & 1u;
        rb.has1 = (has >> ((lane >> 2) + 24)) & 1u;
      }
      const int c_first = k.both ? 0 : (t ^ k.ph) & 1, step = k.both ? 1 : 2;
      const bool any = c_first < k.nc;
#pragma unroll 1
      for (int c = c_first; c < k.nc; c += step, ++n) {
        const int key0 = (p.c0 + c) * kKeys;
        const bool masked = key0 + kKeys > shift;
        if (ok) ok = wait_warp(sy.sfull(t), n & 1);  // (the tile's products before it have ended too)
        fence_after();
        if constexpr (Q8) {
          if (masked) {
            if (p.n <= 64 && ok) ok = wait_warp(sy.mfull(pp), (k.i >> 1) & 1);
            // A V scale that is no number (stale past the end, or a node's) is to meet no
            // weight but of the rows that see its key: theirs become NaN by K's.
            float* ksc = reinterpret_cast<float*>(gb + L::SCALES + (((k.it0 >> 1) + c) & 7) * 1024) + r;
            if (!(fabsf(ksc[128]) < INFINITY)) {
              ksc[0] = nanf("");
              ksc[128] = 0.f;
            }
            named_bar(2 + t, 128);
          }
          if (x.live)
            soften<T, L>(a, x, gb, p, k.i, ra, rb, gb + L::SCALES + (((k.it0 >> 1) + c) & 7) * 1024, masked,
                         key0 - shift, row - x.r, sl2);
        } else if (x.live) {
          float f[kKeys];
          load_scores(x.s, f);
          if (masked) {  // whatever the key's score is
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t m = x.exists ? sees(a, x, key0 + 32 * w - shift, p.n) : 0u;
#pragma unroll
              for (int j = 0; j < 32; ++j) f[32 * w + j] = (m >> j) & 1u ? f[32 * w + j] : -INFINITY;
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < kKeys; j += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) m4[q] = max3(m4[q], f[j + q], f[j + 4 + q]);
          const float top = max3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * sl2;
          const bool move = x.exists && (seen ? top > ref + L::MOVE : top > -INFINITY);
          if (__any_sync(FULL, move && seen)) {  // O and l follow the reference
            const float alpha = move && seen ? dev::ex2(ref - (top - L::LIFT)) : 1.f;
            l *= alpha;
            rescale<L>(x, alpha);
          }
          if (move) {
            ref = top - L::LIFT;
            seen = true;
          }
          float2 ls = make_float2(0.f, 0.f), ls1 = ls;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[16], low[L::SPLIT ? 16 : 1];  // (16 pairs at a time: 8 took 126 us for 120, 32 took 130)
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const int i = 32 * h + 2 * j;
              const float2 e0 = fma2(make_float2(f[i], f[i + 1]), make_float2(sl2, sl2), make_float2(-ref, -ref));
              const float2 e1 = fma2(make_float2(f[i + 2], f[i + 3]), make_float2(sl2, sl2), make_float2(-ref, -ref));
              const float2 w0 = make_float2(dev::ex2(e0.x), dev::ex2(e0.y));
              const float2 w1 = make_float2(dev::ex2(e1.x), dev::ex2(e1.y));
              pk[j] = dev::pack2<T>(w0.x, w0.y);
              pk[j + 1] = dev::pack2<T>(w1.x, w1.y);
              if constexpr (L::SPLIT) {
                low[j] = low_half(w0, pk[j]);
                low[j + 1] = low_half(w1, pk[j + 1]);
                ls = add2(ls, w0);
                ls1 = add2(ls1, w1);
              } else {
                add16x2<T>(ls, pk[j]);  // l sums the rounded weights
                add16x2<T>(ls1, pk[j + 1]);
              }
            }
            tmem_st16(x.s + 16 * h, pk);
            if constexpr (L::SPLIT) tmem_st16(x.s + 64 + 16 * h, low);
          }
          l += (ls.x + ls.y) + (ls1.x + ls1.y);
          wait_st();
        }
        if (masked) {
          const int vi = k.it0 + 2 * c + 1, vs = vi % NS;
          if (ok) ok = __all_sync(FULL, wait_issued(sy.issued(), vi)) && wait_warp(sy.ready(vs), (vi / NS) & 1);
          guard_rows<T, L>(x, gb, gb + L::RING + vs * L::SLOT, (p.c0 + c) & 1, k.both, key0 + r - shift, p.n,
                           c == c_first);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.pfull(t));
      }
      // ---- the piece's end --------------------------------------------------------------
      if (p.last) dev::grid_launch_dependents();
      if (ok && any) ok = wait_warp(sy.pdone(t), (n - 1) & 1);  // O final
      fence_after();
      if constexpr (Q8) {
        l = to_lane(lane, quad_sum(ra.l0), quad_sum(ra.l1), quad_sum(rb.l0), quad_sum(rb.l1));
        ref = to_lane(lane, ra.ref0, ra.ref1, rb.ref0, rb.ref1);
        seen = to_lane(lane, ra.seen0, ra.seen1, rb.seen0, rb.seen1) != 0.f;
      }
      // a row that saw only NaN scores has no reference and a sum of NaN
      const float m = any && seen ? ref : l != l ? 0.f : -INFINITY;
      float M = m, w = m == -INFINITY ? 0.f : 1.f, w_other = 0.f, sum = l;
      if (!k.both) {
        // both warpgroups are done with what the piece before published
        if (ok && k.i >= 1) ok = wait_warp(sy.ofree(pp ^ 1), ((k.i - 1) >> 1) & 1);
        pubs[128 * t + r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.pub(t));
        if (ok) ok = wait_warp(sy.pub(t ^ 1), k.i & 1);  // (after that tile's last product)
        fence_after();
        const float2 other = pubs[128 * (t ^ 1) + r];
        M = fmaxf(m, other.x);
        const float mz = M == -INFINITY ? 0.f : M;
        w = dev::ex2(m - mz);
        w_other = dev::ex2(other.x - mz);
        sum = w * l + w_other * other.y;
      } else {
        __syncwarp();
        if (ok && k.i >= 1) ok = wait_warp(sy.ofree(pp ^ 1), ((k.i - 1) >> 1) & 1);
        if (lane == 0) mbar_arrive(sy.pub(t));
        if (ok) ok = wait_warp(sy.pub(t ^ 1), k.i & 1);
      }
      if (x.live) {
        const float inv = p.slot < 0 && M != -INFINITY ? 1.f / sum : 1.f;
        if (p.slot >= 0 && x.exists && (k.both || t == 0)) {
          a.part_m[p.slot * a.slot_rows + row] = M;
          a.part_l[p.slot * a.slot_rows + row] = sum;
        }
        write_row<T, L>(a, x, p, row, w * inv, w_other * inv, tl + kRowO + 128 * (t ^ 1), !k.both,
                        k.both ? 0 : (D / 2) * t, k.both ? D : (D / 2) * (t + 1));
      }
      if (Q8 && ok) ok = wait_warp(sy.mfull(pp), (k.i >> 1) & 1);  // (every phase is seen in order)
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.ofree(pp));
    }
    if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  } else if (Q8) {
    fewer_registers<L>();
    convert<KT, T, L>(gb, sy);
  }
  teardown(wid, tmem);
}

}  // namespace
}  // namespace pa
