// Attention over a block-scaled cache: shared memory, the E5M2 terms, the planner, the
// queries and the producers.  The ring, the pieces, the waits and tensor memory's
// access are those of the tree attention.
#pragma once

#include "tree_merge.cuh"

namespace pa {
namespace {

constexpr int kParts = 3;  // E5M2 terms of a query or a weight

struct ScaledArgs {
  TreeArgs t;        // (mask and words are not used; scale_log2 has the scale's sign)
  int64_t q_stride;  // elements between tokens
  int32_t q_bf16;
  uint64_t* written;  // [CTAs][2]: the stamp, where that set of partial rows is written
  uint64_t stamp;     // of this launch
};

// R: rows of an item, 8, 16, 32 or 40.
template <int R_>
struct ScaledLay {
  static constexpr int R = R_, D = 128;
  static constexpr int HQ = INT32_MAX;            // (no piece is split over the tiles)
  static constexpr bool Q8 = false, ROWS = false, WORDS = false;
  static constexpr int PRODUCERS = 1;             // threads that announce a slot's bytes
  static constexpr int COLS = (kParts * R + 15) & ~15;  // columns of a product
  static constexpr int QTILE = ((COLS * D + 1023) & ~1023);  // Q of a piece [term][R][128 B], E5M2
  static constexpr int SLOT = kKeys * D;          // one K or V chunk of codes
  static constexpr int P0 = 2 * QTILE;            // P^T [tile][128 keys][128 B: term, row]
  static constexpr int RING = P0 + 2 * 16384;
  static constexpr int NS = R > 16 ? 8 : 10;      // even: K's and V's producers own every other slot
  static constexpr int NL = NS;
  static constexpr int BAR = RING + NS * SLOT;
  static constexpr int EXTRA = 2 * NL + 2 * NS + 23;
  // scales of a chunk, pieces over, factors of a piece, sums published, O^T at rest, O^T read
  static constexpr int NBAR = EXTRA + 24;
  static constexpr int MISC = (BAR + NBAR * 8 + 15) & ~15;
  static constexpr int PIECE = MISC + 128;        // Piece [4]
  static constexpr int PARTS = PIECE + 4 * 48;    // int2 [4 pieces]: the CTA that has the item's first part, its parts
  static constexpr int SC = PARTS + 4 * 8;        // float [8 chunks][K 8, V 8]
  static constexpr int FAC = SC + 8 * 64;         // float [4 pieces][R]
  static constexpr int REF = FAC + 16 * R;        // float [piece parity][2 tiles][R]: minus the references
  static constexpr int SUM = REF + 16 * R;        // float [piece parity][2 tiles][4 warps][R]: l
  static constexpr int TOP = SUM + 64 * R;        // float [piece parity][2 tiles][R]: the references (-inf: none)
  static constexpr int OUT = TOP + 16 * R;        // the outputs' rows: weights of the two tiles, place
  static constexpr int POISON = OUT + 16 * R;     // int [piece parity][2 tiles][128 dims]: first row that sees a NaN there
  static constexpr int MASK = 0;
  static constexpr int SCRATCH = POISON + 2048;   // float [2 tiles][6][R]: maxima of warps, factors of moved references
  static constexpr int BYTES = SCRATCH + 48 * R;
  static constexpr int THREADS = 512;
  static constexpr int HIGH = 176, LOW = 80;
  // Units of work: a chunk; an item's start and end; an item at least, whose chunks wait for
  // each other.  (ITEM 2, 5, 8, 12: 8 rows, 32 kv heads 57, 55, 57, 58 us, 16 rows 53, 54, 54,
  // 55, 32 rows 75, 70, 67, 67, 40 rows 102, 96, 92, 91.  Without LEAST one short
  // sequence is cut in two, 14 us for 9.)
  static constexpr int CHUNK = 2, ITEM = R > 16 ? 10 : 5, LEAST = 12;
  // tensor memory columns: S^T [tile] x COLS, O^T [piece parity, where there is room][tile] x COLS
  static constexpr int OPAR = R > 16 ? 1 : 2;
  static constexpr uint32_t COL_O = 2 * COLS;
  // log2 of how far below its row's maximum of weight x V scale a reference is set, and
  // of how far that maximum may outgrow it: E5M2 terms of f16 values go from 2^15.8
  // down to 2^-16, rounded: 2^-27 of the largest is the most that a weight is off by
  // beyond its f16 rounding.  (Lower references are outgrown less often, higher ones
  // keep more of small weights.)
  static constexpr float LIFT = 10.f, MOVE = 15.5f;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
  static_assert(COL_O + OPAR * 2 * COLS <= static_cast<int>(kTmemCols), "tensor memory");
};

template <typename L>
__device__ __forceinline__ uint32_t scales_full(const Sync<L>& sy, int chunk) { return sy.at(L::EXTRA + (chunk & 7)); }
// The piece is over.  (Of four pieces each its own: the planner, who waits for the last but
// three, may be more than two behind, and a barrier of every second piece would then have
// gone round.)
template <typename L>
__device__ __forceinline__ uint32_t piece_over(const Sync<L>& sy, int piece) { return sy.at(L::EXTRA + 8 + (piece & 3)); }
template <typename L>
__device__ __forceinline__ uint32_t factors_full(const Sync<L>& sy, int piece) {
  return sy.at(L::EXTRA + 12 + (piece & 3));
}
// A tile's sums and references of the piece are written; its products have ended; its
// accumulators and sums are read.
template <typename L>
__device__ __forceinline__ uint32_t sums_full(const Sync<L>& sy, int piece, int tile) {
  return sy.at(L::EXTRA + 16 + 2 * (piece & 1) + tile);
}
template <typename L>
__device__ __forceinline__ uint32_t out_full(const Sync<L>& sy, int piece) { return sy.at(L::EXTRA + 20 + (piece & 1)); }
template <typename L>
__device__ __forceinline__ uint32_t out_free(const Sync<L>& sy, int piece) { return sy.at(L::EXTRA + 22 + (piece & 1)); }

// What the softmax's rare paths share with its loop.
struct KeyLane {
  int t, w4, lane, r;  // tile, warp of the tile, lane, key of the chunk
  uint32_t tl;         // tensor memory at the warp's lanes
  float* scratch;      // the tile's
};

// ---- E5M2 terms --------------------------------------------------------------
// An f16 value is the sum of three E5M2 ones: E5M2 is f16's upper byte, so a term is
// what is left, rounded to its first three bits.  Of 11 bits a term leaves a rest of
// at most half a step, 2^7 units, the next one 2^3, which the last holds: exact, but
// below 2^-16, E5M2's smallest, where it is rounded.  (Differences are exact.  A NaN
// does not come through: a query's goes by its row's factor, a weight's by its row's sum.)
// h: two values in, the terms' pairs out (their upper bytes count).
__device__ __forceinline__ void terms(uint32_t h, uint32_t (&p)[kParts]) {
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    p[i] = h + 0x00800080u;
    if (i + 1 < kParts) {
      const uint32_t t = p[i] & 0xFF00FF00u;
      const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&t));
      h = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}
// The upper bytes of two pairs.
__device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) { return dev::prmt(a, b, 0x7531u); }

// ---- the batch's work ----------------------------------------------------------
// A sequence's items of one kv head, tpi tokens each; item j sees L - n + (j + 1)
// tpi keys at most, and a chunk beyond is not its work.  (Nor one behind the context:
// where the tokens are more than the keys, n > L, the first of them see none.  So a
// context of one chunk has no item that is cut, and needs no merge.)
struct Span {
  int qs, n, L, tiles;
  int a;  // tokens before the new ones, in items
};
__device__ __forceinline__ int context_chunks(const Span& x) { return max(1, (x.L + kKeys - 1) / kKeys); }
// sum of ceil(x / 2^s) over x = 1 .. m.  (In 32 bits it may wrap; differences, which are
// within what the launch was checked for, are right all the same.)
template <typename U>
__device__ __forceinline__ U ceil_sum(U m, int s) {
  const U q = m >> s, r = m - (q << s);
  return (((q & 1 ? q : q + 1) * (q & 1 ? (q + 1) >> 1 : q >> 1)) << s) + r * (q + 1);
}
// units of the items before item k of a kv head; those that have the whole context are at the
// end.  With a thread per key there is none before another: a sequence's tokens, max_q_len
// at most, are one item (item_rows of the call).
template <typename L, typename U>
__device__ __forceinline__ U units_before(const Span& x, int k, int s) {
  if constexpr (!L::ROWS) {
    return 0;
  } else {
    static_assert(L::LEAST == 0, "the sum has no least units of an item");
    const U all = static_cast<U>(context_chunks(x)), from = static_cast<U>(x.a), to = static_cast<U>(x.a + k);
    const U part = min(to, all << s);  // (from is below that: a context holds the tokens before the new ones)
    return static_cast<U>(L::ITEM) * static_cast<U>(k) +
           static_cast<U>(L::CHUNK) * (ceil_sum(part, s) - ceil_sum(from, s) + (to - part) * all);
  }
}
// chunks of item k; with a thread per key it is the sequence's only one
template <typename L>
__device__ __forceinline__ int chunks_of(const Span& x, int k, int s) {
  const int all = context_chunks(x);
  if constexpr (!L::ROWS) return all;
  return k + 1 < x.tiles ? min((x.a + k + (1 << s)) >> s, all) : all;
}
// units of an item of so many chunks
template <typename L>
__device__ __forceinline__ int item_units(int chunks) {
  return max(L::CHUNK * chunks + L::ITEM, L::LEAST);
}
template <typename L, typename U>
__device__ __forceinline__ U units_per_head(const Span& x, int s) {
  return x.tiles == 0 ? 0 : units_before<L, U>(x, x.tiles - 1, s) + item_units<L>(chunks_of<L>(x, x.tiles - 1, s));
}

// A piece's queries, by the outputs' warpgroup: every row scaled by a power of two to
// 2^14 .. 2^15 (a row of small values keeps its bits beside one of large ones), in E5M2
// terms; its factor takes the power back.  A warp has a quarter of the rows.
template <typename L>
__device__ __forceinline__ void load_queries(const ScaledArgs& sa, uint8_t* gb, Sync<L> sy, const Piece& p, int i, bool& ok) {
  constexpr int R = L::R, EACH = R / 4;
  const TreeArgs& a = sa.t;
  const int lane = static_cast<int>(threadIdx.x & 31), w4 = static_cast<int>(threadIdx.x >> 5) & 3;
  const int heads = (1 << a.gl) - 1;
  // all of a warp's rows on their way at once, a lane's 4 values of each (32 rows: 64 us, in halves
  // 68; a warp waits for each flight up to 3 us while the ring fills)
  uint2 x[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int r = EACH * w4 + j, h = r & heads;
    x[j] = make_uint2(0u, 0u);
    if (r < p.rows && h < a.G)
      x[j] = __ldg(reinterpret_cast<const uint2*>(
          static_cast<const uint16_t*>(a.q) + static_cast<size_t>(p.qs + ((p.row0 + r) >> a.gl)) * sa.q_stride +
          static_cast<size_t>(p.g * a.G + h) * L::D + 4 * lane));
  }
  if (ok && i >= 2) ok = wait_warp(sy.qfree(i & 1), ((i - 2) >> 1) & 1);
  float* fac = reinterpret_cast<float*>(gb + L::FAC) + (i & 3) * R;
  uint8_t* to = gb + (i & 1) * L::QTILE + (lane & 3) * 4;
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int r = EACH * w4 + j;
    const float2 lo = sa.q_bf16 ? dev::unpack2<__nv_bfloat16>(x[j].x) : dev::unpack2<__half>(x[j].x);
    const float2 hi = sa.q_bf16 ? dev::unpack2<__nv_bfloat16>(x[j].y) : dev::unpack2<__half>(x[j].y);
    const float f[4] = {lo.x, lo.y, hi.x, hi.y};
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(FULL, top);
    const bool fine = top < 0x7F800000u;  // (else the row's factor is NaN, and so is the row)
    const int k = min(14 - (static_cast<int>(top >> 23) - 127), 100);
    const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    uint32_t p0[kParts], p1[kParts];
    terms(dev::pack2<__half>(f[0] * up, f[1] * up), p0);
    terms(dev::pack2<__half>(f[2] * up, f[3] * up), p1);
#pragma unroll
    for (int e = 0; e < kParts; ++e)
      *reinterpret_cast<uint32_t*>(to + (e * R + r) * 128 + (((lane >> 2) ^ (r & 7)) << 4)) = upper(p0[e], p1[e]);
    if (lane == 0) fac[r] = fine ? a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : NAN;
  }
  dev::fence_proxy_async_smem();
  named_bar(4, 128);
  if (w4 == 0 && lane == 0) {
    mbar_arrive(sy.qfull(i & 1));
    mbar_arrive(factors_full(sy, i));
  }
  __syncwarp();
}

// The planner warp: this CTA's pieces, published up to four ahead.
template <typename L>
__device__ __forceinline__ void plan_scaled(const TreeArgs& a, uint8_t* gb, Sync<L> sy) {
  const int lane = static_cast<int>(threadIdx.x & 31), me = static_cast<int>(blockIdx.x);
  // tokens of an item; log2 of the items to a chunk (exactly as many of the 128-row ones, whose chunks go by it)
  const int tpi = a.item_rows >> a.gl, per = 31 - __clz(kKeys / tpi);
  // Sequences are read 32 at a time, a lane each.  (The code is kept small, one place for
  // each step: what a CTA runs once should not push the loops out of the caches.)
  Span mine{0, 0, 0, 0, 0};
  int group = -1;
  auto read = [&](int g, bool report) {
    if (g == group) return;
    group = g;
    const int b = 32 * g + lane;
    mine = Span{0, 0, 0, 0, 0};
    if (b >= a.B) return;
    const Seq s = seq_of(a, b, report);
    mine = Span{s.qs, s.n, s.L, s.tiles, (max(0, s.L - s.n) + tpi - 1) / tpi};
  };
  // First all units are summed, then the sequence of this CTA's first one is found.
  int64_t sum = 0;
  int most = 0;  // units of the largest item
  int upc = 0, start = 0, end = 0, b = 0, ub = 0;  // units before sequence b: ub
#pragma unroll 1
  for (int g = 0, find = 0;; ++g) {
    if (32 * g >= a.B) {
      if (find) break;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL, sum, off);
      most = __reduce_max_sync(FULL, most);
      // more than the launch was checked for: q_start has ranges that overlap
      if (sum > kMaxUnits && me == 0 && lane == 0) flag(PA_DEVERR_QUERY_RANGE);
      const int total = sum > kMaxUnits ? 0 : static_cast<int>(sum);
      // Few units: equal parts of the largest item, of min_units at least.  (Joining parts takes
      // 2 us and more: a sequence of 600 tokens 8.9 us whole, 11.1 in parts of 2 units; one of
      // 32768 with one kv head 37 us in parts of 2, 21 in parts of 6.)
      upc = (total + a.n_cta - 1) / a.n_cta;
      if (upc < a.min_units) upc = max(a.min_units, (most + max(1, most / a.min_units) - 1) / max(1, most / a.min_units));
      start = static_cast<int>(min(static_cast<int64_t>(me) * upc, static_cast<int64_t>(total)));
      end = min(start + upc, total);
      if (start >= end) break;
      find = 1;
      g = 0;
    }
    read(g, me == 0);
    const int64_t units = units_per_head<L, int64_t>(mine, per) * a.Hkv;
    if (!find) {
      sum += units;
      if (mine.tiles > 0) most = max(most, item_units<L>(chunks_of<L>(mine, mine.tiles - 1, per)));
      continue;
    }
    const int w = static_cast<int>(units);
    int inc = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(FULL, inc, off);
      if (lane >= off) inc += y;
    }
    const unsigned over = __ballot_sync(FULL, ub + inc > start);
    const int f = over ? __ffs(over) - 1 : 31;
    ub += __shfl_sync(FULL, over ? inc - w : inc, f);
    if (over) {
      b = 32 * g + f;
      break;
    }
  }
  Piece* ring = reinterpret_cast<Piece*>(gb + L::PIECE);
  // the item at unit u: tile `tile` of kv head g of sequence b, which is s; `off` of
  // its units are gone
  Span s{0, 0, 0, 0, 0};
  int u = start, g = 0, tile = 0, off = 0, seq = -1;
  bool ok = true, more = true;
  int4 sp0 = make_int4(0, 0, 0, 0), sp1 = sp0;
#pragma unroll 1
  for (int i = 0; more; ++i) {
    if (i >= 4) ok = wait_warp(piece_over(sy, i), ((i - 4) >> 2) & 1);
    if (!ok) break;  // (what is still read is not written over: the others' waits run out in turn)
    Piece p;
    p.live = 0;
#pragma unroll 1
    while (u < end && !p.live) {
      if (seq != b) {  // (b stays below B: its units cover those of the range)
        const int from = b & 31;
        read(b >> 5, false);
        s = Span{__shfl_sync(FULL, mine.qs, from), __shfl_sync(FULL, mine.n, from), __shfl_sync(FULL, mine.L, from),
                 __shfl_sync(FULL, mine.tiles, from), __shfl_sync(FULL, mine.a, from)};
        if (s.tiles == 0 && b + 1 < a.B) {
          ++b;
          continue;
        }
        if (seq < 0) {  // the CTA's first item
          const int U = max(1, static_cast<int>(units_per_head<L, uint32_t>(s, per))), at = start - ub;
          g = at / U;
          off = at - g * U;
          if constexpr (L::ROWS) {
            int hi = s.tiles;  // the last that starts at or before it
#pragma unroll 1
            while (hi - tile > 1) {
              const int mid = (tile + hi) >> 1;
              if (static_cast<int>(units_before<L, uint32_t>(s, mid, per)) <= off)
                tile = mid;
              else
                hi = mid;
            }
            off -= static_cast<int>(units_before<L, uint32_t>(s, tile, per));
          }
        }
        seq = b;
      }
      // a chunk is whose range its first unit lies in
      const int nch = chunks_of<L>(s, tile, per), cost = item_units<L>(nch), stop = min(cost, off + end - u);
      const int first = cost - L::CHUNK * nch;
      p.c0 = max(0, off - first + L::CHUNK - 1) / L::CHUNK;
      p.c1 = max(0, stop - first + L::CHUNK - 1) / L::CHUNK;
      if (p.c1 > p.c0) {  // (else the range ends before the item's first chunk)
        p.live = 1;
        p.b = b;
        p.qs = s.qs;
        p.n = s.n;
        p.L = s.L;
        p.g = g;
        p.row0 = tile * a.item_rows;
        p.rows = min(a.item_rows, (s.n << a.gl) - p.row0);
        // partial rows: an item's first part has the CTA's second set, a later one the first
        p.slot = p.c0 == 0 && p.c1 == nch ? -1 : 2 * me + (p.c0 == 0 ? 1 : 0);
        const int owner = (u - off + first) / upc, parts = (u - off + cost - L::CHUNK) / upc - owner + 1;
        if constexpr (!L::ROWS) {
          if (lane == 0) reinterpret_cast<int2*>(gb + L::PARTS)[i & 3] = make_int2(owner, parts);
        } else if (p.c0 == 0 && p.c1 < nch) {  // the item goes on in the next CTAs: what the merge needs
          sp0 = make_int4(parts, p.slot, s.qs, p.row0);
          sp1 = make_int4(g, p.rows, 1, 0);
        }
      }
      u += stop - off;
      off = 0;  // (the item's end, or the range's)
      if (++tile >= s.tiles) {
        tile = 0;
        if (++g >= a.Hkv) {
          g = 0;
          ++b;
        }
      }
    }
    p.last = u >= end;  // (or only an item's start is left)
    more = p.live;
    if (lane == 0) {
      ring[i & 3] = p;
      mbar_arrive(sy.pieces(i & 3));
    }
    __syncwarp();
  }
  if (lane == 0) {
    if constexpr (L::ROWS) {
      a.split[2 * blockIdx.x] = sp0;
      a.split[2 * blockIdx.x + 1] = sp1;
    }
    if (!ok) flag(PA_DEVERR_TIMEOUT);
  }
}

// A block's scales (K, V) into their places.  A V scale that is no number is to meet no
// weight but of the tokens that see the block: theirs become NaN by K's.
__device__ __forceinline__ void put_scales(float* to, float2 s) {
  const bool fine = fabsf(s.y) < INFINITY;
  to[0] = fine ? s.x : NAN;
  to[8] = fine ? s.y : 0.f;
}

// The producer warps, one for K (and both tensors' scales) and one for V: a piece's
// chunks into their slots of the ring, one 2 KB box per block.
template <typename L, bool V>
__device__ __forceinline__ void produce_scaled(const TreeArgs& a, const CUtensorMap* map, uint8_t* gb, Sync<L> sy) {
  constexpr int NS = L::NS;
  const int lane = static_cast<int>(threadIdx.x & 31);
  bool ok = true;
  int chunk = 0;  // chunks issued
  // Loads behind a full ring take microseconds, so the ids of the next 32 blocks, and
  // their scales, are fetched well ahead.
  auto fetch = [&](const Piece& x, int j0) {  // lane's block id, blocks j0 .. j0 + 31 of the piece
    const int j = j0 + lane;
    if (j >= min((x.L + 15) / 16, x.c1 * kBlk)) return 0;
    int v = a.block_tables[static_cast<size_t>(x.b) * a.max_blocks + j];
    if (v < 0 || v >= a.num_blocks) {
      flag(PA_DEVERR_BLOCK_RANGE);  // block 0 is read instead; flagged
      v = 0;
    }
    return v;
  };
  Piece p, pn;
  bool more = sy.piece(gb, 0, p, ok), more_n = false;
  int ids_next = more ? fetch(p, p.c0 * kBlk) : 0;
  float2 next = make_float2(0.f, 0.f);  // the scales of the lane's block in ids_next
  auto scales = [&](int g) {
    const size_t at = static_cast<size_t>(ids_next) * a.Hkv + g;
    next = make_float2(__ldg(a.k_scale + at), __ldg(a.v_scale + at));
  };
  if (!V && more) scales(p.g);
#pragma unroll 1
  for (int i = 1; more; ++i) {
    p.g = uniform(p.g);
    p.c0 = uniform(p.c0);
    p.c1 = uniform(p.c1);
    const int nblk = uniform((p.L + 15) / 16);
    int ids = 0;
    float2 sc = next;
#pragma unroll 1
    for (int c = p.c0; c < p.c1; ++c, ++chunk) {
      const int k4 = (c - p.c0) & 3;
      if (k4 == 0) {
        ids = ids_next;
        sc = next;
        if (c + 4 < p.c1) ids_next = fetch(p, (c + 4) * kBlk);
      }
      int blk[kBlk];  // the chunk's block ids
#pragma unroll
      for (int k = 0; k < kBlk; ++k) blk[k] = __shfl_sync(FULL, ids, k4 * kBlk + k);
      const int live = max(0, min(kBlk, nblk - c * kBlk));  // those that exist
      const int it = 2 * chunk + (V ? 1 : 0), s = it % NS;
      if (ok && it >= NS) ok = wait_warp(sy.empty(s), (it / NS - 1) & 1);
      if (!ok) break;
      dev::fence_proxy_async_smem();  // the softmax's accesses precede the refill
      const uint32_t bar = sy.full(s), dst = sy.base + L::RING + s * L::SLOT;
      if (lane == 0) {
        dev::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live * 2048));
        if (V) publish(sy.issued(), chunk + 1);
      }
      __syncwarp();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kBlk; ++k) {
          if (k >= live) break;
          dev::tma_load_3d(dst + k * 2048, map, bar, 0, p.g * 16, blk[k]);
        }
      }
      __syncwarp();
      if (!V) {
        // (a place is free: its chunk's scores were read before those two chunks on were computed)
        float* to = reinterpret_cast<float*>(gb + L::SC) + (chunk & 7) * 16;
        if ((lane >> 3) == k4) put_scales(to + (lane & 7), sc);
        __syncwarp();
        if (lane == 0) mbar_arrive(scales_full(sy, chunk));
      }
      // what comes behind these 32 blocks: more of the piece, or the next one's first (asked
      // for once this chunk is on its way: its plan may still be made)
      if (k4 == 0 && c + 4 >= p.c1) {
        more_n = sy.piece(gb, i, pn, ok);
        if (more_n) ids_next = fetch(pn, pn.c0 * kBlk);
      }
      if (!V && (c + 1 == p.c1 ? more_n : k4 == 3)) scales(c + 1 == p.c1 ? pn.g : p.g);
    }
    p = pn;
    more = more_n && ok;
  }
  // no copy may still be landing when the CTA exits
  for (int c = max(0, chunk - NS / 2); c < chunk; ++c) {
    const int it = 2 * c + (V ? 1 : 0);
    wait_thread(sy.full(it % NS), (it / NS) & 1);
  }
  if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  __syncwarp();
}

}  // namespace
}  // namespace pa
