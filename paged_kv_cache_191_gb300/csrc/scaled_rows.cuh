// The block-scaled kernel with a thread per row: items of up to 128 rows.
//
// S = Q K^T (M = 128 rows, N = the chunk's keys) and O += P V with P in tensor memory,
// as in the tree attention's kernel of this kind, whose MMA warp, converters and
// outputs it shares: a warpgroup converts the codes to f16 in shared memory, which at 128
// rows costs less than three E5M2 terms of Q and P would (products of 128 rows: 1074
// clocks a chunk in f16, 1608 in terms).  bf16 queries become f16 too, a piece's at a
// time, each row by a power of two: with K, V and P in bf16, P as two halves, 4
// sequences of 608 tokens behind 1440 took 192 us where they take 121 (f16: 104), with only
// Q and K in bf16 140 (codes reach bf16 by way of f16 and float32).  Two tiles take turns over
// the chunks.  A block's scale is the same for every row, so that a thread
// with its row's 128 scores in registers multiplies 16 of them by one number, and its
// maximum, reference and sum need no other lane.
//
// Prompt chunks of 300 to 1024 tokens in contexts to 4096, 4 sequences of 32 heads,
// 8 kv heads, f16: 117 to 143 us by which chunk stands in which context, 0.67 to 0.72
// PFLOP/s, 36 to 38 % of the library product's rate (the kernel with a thread per key took
// 4 times that).  Over many sizes that is 2470 clocks a chunk, 11900 an item and 14 us a call.
// A chunk is bound by shared memory: 32 KB of codes in and out again, 64 KB of values, 96 KB
// of operands are 1750 clocks.  An item's are one turn of each tile with nothing beside
// it, its rows' way out and the next one's first references; O has no tensor memory for
// two items.  (Items of 256 rows, half of them each tile's, halve the codes and values per
// row and were no faster: 130 us for 127, 74 for 68 at 33 to 60 tokens.  Nor is it the
// exponentials' unit: with every eighth pair by a polynomial those 130 us were 135.)  At 40 rows,
// from HBM: f16 103 us, bf16 121, where the thread per key takes 89 and 90.
// One prompt makes every sequence of the call an item of this kernel, a single token one
// of 1 to 32 rows of 128: 28 single tokens (32 / 8 heads) beside 4 chunks of 512 97 us, 20 and 71 us
// in two calls; 63 (64 / 8 heads, bf16) beside one of 512 166 us, 54 and 64 in two.
#pragma once

#include "scaled_common.cuh"
#include "tree_rows.cuh"

namespace pa {
namespace {

template <typename T>
struct ScaledRowsLay {
  static constexpr bool Q8 = true, ROWS = true, WORDS = false;
  static constexpr bool SPLIT = false;                // (weights are f16)
  static constexpr int D = 128, SPANS = 2, HQ = 128, QP = 1, R = HQ;
  static constexpr int QTILE = HQ * D * 2;
  static constexpr int SLOT = kKeys * D * 2;          // one K or V chunk, 16-bit
  static constexpr int GRP = 1024 * SPANS;            // 8 keys of a slot: [span][8][128 B]
  static constexpr int RING = QP * QTILE;
  static constexpr int NS = 4, NL = 3, PRODUCERS = 1;  // slots; places that codes land in
  static constexpr int STAGE = RING + NS * SLOT;
  static constexpr int BAR = STAGE + NL * kKeys * D;
  static constexpr int EXTRA = 2 * NL + 2 * NS + 23;
  // bf16 queries are made f16, as the codes are: barriers of four pieces' (f16 ones are as they land)
  static constexpr bool QCONV = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int QREADY = QCONV ? EXTRA + 12 : 0;
  static constexpr int NBAR = EXTRA + 16;             // scales of a chunk, pieces over, queries ready
  static constexpr int MISC = (BAR + NBAR * 8 + 15) & ~15;
  static constexpr int PIECE = MISC + 128;            // Piece [4]
  static constexpr int PUB = PIECE + 4 * 48;          // float2 [2 tiles][HQ]
  static constexpr int SC = PUB + 16 * HQ;            // float [8 chunks][K 8, V 8]
  static constexpr int FAC = SC + 8 * 64;             // float [4 pieces][HQ]: takes back the power of a row of queries
  static constexpr int BYTES = FAC + 16 * HQ;
  static constexpr int THREADS = 512;
  // as in the tree attention's Lay
  static constexpr float LIFT = 7.f, MOVE = 15.f;
  static constexpr int HIGH = 176, LOW = 80;
  static constexpr int CHUNK = 1, ITEM = kItem, LEAST = 0;  // of units: a chunk, an item's start and end, an item at least
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// The producer warp: each piece's Q rows, its chunks' codes, a box per block, and their
// scales.
template <typename L>
__device__ __forceinline__ void produce_rows(const TreeArgs& a, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                             const CUtensorMap* tmQ, uint8_t* gb, Sync<L> sy) {
  constexpr int NL = L::NL;
  const int lane = static_cast<int>(threadIdx.x & 31);
  bool ok = true;
  int chunk = 0, q_issued = 0;
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
  // Q of piece i, once the piece before has ended its last scores: boxes of br rows
  // (whole tokens), a lane per (box, span).
  auto load_q = [&](const Piece& x, int i) {
    if (ok && i >= 1) ok = wait_warp(sy.qfree((i - 1) & 1), ((i - 1) >> 1) & 1);
    if (!ok) return;
    ++q_issued;
    const int br = max(32, 1 << a.gl);
    const int sp = lane % L::SPANS, y = lane / L::SPANS * br;
    const bool mine = y < x.rows;
    const uint32_t n = static_cast<uint32_t>(__popc(__ballot_sync(FULL, mine)));
    if (lane == 0) dev::mbar_arrive_expect_tx(sy.qfull(i & 1), n * br * 128);
    __syncwarp();
    if (mine)
      dev::tma_load_3d(sy.base + (sp * L::HQ + y) * 128, tmQ, sy.qfull(i & 1), sp * 64, x.g * a.G,
                       x.qs + ((x.row0 + y) >> a.gl));
    __syncwarp();
  };
  Piece p, pn;
  bool more = sy.piece(gb, 0, p, ok), more_n = false;
  int ids_next = more ? fetch(p, p.c0 * kBlk) : 0;
  float2 next = make_float2(0.f, 0.f);  // the scales of the lane's block in ids_next
  auto scales = [&](int g) {
    const size_t at = static_cast<size_t>(ids_next) * a.Hkv + g;
    next = make_float2(__ldg(a.k_scale + at), __ldg(a.v_scale + at));
  };
  if (more) scales(p.g);
#pragma unroll 1
  for (int i = 1; more; ++i) {
    p.g = uniform(p.g);
    p.c0 = uniform(p.c0);
    p.c1 = uniform(p.c1);
    const int nblk = uniform((p.L + 15) / 16);
    int ids = 0;
    float2 sc = next;
#pragma unroll 1
    for (int c = p.c0; c < p.c1; ++c) {
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
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        const int it = 2 * chunk + v, s = it % NL;
        if (ok && it >= NL) ok = wait_warp(sy.taken(s), (it / NL - 1) & 1);
        if (!ok) break;
        dev::fence_proxy_async_smem();  // the converters' reads precede the refill
        if (lane == 0) dev::mbar_arrive_expect_tx(sy.full(s), static_cast<uint32_t>(live * 2048));
        __syncwarp();
        const CUtensorMap* m = v ? tmV : tmK;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlk; ++k) {
            if (k >= live) break;
            dev::tma_load_3d(sy.base + L::STAGE + s * (L::SLOT / 2) + k * 2048, m, sy.full(s), 0, p.g * 16, blk[k]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      // (a place of the scales is free: three chunks at most are between here and the softmax)
      if ((lane >> 3) == k4) put_scales(reinterpret_cast<float*>(gb + L::SC) + (chunk & 7) * 16 + (lane & 7), sc);
      __syncwarp();
      if (lane == 0) mbar_arrive(scales_full(sy, chunk));
      ++chunk;
      if (c == p.c0) load_q(p, i - 1);  // (the first chunk goes ahead of the wait for Q's place)
      // what comes behind these 32 blocks: more of the piece, or the next one's first
      if (k4 == 0 && c + 4 >= p.c1) {
        more_n = sy.piece(gb, i, pn, ok);
        if (more_n) ids_next = fetch(pn, pn.c0 * kBlk);
      }
      if (c + 1 == p.c1 ? more_n : k4 == 3) scales(c + 1 == p.c1 ? pn.g : p.g);
    }
    p = pn;
    more = more_n && ok;
  }
  // no copy may still be landing when the CTA exits
  for (int i = max(0, q_issued - 2); i < q_issued; ++i) wait_thread(sy.qfull(i & 1), (i >> 1) & 1);
  for (int i = max(0, 2 * chunk - NL); i < 2 * chunk; ++i) wait_thread(sy.full(i % NL), (i / NL) & 1);
  if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  __syncwarp();
}

// A piece's bf16 queries as f16, in their place, by the converters, a thread a row: scaled by
// a power of two to 2^14 .. 2^15, so that a row of any size keeps its 8 bits.
template <typename L>
struct HalfQueries {
  uint8_t* gb;
  Sync<L> sy;
  __device__ __forceinline__ void operator()(const Piece& p, int i, bool& ok) const {
    const int r = static_cast<int>(threadIdx.x) - 384;
    if (ok) ok = wait_warp(sy.qfull(i & 1), (i >> 1) & 1);
    if (r < p.rows) {
      auto at = [&](int ch) {
        return reinterpret_cast<uint4*>(gb + ((ch >> 3) * L::HQ + r) * 128 + (((ch ^ r) & 7) << 4));
      };
      uint32_t top = 0;
#pragma unroll 4
      for (int ch = 0; ch < 8 * L::SPANS; ++ch) {
        const uint4 w = *at(ch);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                     __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
      }
      top = max(top & 0xFFFFu, top >> 16);
      const bool fine = top < 0x7F80u;  // (else the row's factor is NaN, and so is the row)
      const int k = min(14 - (static_cast<int>(top >> 7) - 127), 100);
      const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
      auto half = [&](uint32_t u) {
        const float2 f = dev::unpack2<__nv_bfloat16>(u);
        return dev::pack2<__half>(f.x * up, f.y * up);
      };
#pragma unroll 4
      for (int ch = 0; ch < 8 * L::SPANS; ++ch) {
        const uint4 w = *at(ch);
        *at(ch) = make_uint4(half(w.x), half(w.y), half(w.z), half(w.w));
      }
      reinterpret_cast<float*>(gb + L::FAC)[(i & 3) * L::HQ + r] =
          fine ? __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : NAN;
    }
    dev::fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(factors_full(sy, i));
  }
};

template <typename T>
__global__ void __launch_bounds__(ScaledRowsLay<T>::THREADS, 1)
    scaled_rows(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ ScaledArgs sa) {
  using namespace tcg;
  using L = ScaledRowsLay<T>;
  constexpr int D = L::D, NS = L::NS;
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
    for (int i = 0; i < 4; ++i) dev::mbar_init(piece_over(sy, i), 8);
    for (int i = 0; i < 4; ++i) dev::mbar_init(factors_full(sy, i), 4);
    dev::fence_barrier_init();
  }
  const uint32_t tmem = setup<L>(gb, sy, wid, &tmK, &tmV, &tmQ);

  if (wid == 0) {
    fewer_registers<L>();
    produce_rows<L>(a, &tmK, &tmV, &tmQ, gb, sy);
  } else if (wid == 1) {
    fewer_registers<L>();
    multiply_rows<__half, L>(a, gb, sy, static_cast<uint32_t>(uniform(static_cast<int>(tmem))));
  } else if (wid == 2) {
    fewer_registers<L>();
  } else if (wid == 3) {
    fewer_registers<L>();
    plan_scaled<L>(a, gb, sy);
  } else if (wid < 12) {
    // ---- softmax warpgroups: thread r owns row r of every other chunk ------------------------
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
    bool ok = true;
    int n = 0;  // chunks of this tile so far
    Cursor<L> k;
    k.i = k.it0 = k.ph = 0;
#pragma unroll 1
    for (;; k.close()) {
      k.open(sy, gb, ok);
      // The barriers inside a piece have no limit: where a warp has given up a wait, both
      // warpgroups leave, here.
      ok = !bar_or(1, 256, !ok);
      if (!ok || !__all_sync(FULL, k.live)) break;
      const Piece& p = k.p;
      const int pp = k.i & 1, shift = p.L - p.n;
      x.live = r - lane < p.rows;
      x.exists = r < p.rows && (r & ((1 << a.gl) - 1)) < a.G;
      x.node = (p.row0 + r) >> a.gl;
      float ref = 0.f, l = 0.f;
      bool seen = false;  // the row has a reference
      const int c_first = (t ^ k.ph) & 1;
      const bool any = c_first < k.nc;
#pragma unroll 1
      for (int c = c_first; c < k.nc; c += 2, ++n) {
        const int key0 = (p.c0 + c) * kKeys, chunk = (k.it0 >> 1) + c;
        const bool masked = key0 + kKeys > shift + (p.row0 >> a.gl) + 1;
        if (ok) ok = wait_warp(sy.sfull(t), n & 1);  // (the tile's products before it have ended too)
        if (ok) ok = wait_warp(scales_full(sy, chunk), (chunk >> 3) & 1);
        if constexpr (L::QCONV) {
          if (ok && c == c_first) ok = wait_warp(factors_full(sy, k.i), (k.i >> 2) & 1);
        }
        fence_after();
        if (x.live) {
          const float4* sc = reinterpret_cast<const float4*>(gb + L::SC + (chunk & 7) * 64);
          const float4 s4[4] = {sc[0], sc[1], sc[2], sc[3]};
          const float ks[8] = {s4[0].x, s4[0].y, s4[0].z, s4[0].w, s4[1].x, s4[1].y, s4[1].z, s4[1].w};
          const float vs[8] = {s4[2].x, s4[2].y, s4[2].z, s4[2].w, s4[3].x, s4[3].y, s4[3].z, s4[3].w};
          float sl2 = a.scale_log2;
          if constexpr (L::QCONV) sl2 *= reinterpret_cast<const float*>(gb + L::FAC)[(k.i & 3) * L::HQ + r];
          float f[kKeys];
          load_scores(x.s, f);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const float kb = ks[b] * sl2;
#pragma unroll
            for (int j = 16 * b; j < 16 * b + 16; j += 2) {
              const float2 y = mul2(make_float2(f[j], f[j + 1]), make_float2(kb, kb));
              f[j] = y.x;
              f[j + 1] = y.y;
            }
          }
          if (masked) {  // whatever the key's score is
            const int last = x.exists ? min(shift + x.node, p.L - 1) - key0 : -1;  // the last key that the row sees
#pragma unroll
            for (int j = 0; j < kKeys; ++j) f[j] = j <= last ? f[j] : -INFINITY;
          }
          // references go by the maximum of weight x V scale, which is what is rounded
          float top = -INFINITY;
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int j = 16 * b; j < 16 * b + 16; j += 4) {
              m0 = max3(m0, f[j], f[j + 1]);
              m1 = max3(m1, f[j + 2], f[j + 3]);
            }
            top = fmaxf(top, fmaxf(m0, m1) + log2_scale(vs[b]));
          }
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
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const int i = 32 * h + 2 * j;
              const float2 v2 = make_float2(vs[i >> 4], vs[i >> 4]);
              const float2 e0 = add2(make_float2(f[i], f[i + 1]), make_float2(-ref, -ref));
              const float2 e1 = add2(make_float2(f[i + 2], f[i + 3]), make_float2(-ref, -ref));
              const float2 w0 = make_float2(dev::ex2(e0.x), dev::ex2(e0.y));
              const float2 w1 = make_float2(dev::ex2(e1.x), dev::ex2(e1.y));
              ls = add2(ls, w0);
              ls1 = add2(ls1, w1);
              const float2 y0 = mul2(w0, v2), y1 = mul2(w1, v2);
              pk[j] = dev::pack2<__half>(y0.x, y0.y);
              pk[j + 1] = dev::pack2<__half>(y1.x, y1.y);
            }
            tmem_st16(x.s + 16 * h, pk);
          }
          l += (ls.x + ls.y) + (ls1.x + ls1.y);
          wait_st();
        }
        if (masked) {
          const int vi = k.it0 + 2 * c + 1, vs = vi % NS;
          if (ok) ok = __all_sync(FULL, wait_issued(sy.issued(), vi)) && wait_warp(sy.ready(vs), (vi / NS) & 1);
          guard_rows<__half, L>(x, gb, gb + L::RING + vs * L::SLOT, (p.c0 + c) & 1, false, key0 + r - shift, p.n,
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
      // a row that saw only NaN scores has no reference and a sum of NaN
      const float m = any && seen ? ref : l != l ? 0.f : -INFINITY;
      // both warpgroups are done with what the piece before published
      if (ok && k.i >= 1) ok = wait_warp(sy.ofree(pp ^ 1), ((k.i - 1) >> 1) & 1);
      pubs[128 * t + r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.pub(t));
      if (ok) ok = wait_warp(sy.pub(t ^ 1), k.i & 1);  // (after that tile's last product)
      fence_after();
      const float2 other = pubs[128 * (t ^ 1) + r];
      const float M = fmaxf(m, other.x), mz = M == -INFINITY ? 0.f : M;
      const float w = dev::ex2(m - mz), w_other = dev::ex2(other.x - mz), sum = w * l + w_other * other.y;
      if (x.live) {
        const float inv = p.slot < 0 && M != -INFINITY ? 1.f / sum : 1.f;
        if (p.slot >= 0 && x.exists && t == 0) {
          a.part_m[p.slot * a.slot_rows + r] = M;
          a.part_l[p.slot * a.slot_rows + r] = sum;
        }
        write_row<T, L>(a, x, p, r, w * inv, w_other * inv, tl + kRowO + 128 * (t ^ 1), true, (D / 2) * t,
                        (D / 2) * (t + 1));
      }
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sy.ofree(pp));
        mbar_arrive(piece_over(sy, k.i));
      }
    }
    if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  } else {
    fewer_registers<L>();
    if constexpr (L::QCONV)
      convert<uint8_t, __half, L>(gb, sy, HalfQueries<L>{gb, sy});
    else
      convert<uint8_t, __half, L>(gb, sy);
  }
  teardown(wid, tmem);
}

}  // namespace
}  // namespace pa
