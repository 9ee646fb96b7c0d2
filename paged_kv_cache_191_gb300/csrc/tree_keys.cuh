// The tree-attention kernel with a thread per key: items of up to 64 rows (32 with
// bf16 weights: their low halves are columns 32 .. of P^T, and O^T's columns 32
// .. their product, added at the end).
//
// The products are transposed: S^T = K Q^T (M = the chunk's 128 keys, N = rows)
// and O^T += V^T P^T (M = dims, N = rows), so the tensor cores and the
// exponentials do work in proportion to the rows, 16 at a time, and a whole
// warpgroup is busy however few they are.  Thread r of a warpgroup owns key r
// of the chunk: a key's scales are its own registers, P^T leaves through shared
// memory (one 128-byte row per key), and an output column needs no exchange
// between lanes.  The two warpgroups take alternate chunks, each with its own
// accumulator and references, and the one that had the last chunk joins the two
// while the other starts on the next piece.
//
// A row's reference goes by the maximum of the first chunk in which it sees a key
// (Lay::LIFT), kept in tensor memory beside the scores (read as cheaply as they are,
// where shared memory, which feeds the MMAs, has no bandwidth to spare); it moves,
// O^T and l with it, only when a later maximum outgrows it by 8 octaves.
//
// Bound by HBM.  32 sequences of 32 kv heads, 9 .. 26 nodes, f16, mean context
// 1044: 101 us, 5.5 TB/s, 82 % of the copy rate; what is missing is the launch,
// the merge (8 us together) and the ~5000 cycles around the first and the last
// chunk of an item, of which a CTA has 7 here.  With contexts of 2048 .. 4096 it
// reaches 86 %.
#pragma once

#include "tree_common.cuh"

namespace pa {
namespace {

// tensor memory columns: S^T [tile] x 64, minus the references [tile] x 64, O^T
// [piece parity][tile] x 64
constexpr uint32_t kColS = 0, kColR = 128, kColO = 256;

// The MMA warp: S^T of a chunk once K has landed and the score buffer is
// read, O^T += V^T P^T once P^T is written and V has landed.  It alone waits on
// those barriers, in order, so their parities are unambiguous.  The warp runs
// converged on values that the compiler can see are uniform, and one elected
// lane issues: operands then sit in uniform registers (fetching them from a
// lane's registers cost about 100 cycles an MMA).
template <typename T, typename L>
__device__ __forceinline__ void multiply(const TreeArgs& a, uint8_t* gb, Sync<L> sy, uint32_t tmem) {
  using namespace tcg;
  constexpr int NS = L::NS, D = L::D;
  volatile uint32_t* force = reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 32);
  bool ok = true;
  Cursor<L> s, o;
  auto same = [&](Cursor<L>& x) {
    x.live = uniform(x.live);
    x.p.rows = uniform(x.p.rows);
    x.nc = uniform(x.nc);
  };
  s.start(sy, gb, ok);
  o.start(sy, gb, ok);
  same(s);
  same(o);
  int ahead = 0, spin = 0;                 // chunks whose S^T is issued and O^T not
  int ns0 = 0, ns1 = 0, no0 = 0, no1 = 0;  // S^T and O^T issued per tile
  int pieces_over = 0;                     // pieces that both warpgroups are done with
  uint64_t t0 = 0;
  auto test = [&](uint32_t bar, int parity) { return __all_sync(FULL, dev::mbar_test(bar, parity & 1)) != 0; };
  auto landed = [&](int i) { return test(sy.ready(i % NS), i / NS); };
#pragma unroll 1
  while (o.live) {
    bool moved = false;
    if (ahead > 0) {
      const int t = o.tile(), i = o.it0 + 2 * o.c + 1;
      if (test(sy.pfull(t), t ? no1 : no0) && landed(i)) {
        fence_after();
        // A = V^T (M-major), B = P^T (N-major)
        const int n = ((o.p.rows + 15) & ~15) + (L::SPLIT ? 32 : 0);
        const uint32_t id = idesc<T>(n, true) | (1u << 15);
        const uint64_t vd = sdesc(sy.base + L::RING + (i % NS) * L::SLOT, D == 128 ? 1024 : 0, L::GRP);
        const uint64_t pd = sdesc(sy.base + L::P0 + t * 16384, 16384, 1024);
        const uint32_t od = tmem + kColO + 128 * (o.i & 1) + 64 * t;
        const uint32_t forced = uniform(force[t]);
        const uint32_t acc = o.c >= 2 || forced ? 1u : 0u;
        if (elect_one()) {
          if (forced) force[t] = 0;
#pragma unroll
          for (int kk = 0; kk < kBlk; ++kk)
            mma_ss(od, vd + ((kk * 2 * L::GRP) >> 4), pd + ((kk * 2048) >> 4), id, kk > 0 ? 1u : acc);
          commit(sy.pdone(t));
          commit(sy.empty(i % NS));
        }
        __syncwarp();
        ++(t ? no1 : no0);
        --ahead;
        if (o.next(sy, gb, ok)) same(o);
        moved = true;
      }
    }
    if (s.live && ahead < 2) {
      const int t = s.tile(), i = s.it0 + 2 * s.c, qb = s.i & 1;
      // The tile's last scores are read.  A first chunk also waits for the piece
      // before last to be over, whose O^T its piece will overwrite.
      const int n = t ? ns1 : ns0, over = s.c == 0 ? s.i - 1 : 0;
      if (pieces_over < over && test(sy.ofree(pieces_over & 1), pieces_over >> 1)) ++pieces_over;
      if (pieces_over >= over && (n == 0 || test(sy.sfree(t), n - 1)) &&
          (s.c > 0 || test(sy.qfull(qb), s.i >> 1)) && landed(i)) {
        fence_after();
        const uint32_t id = idesc<T>((s.p.rows + 15) & ~15, false) | (a.negate << 14);
        const uint64_t kd = sdesc(sy.base + L::RING + (i % NS) * L::SLOT, 16, L::GRP);
        const uint64_t qd = sdesc(sy.base + s.i % L::QP * L::QTILE, 16, 1024);
        const uint32_t sd = tmem + kColS + 64 * t;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(sd, kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                   qd + (((kk >> 2) * (L::HQ * 128) + (kk & 3) * 32) >> 4), id, kk > 0 ? 1u : 0u);
          commit(sy.sfull(t));
          commit(sy.empty(i % NS));
          if (s.c + 1 == s.nc) commit(sy.qfree(qb));
        }
        __syncwarp();
        ++(t ? ns1 : ns0);
        ++ahead;
        if (s.next(sy, gb, ok)) same(s);
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

// What the softmax's rare paths share with its loop.
struct Lane {
  int t, w4, lane, r;   // tile, warp of the tile, lane, key of the chunk
  uint32_t tl;          // tensor memory at the warp's lanes
  float* scratch;       // the tile's P^T buffer, between a product's end and the next P^T
};

// The rows (bits) that see the lane's key, node jn of its sequence.  (64 rows: at
// most 64 nodes, a mask word each.)
template <typename L>
__device__ __forceinline__ uint2 visible(const TreeArgs& a, const uint8_t* gb, const Piece& p, int piece, int jn) {
  uint32_t vis[2] = {0u, 0u};
  const uint64_t* words = reinterpret_cast<const uint64_t*>(gb + L::MASK) + (piece & 1) * 64;
  const uint32_t each = a.gl >= 5 ? FULL : (1u << (1 << a.gl)) - 1u;
  const int per = a.gl >= 5 ? 1 : 32 >> a.gl;  // nodes of a word
  if (jn < 0) return make_uint2(FULL, FULL);
  if (jn >= p.n) return make_uint2(0u, 0u);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int n0 = (32 * w) >> a.gl, cnt = min(per, p.n - n0);
#pragma unroll 2
    for (int i = 0; i < cnt; ++i) {
      if ((words[n0 + i] >> jn) & 1) vis[w] |= each << (i << a.gl);
    }
  }
  return make_uint2(vis[0], vis[1]);
}

// New references from the scores in tensor memory, where a row has none yet or
// an exponent outgrew it; O^T moves with them.  alpha: what the rows' l are to
// be multiplied by, in scratch[320 ..], if the result's bit 0 is set.  Bit 1:
// some row still has no reference.
template <typename L>
__device__ __forceinline__ int settle(const Lane& x, uint32_t sc, float ks, float lv, uint2 vis, int words, uint32_t oc,
                                      bool exists, bool& seen, float& ref) {
  const int bar = 2 + x.t;
  float best0 = -INFINITY, best1 = -INFINITY;  // of rows lane, 32 + lane
#pragma unroll 1
  for (int j = 0; j < 32 * words; j += 8) {
    uint32_t u[8];
    tmem_ld8(sc + j, u);
    const uint32_t v = (j & 32 ? vis.y : vis.x) >> (j & 31);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = warp_max((v >> e) & 1u ? fmaf(__uint_as_float(u[e]), ks, lv) : -INFINITY);
      if (x.lane == (j & 31) + e) {
        if (j & 32)
          best1 = m;
        else
          best0 = m;
      }
    }
  }
  x.scratch[64 * x.w4 + x.lane] = best0;
  x.scratch[64 * x.w4 + 32 + x.lane] = best1;
  named_bar(bar, 128);
  bool rescale = false;
  if (x.r < 32 * words) {
    const float cm =
        fmaxf(fmaxf(x.scratch[x.r], x.scratch[64 + x.r]), fmaxf(x.scratch[128 + x.r], x.scratch[192 + x.r]));
    float alpha = 1.f;
    if (exists && (seen ? cm > ref + L::MOVE : cm > -INFINITY)) {
      rescale = seen;
      if (seen) alpha = dev::ex2(ref - (cm - L::LIFT));
      ref = cm - L::LIFT;
      seen = true;
    }
    x.scratch[256 + x.r] = exists ? -ref : -INFINITY;  // rows that do not exist get weight 0
    x.scratch[320 + x.r] = alpha;
  }
  rescale = bar_or(bar, 128, rescale);
#pragma unroll 1
  for (int j = 0; j < 32 * words; j += 8) {
    const uint4* f = reinterpret_cast<const uint4*>(x.scratch + 256 + j);
    const uint32_t u[8] = {f[0].x, f[0].y, f[0].z, f[0].w, f[1].x, f[1].y, f[1].z, f[1].w};
    tmem_st8(x.tl + kColR + 64 * x.t + j, u);
    if (rescale) {
#pragma unroll 1
      for (int at = j; at < (L::SPLIT ? 64 : 32 * words); at += L::SPLIT ? 32 : 64) {
        uint32_t o[8];
        tmem_ld8(oc + at, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * x.scratch[320 + j + e]);
        tmem_st8(oc + at, o);
      }
    }
  }
  tcg::wait_st();
  const bool unset = bar_or(bar, 128, x.r < 64 && !seen);
  return (rescale ? 1 : 0) | (unset ? 2 : 0);
}

// V rows that must not reach the product: past the context's end, or a node's
// with an infinity or NaN.  Thread r checks key r.  Such a node is added to O^T
// by hand, where its weight (its row of P^T, just written) is not 0.
template <typename T, typename L>
__device__ __forceinline__ void guard(const Lane& x, uint8_t* gb, uint8_t* vslot, const uint8_t* pbuf, int parity,
                                      int jn, int n, int words, uint32_t oc, bool fresh) {
  volatile uint32_t* force = reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 32);
  volatile uint32_t* bw =
      reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 64) + parity * 8 + 4 * x.t;
  const int bar = 2 + x.t;
  uint8_t* vrow = vslot + (x.r >> 3) * L::GRP + (x.r & 7) * 128;
  auto clear = [&]() {  // (in the order that the lanes' banks differ)
#pragma unroll 4
    for (int ch = 0; ch < 8 * L::SPANS; ++ch)
      *reinterpret_cast<uint4*>(vrow + (ch >> 3) * 1024 + ((ch ^ x.r) & 7) * 16) = make_uint4(0, 0, 0, 0);
  };
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
  named_bar(bar, 128);
  if (!(bw[0] | bw[1] | bw[2] | bw[3])) return;
  const bool first = fresh;
#pragma unroll 1
  for (int key = 0; key < kKeys; ++key) {
    if (!((bw[key >> 5] >> (key & 31)) & 1u)) continue;
    const int d = x.r & (L::D - 1);
    const uint16_t raw = *reinterpret_cast<const uint16_t*>(vslot + (key >> 3) * L::GRP + (key & 7) * 128 +
                                                            (d >> 6) * 1024 + ((((d & 63) >> 3) ^ (key & 7)) << 4) +
                                                            (d & 7) * 2);
    const float v = dev::unpack2<T>(raw).x;
#pragma unroll 1
    for (int j = 0; j < 32 * words; j += 8) {
      uint32_t u[8];
      tmem_ld8(oc + j, u);
      auto weights = [&](int chunk) {
        return *reinterpret_cast<const uint4*>(pbuf + (key >> 3) * 1024 + (key & 7) * 128 +
                                               ((chunk ^ (key & 7)) << 4));
      };
      const uint4 q = weights(j >> 3), q2 = L::SPLIT ? weights(4 + (j >> 3)) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w}, w2[4] = {q2.x, q2.y, q2.z, q2.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 a = dev::unpack2<T>(w[e >> 1]), b = dev::unpack2<T>(w2[e >> 1]);
        const float pj = e & 1 ? a.y + b.y : a.x + b.x;
        const float o0 = fresh ? 0.f : __uint_as_float(u[e]);
        u[e] = __float_as_uint(pj == 0.f ? o0 : o0 + pj * v);
      }
      tmem_st8(oc + j, u);
      if (L::SPLIT && fresh) {
        const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        tmem_st8(oc + 32 + j, none);
      }
    }
    tcg::wait_st();
    fresh = false;
  }
  if (first && x.r == 0) force[x.t] = 1;  // the product adds to O^T
  named_bar(bar, 128);                    // every reader is done with the rows
  if ((bw[x.w4] >> x.lane) & 1u) clear();
  dev::fence_proxy_async_smem();
  named_bar(bar, 128);
}

// The rows of a piece out, by the warpgroup that joins: O^T of both tiles times
// the rows' weights, a warp 32 dims of a row at a time.
template <typename T, typename L>
__device__ __forceinline__ void write_rows(const TreeArgs& a, const Lane& x, const Piece& p, const float2* pubs,
                                           uint32_t oa, bool exists) {
  constexpr int D = L::D;
  const bool direct = p.slot < 0, narrow = direct && !a.out_f32;
  float* wts = x.scratch + 512;  // [2 accumulators][64]
  int* place = reinterpret_cast<int*>(x.scratch + 640);
  float* to32 = (direct ? static_cast<float*>(a.out) : a.part_o) + x.r;
  T* to16 = static_cast<T*>(a.out) + x.r;
  if (x.r < 64) {
    const float2 c0 = pubs[x.r], c1 = pubs[64 + x.r];
    const float m = fmaxf(c0.x, c1.x), mz = m == -INFINITY ? 0.f : m;
    const float w0 = dev::ex2(c0.x - mz), w1 = dev::ex2(c1.x - mz);
    const float sum = w0 * c0.y + w1 * c1.y;
    const float inv = direct && m != -INFINITY ? 1.f / sum : 1.f;
    wts[x.r] = w0 * inv;
    wts[64 + x.r] = w1 * inv;
    // where the row goes, in rows of out or of the partials
    const int h = x.r & ((1 << a.gl) - 1);
    place[x.r] = !exists ? -1 : direct ? (p.qs + (x.r >> a.gl)) * a.Hq + p.g * a.G + h : p.slot * a.slot_rows + x.r;
    if (!direct && exists) {
      a.part_m[place[x.r]] = m;
      a.part_l[place[x.r]] = sum;
    }
  }
  named_bar(2 + x.t, 128);
  if (D == 64 && x.w4 >= 2) return;  // lanes 64 .. 127 repeat the dims
#pragma unroll 1
  for (int j0 = 0; j0 < p.rows; j0 += 8) {
    uint32_t u[8], v[8];
    tmem_ld8(oa + j0, u);
    tmem_ld8(oa + 64 + j0, v);
    uint32_t u2[8], v2[8];
    if constexpr (L::SPLIT) {
      tmem_ld8(oa + 32 + j0, u2);
      tmem_ld8(oa + 96 + j0, v2);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float w0 = wts[j0 + e], w1 = wts[64 + j0 + e];
      if constexpr (L::SPLIT) {
        u[e] = __float_as_uint(__uint_as_float(u[e]) + __uint_as_float(u2[e]));
        v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(v2[e]));
      }
      float o = w0 == 0.f ? 0.f : __uint_as_float(u[e]) * w0;
      if (w1 != 0.f) o = fmaf(__uint_as_float(v[e]), w1, o);
      const int at = place[j0 + e];
      if (at < 0) continue;
      if (narrow)
        to16[static_cast<size_t>(at) * D] = static_cast<T>(o);
      else
        to32[static_cast<size_t>(at) * D] = o;
    }
  }
  __syncwarp();
}

template <typename KT, typename T, int D>
__global__ void __launch_bounds__(Lay<KT, T, D, false>::THREADS, 1)
    tree_keys(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TreeArgs a) {
  using namespace tcg;
  using L = Lay<KT, T, D, false>;
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
    multiply<T, L>(a, gb, sy, static_cast<uint32_t>(uniform(static_cast<int>(tmem))));
  } else if (wid == 2) {
    fewer_registers<L>();
    if constexpr (L::PRODUCERS == 2) produce<KT, L>(a, &tmK, &tmV, &tmQ, gb, sy, 1);
  } else if (wid == 3) {
    fewer_registers<L>();
    plan<L>(a, gb, sy);
  } else if (wid < 12) {
    // ---- softmax warpgroups: thread r owns key r of a chunk -----------------------------
    more_registers<L>();
    Lane x;
    x.t = (wid - 4) >> 2;
    x.w4 = wid & 3;
    x.lane = lane;
    x.r = 32 * x.w4 + lane;
    x.tl = tmem + (static_cast<uint32_t>(32 * x.w4) << 16);
    uint8_t* pbuf = gb + L::P0 + x.t * 16384;
    x.scratch = reinterpret_cast<float*>(pbuf);
    const int t = x.t, r = x.r, bar = 2 + t;
    float2* pubs = reinterpret_cast<float2*>(gb + L::PUB);
    uint8_t* prow = pbuf + (r >> 3) * 1024 + (r & 7) * 128;  // the key's row of P^T, swizzled by r & 7
    const float sl2 = a.scale_log2;
    bool ok = true;
    int n = 0;  // chunks of this tile so far
    Cursor<L> k;
    k.i = k.it0 = k.ph = 0;
#pragma unroll 1
    for (;; k.close()) {
      k.open(sy, gb, ok);
      // The barriers inside a piece have no limit, so where one warp has given up a
      // wait the whole warpgroup leaves, here.  (And every warp has read the sums of l
      // that the piece before left in the scratch.)
      ok = !bar_or(bar, 128, !ok);
      if (!ok || !__all_sync(FULL, k.live)) break;
      const Piece& p = k.p;
      const int words = !L::SPLIT && p.rows > 32 ? 2 : 1, pp = k.i & 1, shift = p.L - p.n;
      const uint32_t oc = x.tl + kColO + 128 * pp + 64 * t;
      const bool exists = r < p.rows && (r & ((1 << a.gl) - 1)) < a.G;  // row r (r < 64)
      bool seen = !exists, unset = true;  // row r has a reference; some row may have none
      float ref = 0.f;
      float2 l[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) l[j] = make_float2(0.f, 0.f);
      const int c_first = (t ^ k.ph) & 1;
      const bool any = c_first < k.nc;
#pragma unroll 1
      for (int c = c_first; c < k.nc; c += 2, ++n) {
        const int key0 = (p.c0 + c) * kKeys, jn = key0 + r - shift;  // node that key r is
        const bool masked = key0 + kKeys > shift;
        if (ok) ok = wait_warp(sy.sfull(t), n & 1);
        fence_after();
        float ks = sl2, vsc = 1.f, lv = 0.f;  // the key's scales, log2 of V's
        if constexpr (Q8) {
          const float* scales = reinterpret_cast<const float*>(gb + L::SCALES + (((k.it0 >> 1) + c) & 7) * 1024);
          if (key0 + r < p.L) {  // (stale past the end)
            ks = sl2 * scales[r];
            vsc = scales[128 + r];
            lv = log2_scale(vsc);
          }
        }
        uint2 vis = make_uint2(FULL, FULL);  // the rows that see the key
        if (masked) {
          if (ok) ok = wait_warp(sy.mfull(pp), (k.i >> 1) & 1);
          vis = visible<L>(a, gb, p, k.i, jn);
          __syncwarp();
        }
        const uint32_t sc = x.tl + kColS + 64 * t;
        uint32_t pk[32];  // weights, 16-bit pairs of rows
        bool moved = unset;
        for (;;) {
          if (moved) {
            if (ok && n > 0) ok = wait_warp(sy.pdone(t), (n - 1) & 1);  // (P^T free, O^T at rest)
            fence_after();
            const int what = settle<L>(x, sc, ks, lv, vis, words, oc, exists, seen, ref);
            unset = what & 2;
            if (what & 1) {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float2 al = *reinterpret_cast<const float2*>(x.scratch + 320 + 2 * j);
                if (j < 16 || words == 2) l[j] = make_float2(l[j].x * al.x, l[j].y * al.y);
              }
              named_bar(bar, 128);  // the scratch is read before P^T takes its place
            }
          }
          float top = -INFINITY;
          auto put = [&](int i, float2 w) {
            pk[i] = dev::pack2<T>(w.x, w.y);
            if constexpr (L::SPLIT) pk[(i + 16) & 31] = low_half(w, pk[i]);
          };
          // 16 rows.  16-bit caches: exponents, their maximum, weights in one pass.
          // 1-byte caches: the maximum first, so that l can sum the weights as they
          // are and only their product with V's scale, the key's, is rounded.
          auto part = [&](auto q_c, auto pass_c) {
            constexpr int Q = decltype(q_c)::value, PASS = decltype(pass_c)::value;
            uint32_t u[16], v[16];
            tmem_ld16x2(sc + 16 * Q, x.tl + kColR + 64 * t + 16 * Q, u, v);
            float2 e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              e[j] = fma2(make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])), make_float2(ks, ks),
                          make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])));
            if (masked) {  // whatever the key's score and scale are
              const uint32_t m = (Q & 2 ? vis.y : vis.x) >> (16 * (Q & 1));
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                e[j].x = (m >> (2 * j)) & 1u ? e[j].x : -INFINITY;
                e[j].y = (m >> (2 * j + 1)) & 1u ? e[j].y : -INFINITY;
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if constexpr (!Q8 || PASS == 0) top = max3(top, e[j].x, e[j].y);
              if constexpr (!Q8) {
                put(8 * Q + j, make_float2(dev::ex2(e[j].x), dev::ex2(e[j].y)));
              } else if constexpr (PASS == 1) {
                const float2 w = make_float2(dev::ex2(e[j].x), dev::ex2(e[j].y));
                l[8 * Q + j] = add2(l[8 * Q + j], w);
                const float2 y = mul2(w, make_float2(vsc, vsc));
                // (a weight of 0 must not meet a NaN scale)
                put(8 * Q + j, make_float2(w.x == 0.f ? 0.f : y.x, w.y == 0.f ? 0.f : y.y));
              }
            }
          };
          auto parts = [&](auto pass_c) {
            part(std::integral_constant<int, 0>{}, pass_c);
            part(std::integral_constant<int, 1>{}, pass_c);
            if (words == 2) {
              part(std::integral_constant<int, 2>{}, pass_c);
              part(std::integral_constant<int, 3>{}, pass_c);
            }
          };
          if (!Q8 || !moved) parts(std::integral_constant<int, 0>{});
          if (!moved && bar_or(bar, 128, top > L::MOVE - lv)) {
            moved = true;
            continue;
          }
          if constexpr (Q8) parts(std::integral_constant<int, 1>{});
          break;
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.sfree(t));  // the scores are read
        if constexpr (!Q8) {  // l sums the rounded weights
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            add16x2<T>(l[j], pk[j]);
            if constexpr (L::SPLIT) add16x2<T>(l[j], pk[16 + j]);
          }
          if (words == 2) {
#pragma unroll
            for (int j = 16; j < 32; ++j) add16x2<T>(l[j], pk[j]);
          }
        }
        if (ok && n > 0) ok = wait_warp(sy.pdone(t), (n - 1) & 1);  // P^T's buffer is free
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(prow + ((j ^ (r & 7)) << 4)) =
              make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        if (L::SPLIT || words == 2) {
#pragma unroll
          for (int j = 4; j < 8; ++j)
            *reinterpret_cast<uint4*>(prow + ((j ^ (r & 7)) << 4)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        }
        if (masked) {
          const int vi = k.it0 + 2 * c + 1, vs = vi % NS;
          if (ok) ok = __all_sync(FULL, wait_issued(sy.issued(), vi)) && wait_warp(sy.ready(vs), (vi / NS) & 1);
          fence_after();
          guard<T, L>(x, gb, gb + L::RING + vs * L::SLOT, pbuf, (p.c0 + c) & 1, jn, p.n, words, oc,
                      c == c_first);
        }
        dev::fence_proxy_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.pfull(t));
      }
      // ---- the piece's end --------------------------------------------------------------
      if (p.last) dev::grid_launch_dependents();
      if (ok && any) ok = wait_warp(sy.pdone(t), (n - 1) & 1);  // O^T final, P^T's buffer free
      fence_after();
      if (any) {  // l over the 128 keys' lanes
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (w < words) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = j & 1 ? l[16 * w + (j >> 1)].y : l[16 * w + (j >> 1)].x;
            x.scratch[64 * x.w4 + 32 * w + lane] = warp_sums(v, lane);
          }
        }
      }
      // both warpgroups are done with what the piece before published
      if (ok && k.i >= 1) ok = wait_warp(sy.ofree(pp ^ 1), ((k.i - 1) >> 1) & 1);
      named_bar(bar, 128);
      if (r < 64) {
        const bool have = any && r < 32 * words;
        const float sum =
            have ? (x.scratch[r] + x.scratch[64 + r]) + (x.scratch[128 + r] + x.scratch[192 + r]) : 0.f;
        pubs[64 * t + r] = make_float2(have && exists && seen ? ref : sum != sum ? 0.f : -INFINITY, sum);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.pub(t));
      // the warpgroup with the last chunk joins both accumulators
      if (((k.ph + k.nc - 1) & 1) == t) {
        if (ok) ok = wait_warp(sy.pub(t ^ 1), k.i & 1);  // (after that tile's last product)
        named_bar(bar, 128);
        fence_after();
        write_rows<T, L>(a, x, p, pubs, x.tl + kColO + 128 * pp, exists);
      }
      if (ok) ok = wait_warp(sy.mfull(pp), (k.i >> 1) & 1);  // (every phase is seen in order)
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
