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
// (node, head of the group), the group padded to a power of two; they all read
// the same K/V, so an item is up to 128 of them, and streams the context in
// chunks of 128 keys (8 blocks).  One unit of work is one chunk of one item (an item's start
// and end count as kItem more); the
// launch has one persistent CTA per SM, and CTA k takes units [k u, (k + 1) u)
// of the batch in order, u = ceil(units / CTAs): every CTA streams the same
// number of chunks whatever the lengths.  The lengths stay on the device: each
// CTA counts the units itself from context_lens and q_start.  An item that
// spans CTAs leaves partial rows (o, m, l), at most two sets per CTA, merged by
// tree_merge with log-sum-exp weights.
//
// The products are transposed: S^T = K Q^T (M = the chunk's 128 keys, N = rows)
// and O^T += V^T P^T (M = dims, N = rows), so the tensor cores and the
// exponentials do work in proportion to the rows, 16 at a time, and a whole
// warpgroup is busy however few they are.  Thread r of a warpgroup owns key r
// of the chunk: a key's scales are its own registers, P^T leaves through shared
// memory (one 128-byte row per key), and an output column needs no exchange
// between lanes.  Inside a CTA:
//   warp 0       producer: Q rows and the K and V chunks into a ring of slots
//                by TMA (128-byte swizzle, one box per block);
//   warp 1       issues the MMAs from one thread, S^T ahead of O^T;
//   warp 3       planner: the CTA's pieces of items, published a few ahead, and
//                their mask words;
//   warps 4-7,   two softmax warpgroups.  Up to 64 rows: they take alternate
//   8-11         chunks, each with its own accumulator and references, and the
//                one that had the last chunk joins the two while the other
//                starts on the next piece.  65 .. 128 rows: each takes half of
//                the rows and every chunk, and one MMA serves both;
//   warps 12-15  1-byte caches only: convert a landed slot's codes in place to
//                the 16-bit layouts the MMAs read.
// A row's reference is the maximum of the first chunk in which it sees a key,
// kept in tensor memory beside the scores (read as cheaply as they are, where
// shared memory, which feeds the MMAs, has no bandwidth to spare); it moves,
// O^T and l with it, only when an exponent outgrows it by 2^8.  P is rounded to
// the 16 bits of V's type, which the product shares, and normalised by the sum
// of the rounded weights, so a row that rests on one key returns that key's
// value; the rounding (half a step, independent over keys) adds as much as the
// rounding of a 16-bit output.  References, l and O are float32.
//
// What bounds it: HBM while the rows per kv head stay below ~290 (4 D flops
// per key and row against 4 D bytes per key at 16 bits), the exponentials and
// the MMAs above that.  The hot loops are kept short and the rest out of their
// way: the instruction cache, not the issue rate, limits a kernel of this many
// roles.
//
// Values in masked places: a masked exponent is replaced; V rows past the
// context's end are zeroed in shared memory, and a node's V row that holds an
// infinity or NaN (a slot nothing was ever written to) is zeroed too and added
// to O^T by hand for the rows that do see it, so it reaches no other row.
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
constexpr int kKeys = 128;  // keys per chunk
constexpr int kBlk = kKeys / 16;
constexpr int kRows = 128;  // rows of an item
constexpr float kMove = 8.f;  // log2 of how far an exponent may outgrow its reference
constexpr uint32_t kTmemCols = 512;
// tensor memory columns: S^T [tile] x 64, minus the references [tile] x 64, O^T
// [piece parity][tile] x 64.  Pieces of more than 64 rows keep O^T in the first
// of its two places and use the other as a second S^T, for odd chunks.
constexpr uint32_t kColS = 0, kColR = 128, kColO = 256, kColS2 = 384;
constexpr uint64_t kLimit = 2000000000ull;

struct TreeArgs {
  const void* q;
  const int32_t* q_start;
  const uint64_t* mask;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* part_o;    // [2 * CTAs][rows of an item][D], then m and l [2 * CTAs][rows]
  float* part_m;
  float* part_l;
  int4* split;      // [CTAs][2]: the item that CTA k leaves unfinished (Split), parts 0: none
  int32_t B, T, Hq, Hkv, G, max_blocks, num_blocks, max_context_len, max_q_len, words;
  int32_t gl;         // log2 of the rows of a node: its heads, up to a power of two
  int32_t min_units;  // units a CTA takes at least
  int32_t n_cta;
  float scale_log2;   // |scale| log2 e
  uint32_t negate;    // 1 when scale < 0: the products negate Q
  int32_t out_f32;
};

using tcg::mbar_arrive;

// ---- the batch's work ------------------------------------------------------
struct Seq {
  int qs, n, L;   // first query row, nodes, context length
  int tiles, nch;  // items per kv head, chunks
};
// Sequence b's view, clamped to what the launch can serve; violations are
// flagged by the one thread that reports.
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b, bool report) {
  Seq s;
  s.qs = a.q_start[b];
  s.n = a.q_start[b + 1] - s.qs;
  s.L = a.context_lens[b];
  uint32_t err = 0;
  if (s.qs < 0 || s.n < 0 || s.n > a.max_q_len || s.qs > a.T - s.n) {
    err |= PA_DEVERR_QUERY_RANGE;
    s.qs = s.n = 0;
  }
  const int cap = min(a.max_context_len, a.max_blocks * 16);
  if (s.L < 0 || s.L > cap || s.n > s.L) err |= PA_DEVERR_CONTEXT_LEN;
  s.L = max(0, min(s.L, cap));
  if (report && err) atomicOr(&g_tree_err, err);
  s.tiles = ((s.n << a.gl) + kRows - 1) / kRows;
  s.nch = max(1, (s.L + kKeys - 1) / kKeys);  // a sequence without keys still owns its zero rows
  return s;
}
// An item's cost in units: its chunks, and kItem for its start and end.
constexpr int kItem = 3;
__device__ __forceinline__ int units_of(const TreeArgs& a, const Seq& s) { return s.tiles * a.Hkv * (s.nch + kItem); }
__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL, v, off);
  return v;
}

// One item's run of chunks [c0, c1) for a CTA.
struct __align__(16) Piece {
  int qs, n, L, row0;    // the sequence; the item's first row
  int g, rows, c0, c1;   // kv head; the item's rows; chunks
  int b, slot, live, last;  // slot: its set of partial rows (-1: the whole item); live 0: no more pieces
};

// ---- shared memory -----------------------------------------------------------
template <typename KT, int D_>
struct Lay {
  static constexpr bool Q8 = sizeof(KT) == 1;
  static constexpr int D = D_;
  static constexpr int SPANS = D / 64;               // 128-byte spans of a 16-bit row
  // Q of a piece [span][rows][128 B]: 128 rows, or in either half of the place 64
  static constexpr int QTILE = kRows * D * 2;
  static constexpr int SLOT = kKeys * D * 2;         // one K or V chunk, 16-bit
  static constexpr int GRP = 1024 * SPANS;           // 8 keys of a slot: [span][8][128 B]
  static constexpr int P0 = QTILE;                   // P^T [tile][128 keys][128 B]
  static constexpr int RING = P0 + 2 * 16384;
  static constexpr int NS = D == 64 ? 10 : Q8 ? 4 : 5;
  static constexpr int SCALES = RING + NS * SLOT;    // 1-byte codes: [8 chunks][K 128, V 128] float
  static constexpr int BAR = SCALES + (Q8 ? 8 * 1024 : 0);
  static constexpr int NBAR = 3 * NS + 28;
  static constexpr int MISC = (BAR + NBAR * 8 + 15) & ~15;  // tensor memory, items issued, force; at 64: bad keys
  static constexpr int PIECE = MISC + 128;           // Piece [4]
  static constexpr int PUB = PIECE + 4 * 48;         // float2 [2 tiles][64]
  static constexpr int MASK = PUB + 1024;            // uint64 [2 pieces][64 nodes]
  static constexpr int BYTES = MASK + 1024;
  static constexpr int THREADS = Q8 ? 512 : 384;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// ---- waits -------------------------------------------------------------------
// Bounded: each try sleeps up to a microsecond.  (Inlined and without a clock,
// to keep the code small; a function call would tie every role to one register
// count.)
constexpr int kTries = 2000000;
__device__ __forceinline__ bool wait_thread(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < kTries; ++i)
    if (dev::mbar_try_wait_sleep(bar, parity, 1000u)) return true;
  return false;
}
// A bounded wait whose outcome is the same in every lane, so the
// warp-collective instructions that follow stay converged.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
  return __all_sync(FULL, wait_thread(bar, parity));
}
// Wait until the producer has issued ring item i.  A slot's full barrier tells
// one phase from the next by parity only; with the item issued, the slot's
// phase before it is over.
__device__ __forceinline__ bool wait_issued(uint32_t count, int item) {
#pragma unroll 1
  for (int i = 0; i < kTries; ++i) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(count) : "memory");
    if (v > item) return true;
    __nanosleep(200);
  }
  return false;
}
__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_tree_err, bits); }

__device__ __forceinline__ void named_bar(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Barrier that returns whether any thread's x holds.
__device__ __forceinline__ bool bar_or(int id, int threads, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Registers move from the single-thread roles (and the converters) to the
// softmax warpgroups: 384 x 168 = 256 x 200 + 128 x 104, and with converters
// 512 x 128 = 256 x 176 + 256 x 80.  Every warp calls its one.  (A spilled
// register goes to L2 here: shared memory leaves the L1 no room.)
template <bool Q8>
__device__ __forceinline__ void fewer_registers() {
  if constexpr (Q8)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
}
template <bool Q8>
__device__ __forceinline__ void more_registers() {
  if constexpr (Q8)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
}

// ---- tensor memory -----------------------------------------------------------
// Loads that have arrived when they return (load and wait in one statement, so
// no use of the registers can be scheduled between them).
#define PA_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
// 16 columns at two places under one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, uint32_t (&r)[16], uint32_t (&s)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : PA_R8(r, 0), PA_R8(r, 8), PA_R8(s, 0), PA_R8(s, 8)
      : "r"(ta), "r"(tb)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : PA_R8(r, 0)
      : "r"(taddr)
      : "memory");
}
#undef PA_R8
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// ---- arithmetic --------------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b));
  return d;
}
// l += a pair of 16-bit weights, without unpacking it.
template <typename T>
__device__ __forceinline__ void add16x2(float2& l, uint32_t pair) {
  if constexpr (std::is_same<T, __half>::value)
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.f16 %0, x, %0;\n\tadd.rn.f32.f16 %1, y, %1;\n\t}"
        : "+f"(l.x), "+f"(l.y)
        : "r"(pair));
  else
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.bf16 %0, x, %0;\n\tadd.rn.f32.bf16 %1, y, %1;\n\t}"
        : "+f"(l.x), "+f"(l.y)
        : "r"(pair));
}
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
// Sum over the warp's lanes of 32 values a lane: lane j gets value j's.
__device__ __forceinline__ float warp_sums(float (&v)[32], int lane) {
#pragma unroll
  for (int h = 16; h > 0; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int j = 0; j < h; ++j) {
      const float give = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
      v[j] = keep + __shfl_xor_sync(FULL, give, h);
    }
  }
  return v[0];
}
template <typename T>
__device__ __forceinline__ bool bad16(uint32_t w) {  // a pair holds an infinity or NaN
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  return (w & E) == E || ((w >> 16) & E) == E;
}

// One lane of a converged warp, the same every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
  return x != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(FULL, x, 0); }

// ---- roles -------------------------------------------------------------------
// The CTA's barriers and words in shared memory.
template <typename L>
struct Sync {
  uint32_t base;
  __device__ __forceinline__ uint32_t at(int i) const { return base + L::BAR + 8 * i; }
  __device__ __forceinline__ uint32_t full(int s) const { return at(s); }                // slot s landed
  __device__ __forceinline__ uint32_t conv(int s) const { return at(L::NS + s); }        // its codes converted
  __device__ __forceinline__ uint32_t empty(int s) const { return at(2 * L::NS + s); }   // its last product ended
  __device__ __forceinline__ uint32_t ready(int s) const { return L::Q8 ? conv(s) : full(s); }
  __device__ __forceinline__ uint32_t ext(int i) const { return at(3 * L::NS + i); }
  __device__ __forceinline__ uint32_t sfull(int t, int b) const { return ext(2 * t + b); }      // S^T of tile t, buffer b
  __device__ __forceinline__ uint32_t sfree(int t, int b) const { return ext(4 + 2 * t + b); }  // and read
  __device__ __forceinline__ uint32_t pfull(int t) const { return ext(8 + t); }     // P^T in shared memory
  __device__ __forceinline__ uint32_t pdone(int t) const { return ext(10 + t); }    // O^T += V^T P^T ended
  __device__ __forceinline__ uint32_t qfull(int i) const { return ext(12 + i); }    // Q of a piece landed
  __device__ __forceinline__ uint32_t qfree(int i) const { return ext(14 + i); }    // its last S^T ended
  __device__ __forceinline__ uint32_t ofree(int i) const { return ext(16 + i); }    // piece parity i: both warpgroups are done
  __device__ __forceinline__ uint32_t pub(int t) const { return ext(18 + t); }      // tile t's l and references of the piece
  __device__ __forceinline__ uint32_t mfull(int i) const { return ext(20 + i); }    // mask words of a piece
  __device__ __forceinline__ uint32_t pieces(int i) const { return ext(22 + i); }   // piece i % 4 published
  __device__ __forceinline__ uint32_t mdone() const { return ext(26); }             // after a timeout: products have ended
  __device__ __forceinline__ uint32_t issued() const { return base + L::MISC + 16; }
  // piece i of the CTA; false after the last (or a timeout)
  __device__ __forceinline__ bool piece(const uint8_t* gb, int i, Piece& p, bool& ok) const {
    if (ok) ok = wait_thread(pieces(i & 3), (i >> 2) & 1);
    const int4* s = reinterpret_cast<const int4*>(gb + L::PIECE + (i & 3) * sizeof(Piece));
    int4* d = reinterpret_cast<int4*>(&p);
    d[0] = s[0];
    d[1] = s[1];
    d[2] = s[2];
    return ok && p.live;
  }
};

// The planner warp: this CTA's pieces, and the mask words of trees of at most
// 64 nodes.
template <typename L>
__device__ __forceinline__ void plan(const TreeArgs& a, uint8_t* gb, Sync<L> sy) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const bool report = blockIdx.x == 0;
  // units of the batch, 32 sequences at a time; then the first of this CTA's
  int total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32) total += b0 + lane < a.B ? units_of(a, seq_of(a, b0 + lane, report)) : 0;
  total = warp_sum(total);
  const int upc = max((total + a.n_cta - 1) / a.n_cta, a.min_units);
  const int start = min(static_cast<int>(blockIdx.x) * upc, total), end = min(start + upc, total);
  int b = 0, ub = 0;  // the sequence of unit `u`, and the units before it
#pragma unroll 1
  for (int b0 = 0; start < end; b0 += 32) {
    const int w = b0 + lane < a.B ? units_of(a, seq_of(a, b0 + lane, false)) : 0;
    int inc = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(FULL, inc, off);
      if (lane >= off) inc += y;
    }
    const unsigned over = __ballot_sync(FULL, ub + inc > start);
    if (over) {
      const int f = __ffs(over) - 1;
      b = b0 + f;
      ub += __shfl_sync(FULL, inc - w, f);
      break;
    }
    ub += __shfl_sync(FULL, inc, 31);
  }
  Piece* ring = reinterpret_cast<Piece*>(gb + L::PIECE);
  uint64_t* words = reinterpret_cast<uint64_t*>(gb + L::MASK);
  int u = start, pieces = INT32_MAX;
  bool ok = true;
  int4 sp0 = make_int4(0, 0, 0, 0), sp1 = sp0;
  // Step i: piece i is published and piece i - 2's mask words are fetched, once
  // piece i - 4 is over (their places are free then).
#pragma unroll 1
  for (int i = 0; i < pieces || i - 2 < pieces; ++i) {
    if (ok && i >= 4) ok = wait_warp(sy.ofree(i & 1), ((i - 4) >> 1) & 1);
    if (i <= pieces && pieces == INT32_MAX) {
      Piece p;
      p.live = 0;
#pragma unroll 1
      while (u < end && !p.live) {
        Seq s = seq_of(a, b, false);
#pragma unroll 1
        while (u >= ub + units_of(a, s)) {
          ub += units_of(a, s);
          s = seq_of(a, ++b, false);
        }
        const int cost = s.nch + kItem, at = u - ub, item = at / cost, off = at - item * cost;
        const int stop = min(cost, off + end - u);  // of the item, for this CTA
        p.c0 = max(0, off - kItem);
        p.c1 = stop - kItem;
        u += stop - off;
        if (p.c1 <= p.c0) continue;  // the range ends before the item's first chunk
        p.live = 1;
        p.b = b;
        p.qs = s.qs;
        p.n = s.n;
        p.L = s.L;
        p.g = item / s.tiles;
        p.row0 = (item - p.g * s.tiles) * kRows;
        p.rows = min(kRows, (s.n << a.gl) - p.row0);
        p.slot = p.c0 == 0 && p.c1 == s.nch ? -1 : 2 * static_cast<int>(blockIdx.x) + (i == 0 ? 0 : 1);
        if (p.c0 == 0 && p.c1 < s.nch) {  // the item goes on in the next CTAs: what tree_merge needs
          sp0 = make_int4((ub + (item + 1) * cost - 1) / upc - static_cast<int>(blockIdx.x) + 1, p.slot, s.qs, p.row0);
          sp1 = make_int4(p.g, p.rows, 0, 0);
        }
      }
      p.last = u >= end;  // (or only an item's start is left)
      if (!p.live) pieces = i;
      if (lane == 0) {
        ring[i & 3] = p;
        mbar_arrive(sy.pieces(i & 3));
      }
      __syncwarp();
    }
    const int m = i - 2;
    if (m >= 0 && m < pieces) {
      const Piece& x = ring[m & 3];
      if (x.n <= 64 && x.c1 * kKeys > x.L - x.n)
        for (int k = lane; k < x.n; k += 32) words[(m & 1) * 64 + k] = a.mask[static_cast<size_t>(x.qs + k) * a.words];
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.mfull(m & 1));
    }
  }
  if (lane == 0) {
    a.split[2 * blockIdx.x] = sp0;
    a.split[2 * blockIdx.x + 1] = sp1;
    if (!ok) flag(PA_DEVERR_TIMEOUT);
  }
}

// The producer warp: each piece's Q rows, and its K and V chunks into the ring
// (lane i < 8 issues block i).
template <typename KT, typename L>
__device__ __forceinline__ void produce(const TreeArgs& a, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                     const CUtensorMap* tmQ, uint8_t* gb, Sync<L> sy) {
  constexpr int NS = L::NS, D = L::D;
  const int lane = static_cast<int>(threadIdx.x & 31);
  bool ok = true;
  int it = 0, q_issued = 0, q_free = 0;  // ring items, Qs of pieces, pieces done with theirs
  bool before_pair = false;
  // Loads that wait behind a full ring take microseconds, so the block ids of
  // the next 32 blocks, and the next piece's first, are fetched well ahead.
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
  // Q of piece i: boxes of br rows (whole nodes), a lane per (box, span).  Its
  // place is free once `need` pieces have ended their last S^T.
  auto load_q = [&](const Piece& x, int i, int need) {
#pragma unroll 1
    for (; q_free < need; ++q_free)
      if (ok) ok = wait_warp(sy.qfree(q_free & 1), (q_free >> 1) & 1);
    if (!ok) return;
    ++q_issued;
    const bool pair = x.rows > 64;
    const int br = max(32, 1 << a.gl);
    const int sp = lane % L::SPANS, y = lane / L::SPANS * br;
    const bool mine = y < x.rows;
    const uint32_t n = static_cast<uint32_t>(__popc(__ballot_sync(FULL, mine)));
    if (lane == 0) dev::mbar_arrive_expect_tx(sy.qfull(i & 1), n * br * 128);
    __syncwarp();
    if (mine)
      dev::tma_load_3d(sy.base + (pair ? sp * 16384 : (i & 1) * (L::QTILE / 2) + sp * 8192) + y * 128, tmQ,
                       sy.qfull(i & 1), sp * 64, x.g * a.G, x.qs + ((x.row0 + y) >> a.gl));
    __syncwarp();
  };
  Piece p, pn;
  bool more = sy.piece(gb, 0, p, ok);
  int ids_next = more ? fetch(p, p.c0 * kBlk) : 0;
#pragma unroll 1
  for (int i = 1; more; ++i) {
    const bool more_n = sy.piece(gb, i, pn, ok);
    p.g = uniform(p.g);
    p.c0 = uniform(p.c0);
    p.c1 = uniform(p.c1);
    const int nblk = uniform((p.L + 15) / 16), ids_n = more_n ? fetch(pn, pn.c0 * kBlk) : 0;
    int ids = 0;
    // 64 rows in alternate halves; 128 rows, and what follows them, want the
    // whole place, which frees late: the first chunk then goes ahead
    const bool late = p.rows > 64 || before_pair;
    before_pair = p.rows > 64;
    if (!late) load_q(p, i - 1, i - 2);
#pragma unroll 1
    for (int c = p.c0; c < p.c1; ++c) {
      const int k4 = (c - p.c0) & 3;
      if (k4 == 0) {
        ids = ids_next;
        ids_next = c + 4 < p.c1 ? fetch(p, (c + 4) * kBlk) : ids_n;
      }
      int blk[kBlk];  // the chunk's block ids
#pragma unroll
      for (int k = 0; k < kBlk; ++k) blk[k] = __shfl_sync(FULL, ids, k4 * kBlk + k);
      const int live = max(0, min(kBlk, nblk - c * kBlk));  // blocks of this chunk that exist
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        const int s = it % NS;
        if (ok && it >= NS) ok = wait_warp(sy.empty(s), (it / NS - 1) & 1);
        if (!ok) break;
        dev::fence_proxy_async_smem();  // the softmax's and converters' accesses precede the refill
        const uint32_t dst = sy.base + L::RING + s * L::SLOT, bar = sy.full(s);
        ++it;
        if (lane == 0) {
          // codes land in the upper half of the slot; K's with both scale rows
          const int bytes = L::Q8 ? 16 * D + (v ? 0 : 128) : 32 * D;
          dev::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live * bytes));
          asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(sy.issued()), "r"(it) : "memory");
        }
        __syncwarp();
        const CUtensorMap* m = v ? tmV : tmK;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlk; ++k) {
            if (k >= live) break;
            if constexpr (L::Q8) {
              dev::tma_load_3d(dst + L::SLOT / 2 + k * 2048, m, bar, 0, p.g * 16, blk[k]);
              if (v == 0) {
                const uint32_t sc = sy.base + L::SCALES + (((it - 1) >> 1) & 7) * 1024 + k * 64;
                dev::bulk_load(sc, a.k_scale + static_cast<size_t>(blk[k]) * 16, 64, bar);
                dev::bulk_load(sc + 512, a.v_scale + static_cast<size_t>(blk[k]) * 16, 64, bar);
              }
            } else if constexpr (D == 64) {  // [block][16][128 B]
              dev::tma_load_3d(dst + k * 2048, m, bar, 0, p.g * 16, blk[k]);
            } else {                         // [block][group of 8][span][8][128 B]
              dev::tma_load_5d(dst + k * 4096, m, bar, 0, 0, 0, 2 * p.g, blk[k]);
            }
          }
        }
        __syncwarp();
      }
      if (late && c == p.c0) load_q(p, i - 1, i - 1);
    }
    p = pn;
    more = more_n && ok;
  }
  // no copy may still be landing when the CTA exits
  for (int i = max(0, q_issued - 2); i < q_issued; ++i) wait_thread(sy.qfull(i & 1), (i >> 1) & 1);
  for (int i = max(0, it - NS); i < it; ++i) wait_thread(sy.full(i % NS), (i / NS) & 1);
  if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  __syncwarp();
}

// A walk over the chunks of all pieces, in order.
template <typename L>
struct Cursor {
  Piece p;
  int i, c, nc, it0, ph;  // piece, chunk, its chunks, ring items before it, tile of its chunk 0
  bool live, pair;        // pair: each tile half of the rows; else alternate chunks
  __device__ __forceinline__ void open(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    live = sy.piece(gb, i, p, ok);
    c = 0;
    nc = p.c1 - p.c0;
    pair = p.rows > 64;
  }
  __device__ __forceinline__ void start(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    i = it0 = ph = 0;
    open(sy, gb, ok);
  }
  __device__ __forceinline__ void close() {
    it0 += 2 * nc;
    if (!pair) ph ^= nc & 1;
    ++i;
  }
  // true: the next chunk is another piece's
  __device__ __forceinline__ bool next(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    if (++c < nc) return false;
    close();
    open(sy, gb, ok);
    return true;
  }
  __device__ __forceinline__ int tile() const { return pair ? 0 : (ph + c) & 1; }
};

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
    x.pair = x.p.rows > 64;
  };
  s.start(sy, gb, ok);
  o.start(sy, gb, ok);
  same(s);
  same(o);
  int ahead = 0, spin = 0;                 // chunks whose S^T is issued and O^T not
  int ns00 = 0, ns01 = 0, ns10 = 0, ns11 = 0;  // S^T issued per tile and buffer
  int no0 = 0, no1 = 0, pieces_over = 0;       // O^T per tile; pieces that both warpgroups are done with
  uint64_t t0 = 0;
  auto test = [&](uint32_t bar, int parity) { return uniform(dev::mbar_test(bar, parity & 1)) != 0; };
  auto landed = [&](int i) { return test(sy.ready(i % NS), i / NS); };
#pragma unroll 1
  while (o.live) {
    bool moved = false;
    if (ahead > 0) {
      const int t = o.tile(), i = o.it0 + 2 * o.c + 1;
      if (test(sy.pfull(t), t ? no1 : no0) && (!o.pair || test(sy.pfull(1), no1)) && landed(i)) {
        fence_after();
        // A = V^T (M-major), B = P^T (N-major)
        const uint32_t id = idesc<T>((o.p.rows + 15) & ~15, true) | (1u << 15);
        const uint64_t vd = sdesc(sy.base + L::RING + (i % NS) * L::SLOT, D == 128 ? 1024 : 0, L::GRP);
        const uint64_t pd = sdesc(sy.base + L::P0 + t * 16384, 16384, 1024);
        const uint32_t od = tmem + kColO + (o.pair ? 0 : 128 * (o.i & 1) + 64 * t);
        const uint32_t forced = uniform(force[t]);
        const uint32_t acc = o.c >= (o.pair ? 1 : 2) || forced ? 1u : 0u;
        if (elect_one()) {
          if (forced) force[0] = force[1] = 0;
#pragma unroll
          for (int kk = 0; kk < kBlk; ++kk)
            mma_ss(od, vd + ((kk * 2 * L::GRP) >> 4), pd + ((kk * 2048) >> 4), id, kk > 0 ? 1u : acc);
          commit(sy.pdone(t));
          if (o.pair) commit(sy.pdone(1));
          commit(sy.empty(i % NS));
        }
        __syncwarp();
        no0 += o.pair || t == 0;
        no1 += o.pair || t == 1;
        --ahead;
        if (o.next(sy, gb, ok)) same(o);
        moved = true;
      }
    }
    if (s.live && ahead < 2) {
      const int t = s.tile(), i = s.it0 + 2 * s.c, qb = s.i & 1;
      // The buffer's last scores are read.  A first chunk also waits for the
      // piece before last to be over; a pair's second buffer may hold O^T of the
      // piece before.
      const int sb = s.pair ? s.c & 1 : 0, n0 = sb ? ns01 : ns00, n1 = sb ? ns11 : ns10;
      const int over = sb && s.c == 1 ? s.i : s.c == 0 ? s.i - 1 : 0;
      if (pieces_over < over && test(sy.ofree(pieces_over & 1), pieces_over >> 1)) ++pieces_over;
      if (pieces_over >= over && (t == 1 || n0 == 0 || test(sy.sfree(0, sb), n0 - 1)) &&
          ((t == 0 && !s.pair) || n1 == 0 || test(sy.sfree(1, sb), n1 - 1)) &&
          (s.c > 0 || test(sy.qfull(qb), s.i >> 1)) && landed(i)) {
        fence_after();
        const uint32_t id = idesc<T>((s.p.rows + 15) & ~15, false) | (a.negate << 14);
        const uint64_t kd = sdesc(sy.base + L::RING + (i % NS) * L::SLOT, 16, L::GRP);
        const uint64_t qd = sdesc(sy.base + (s.pair ? 0 : qb * (L::QTILE / 2)), 16, 1024);
        const uint32_t span = (s.pair ? 16384 : 8192) >> 4;
        const uint32_t sd = tmem + (sb ? kColS2 : kColS + 64 * t);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(sd, kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                   qd + (kk >> 2) * span + (((kk & 3) * 32) >> 4), id, kk > 0 ? 1u : 0u);
          commit(sy.sfull(t, sb));
          if (s.pair) commit(sy.sfull(1, sb));
          commit(sy.empty(i % NS));
          if (s.c + 1 == s.nc) commit(sy.qfree(qb));
        }
        __syncwarp();
        if (s.pair || t == 0) ++(sb ? ns01 : ns00);
        if (s.pair || t == 1) ++(sb ? ns11 : ns10);
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

// The converter warpgroup (1-byte caches): codes of a landed slot -> 16-bit
// values, in place, in the layout the MMAs read.
template <typename KT, typename T, typename L>
__device__ __forceinline__ void convert(uint8_t* gb, Sync<L> sy) {
  constexpr int NS = L::NS;
  const int lane = static_cast<int>(threadIdx.x & 31), i0 = static_cast<int>(threadIdx.x) - 384;
  bool ok = true;
  int it = 0;
  Piece p;
#pragma unroll 1
  for (int i = 0; sy.piece(gb, i, p, ok); ++i) {
    const int n = 2 * (p.c1 - p.c0);
#pragma unroll 1
    for (int k = 0; k < n; ++k, ++it) {
      const int s = it % NS;
      if (ok) ok = wait_warp(sy.full(s), (it / NS) & 1);
      uint8_t* st = gb + L::RING + s * L::SLOT;
      uint4 w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // 16 codes: chunk c16 of row `key`
        const int x = i0 + 128 * j, key = x >> 3, c16 = x & 7;
        w[j] = *reinterpret_cast<const uint4*>(st + L::SLOT / 2 + key * 128 + ((c16 ^ (key & 7)) << 4));
      }
      named_bar(4, 128);  // every code is in registers before the slot is rewritten
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = i0 + 128 * j, key = x >> 3, c16 = x & 7, cc = 2 * (c16 & 3);
        uint32_t f[8];
        dev::code8x4_to<KT, T>(w[j].x, f[0], f[1]);
        dev::code8x4_to<KT, T>(w[j].y, f[2], f[3]);
        dev::code8x4_to<KT, T>(w[j].z, f[4], f[5]);
        dev::code8x4_to<KT, T>(w[j].w, f[6], f[7]);
        uint8_t* row = st + (key >> 3) * L::GRP + (c16 >> 2) * 1024 + (key & 7) * 128;
        *reinterpret_cast<uint4*>(row + ((cc ^ (key & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(row + (((cc + 1) ^ (key & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
      dev::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.conv(s));
    }
  }
  if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
}

// What the softmax's rare paths share with its loop.
struct Lane {
  int t, w4, lane, r;   // tile, warp of the tile, lane, key of the chunk
  uint32_t tl;          // tensor memory at the warp's lanes
  float* scratch;       // the tile's P^T buffer, between a product's end and the next P^T
};

// The rows (bits) that see the lane's key, node jn of its sequence.
template <typename L>
__device__ __forceinline__ uint2 visible(const TreeArgs& a, const uint8_t* gb, const Piece& p, int piece, int row0, int jn) {
  uint32_t vis[2] = {0u, 0u};
  const uint64_t* words = reinterpret_cast<const uint64_t*>(gb + L::MASK) + (piece & 1) * 64;
  const uint32_t each = a.gl >= 5 ? FULL : (1u << (1 << a.gl)) - 1u;
  const int per = a.gl >= 5 ? 1 : 32 >> a.gl;  // nodes of a word
  if (jn < 0) return make_uint2(FULL, FULL);
  if (jn >= p.n) return make_uint2(0u, 0u);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int n0 = (row0 + 32 * w) >> a.gl, cnt = min(per, p.n - n0);
#pragma unroll 2
    for (int i = 0; i < cnt; ++i) {
      const uint64_t m =
          p.n <= 64 ? words[n0 + i] : a.mask[static_cast<size_t>(p.qs + n0 + i) * a.words + (jn >> 6)];
      if ((m >> (jn & 63)) & 1) vis[w] |= each << (i << a.gl);
    }
  }
  return make_uint2(vis[0], vis[1]);
}

// New references from the scores in tensor memory, where a row has none yet or
// an exponent outgrew it; O^T moves with them.  alpha: what the rows' l are to
// be multiplied by, in scratch[320 ..], if the result's bit 0 is set.  Bit 1:
// some row still has no reference.
template <typename L>
__device__ __forceinline__ int settle(const Lane& x, uint32_t sc, float ks, uint2 vis, int words, uint32_t oc, bool exists, bool& seen,
                                   float& ref) {
  const int bar = 2 + x.t;
  float best0 = -INFINITY, best1 = -INFINITY;  // of rows lane, 32 + lane
#pragma unroll 1
  for (int j = 0; j < 32 * words; j += 8) {
    uint32_t u[8];
    tmem_ld8(sc + j, u);
    const uint32_t v = (j & 32 ? vis.y : vis.x) >> (j & 31);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = warp_max((v >> e) & 1u ? __uint_as_float(u[e]) * ks : -INFINITY);
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
    const float cm = fmaxf(fmaxf(x.scratch[x.r], x.scratch[64 + x.r]), fmaxf(x.scratch[128 + x.r], x.scratch[192 + x.r]));
    float alpha = 1.f;
    if (exists && (seen ? cm > ref + kMove : cm > -INFINITY)) {
      rescale = seen;
      if (seen) alpha = dev::ex2(ref - cm);
      ref = cm;
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
      uint32_t o[8];
      tmem_ld8(oc + j, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * x.scratch[320 + j + e]);
      tmem_st8(oc + j, o);
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
                                      bool pair, int jn, int n, int words, uint32_t oc, bool fresh) {
  volatile uint32_t* force = reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 32);
  volatile uint32_t* bw =
      reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 64) + parity * 8 + (pair ? 0 : 4 * x.t);
  const bool scan = !pair || x.t == 0;
  const int bar_id = pair ? 1 : 2 + x.t, bar_n = pair ? 256 : 128;
  uint8_t* vrow = vslot + (x.r >> 3) * L::GRP + (x.r & 7) * 128;
  auto clear = [&]() {
#pragma unroll 4
    for (int ch = 0; ch < 8 * L::SPANS; ++ch)
      *reinterpret_cast<uint4*>(vrow + (ch >> 3) * 1024 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
  };
  if (scan) {
    bool bad = false;
    if (jn >= n) {
      clear();
    } else if (jn >= 0) {
#pragma unroll 4
      for (int ch = 0; ch < 8 * L::SPANS; ++ch) {
        const uint4 v = *reinterpret_cast<const uint4*>(vrow + (ch >> 3) * 1024 + (ch & 7) * 16);
        bad |= bad16<T>(v.x) | bad16<T>(v.y) | bad16<T>(v.z) | bad16<T>(v.w);
      }
    }
    const uint32_t word = __ballot_sync(FULL, bad);
    if (x.lane == 0) bw[x.w4] = word;
    dev::fence_proxy_async_smem();
  }
  named_bar(bar_id, bar_n);
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
      const uint4 q = *reinterpret_cast<const uint4*>(pbuf + (key >> 3) * 1024 + (key & 7) * 128 +
                                                      (((j >> 3) ^ (key & 7)) << 4));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float pj = e & 1 ? dev::unpack2<T>(w[e >> 1]).y : dev::unpack2<T>(w[e >> 1]).x;
        const float o0 = fresh ? 0.f : __uint_as_float(u[e]);
        u[e] = __float_as_uint(pj == 0.f ? o0 : o0 + pj * v);
      }
      tmem_st8(oc + j, u);
    }
    tcg::wait_st();
    fresh = false;
  }
  if (first && x.r == 0) force[x.t] = 1;  // the product adds to O^T
  named_bar(bar_id, bar_n);               // every reader is done with the rows
  if (scan && ((bw[x.w4] >> x.lane) & 1u)) clear();
  dev::fence_proxy_async_smem();
  named_bar(bar_id, bar_n);
}

// The rows of a piece out, by the warpgroup that joins: O^T of both tiles (or
// of its own) times the rows' weights, a warp 32 dims of a row at a time.
template <typename T, typename L>
__device__ __forceinline__ void write_rows(const TreeArgs& a, const Lane& x, const Piece& p, const float2* pubs, uint32_t oa,
                                        bool both, int row0, int rows, bool exists) {
  constexpr int D = L::D;
  const bool direct = p.slot < 0, narrow = direct && !a.out_f32;
  const int base = p.row0 + row0;
  float* wts = x.scratch + 512;  // [2 accumulators][64]
  int* place = reinterpret_cast<int*>(x.scratch + 640);
  float* to32 = (direct ? static_cast<float*>(a.out) : a.part_o) + x.r;
  T* to16 = static_cast<T*>(a.out) + x.r;
  if (x.r < 64) {
    const float2 c0 = pubs[(both ? 0 : 64 * x.t) + x.r], c1 = both ? pubs[64 + x.r] : make_float2(-INFINITY, 0.f);
    const float m = fmaxf(c0.x, c1.x), mz = m == -INFINITY ? 0.f : m;
    const float w0 = dev::ex2(c0.x - mz), w1 = dev::ex2(c1.x - mz);
    const float sum = w0 * c0.y + w1 * c1.y;
    const float inv = direct && m != -INFINITY ? 1.f / sum : 1.f;
    wts[x.r] = w0 * inv;
    wts[64 + x.r] = w1 * inv;
    // where the row goes, in rows of out or of the partials
    const int row = base + x.r, h = row & ((1 << a.gl) - 1);
    place[x.r] = !exists ? -1 : direct ? (p.qs + (row >> a.gl)) * a.Hq + p.g * a.G + h : p.slot * kRows + row0 + x.r;
    if (!direct && exists) {
      a.part_m[place[x.r]] = m;
      a.part_l[place[x.r]] = sum;
    }
  }
  named_bar(2 + x.t, 128);
  if (D == 64 && x.w4 >= 2) return;  // lanes 64 .. 127 repeat the dims
#pragma unroll 1
  for (int j0 = 0; j0 < rows; j0 += 8) {
    uint32_t u[8], v[8];
    tmem_ld8(oa + j0, u);
    if (both) tmem_ld8(oa + 64 + j0, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float w0 = wts[j0 + e], w1 = wts[64 + j0 + e];
      float o = w0 == 0.f ? 0.f : __uint_as_float(u[e]) * w0;
      if (both && w1 != 0.f) o = fmaf(__uint_as_float(v[e]), w1, o);
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
__global__ void __launch_bounds__(Lay<KT, D>::THREADS, 1)
    tree_main(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TreeArgs a) {
  using namespace tcg;
  using L = Lay<KT, D>;
  constexpr bool Q8 = L::Q8;
  constexpr int NS = L::NS;
  using W = std::conditional_t<Q8, __half, T>;  // of the weights before V's scale: at most 2^kMove
  extern __shared__ __align__(1024) uint8_t gb[];
  const Sync<L> sy{dev::smem_addr(gb)};
  if (sy.base & 1023u) {  // the swizzled tiles need it; a launch without static shared memory has it
    if (threadIdx.x == 0) flag(PA_DEVERR_TIMEOUT);
    return;
  }
  const int wid = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      dev::mbar_init(sy.full(s), 1);
      dev::mbar_init(sy.conv(s), 4);
      dev::mbar_init(sy.empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int b = 0; b < 2; ++b) {
        dev::mbar_init(sy.sfull(t, b), 1);
        dev::mbar_init(sy.sfree(t, b), 4);
      }
      dev::mbar_init(sy.pfull(t), 4);
      dev::mbar_init(sy.pdone(t), 1);
      dev::mbar_init(sy.qfull(t), 1);
      dev::mbar_init(sy.qfree(t), 1);
      dev::mbar_init(sy.ofree(t), 8);
      dev::mbar_init(sy.pub(t), 4);
      dev::mbar_init(sy.mfull(t), 1);
    }
    for (int i = 0; i < 4; ++i) dev::mbar_init(sy.pieces(i), 1);
    dev::mbar_init(sy.mdone(), 1);
    dev::fence_barrier_init();
    *reinterpret_cast<volatile int*>(gb + L::MISC + 16) = 0;                                       // items issued
    reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 32)[0] = 0;                                // force
    reinterpret_cast<volatile uint32_t*>(gb + L::MISC + 32)[1] = 0;
    dev::prefetch_tensormap(&tmK);
    dev::prefetch_tensormap(&tmV);
    dev::prefetch_tensormap(&tmQ);
  }
  if (wid == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sy.base + L::MISC),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  dev::grid_dependency_wait();  // the cache write before this kernel is visible
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gb + L::MISC);

  if (wid == 0) {
    fewer_registers<Q8>();
    produce<KT, L>(a, &tmK, &tmV, &tmQ, gb, sy);
  } else if (wid == 1) {
    fewer_registers<Q8>();
    multiply<T, L>(a, gb, sy, static_cast<uint32_t>(uniform(static_cast<int>(tmem))));
  } else if (wid == 2) {
    fewer_registers<Q8>();
  } else if (wid == 3) {
    fewer_registers<Q8>();
    plan<L>(a, gb, sy);
  } else if (wid < 12) {
    // ---- softmax warpgroups: thread r owns key r of a chunk -----------------------------
    more_registers<Q8>();
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
    int n = 0, n_s0 = 0, n_s1 = 0;  // chunks of this tile so far; per score buffer
    Cursor<L> k;
    k.i = k.it0 = k.ph = 0;
#pragma unroll 1
    for (;; k.close()) {
      k.open(sy, gb, ok);
      ok = __all_sync(FULL, ok);
      if (!__all_sync(FULL, k.live)) break;
      const Piece& p = k.p;
      const int half = k.pair ? 64 * t : 0, rows = k.pair ? min(64, p.rows - half) : p.rows;
      const int words = rows > 32 ? 2 : 1, pp = k.i & 1, shift = p.L - p.n;
      const uint32_t oc = x.tl + kColO + (k.pair ? 0 : 128 * pp) + 64 * t;
      const bool exists = r < rows && ((p.row0 + half + r) & ((1 << a.gl) - 1)) < a.G;  // row r (r < 64)
      bool seen = !exists, unset = true;  // row r has a reference; some row may have none
      float ref = 0.f;
      float2 l[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) l[j] = make_float2(0.f, 0.f);
      const int c_first = k.pair ? 0 : (t ^ k.ph) & 1, step = k.pair ? 1 : 2;
      const bool any = c_first < k.nc;
#pragma unroll 1
      for (int c = c_first; c < k.nc; c += step, ++n) {
        const int key0 = (p.c0 + c) * kKeys, jn = key0 + r - shift;  // node that key r is
        const bool masked = key0 + kKeys > shift;
        const int sb = k.pair ? c & 1 : 0;
        if (ok) ok = wait_warp(sy.sfull(t, sb), (sb ? n_s1 : n_s0) & 1);
        ++(sb ? n_s1 : n_s0);
        fence_after();
        float ks = sl2, vsc = 1.f;
        if constexpr (Q8) {
          const float* scales = reinterpret_cast<const float*>(gb + L::SCALES + (((k.it0 >> 1) + c) & 7) * 1024);
          if (key0 + r < p.L) {  // (stale past the end)
            ks = sl2 * scales[r];
            vsc = scales[128 + r];
          }
        }
        uint2 vis = make_uint2(FULL, FULL);  // the rows that see the key
        if (masked) {
          if (p.n <= 64 && ok) ok = wait_warp(sy.mfull(pp), (k.i >> 1) & 1);
          vis = visible<L>(a, gb, p, k.i, p.row0 + half, jn);
          __syncwarp();
        }
        const uint32_t sc = x.tl + (sb ? kColS2 : kColS) + 64 * t;
        uint32_t pk[32];  // weights, 16-bit pairs of rows
        bool moved = unset;
        for (;;) {
          if (moved) {
            if (ok && n > 0) ok = wait_warp(sy.pdone(t), (n - 1) & 1);  // (P^T free, O^T at rest)
            fence_after();
            const int what = settle<L>(x, sc, ks, vis, words, oc, exists, seen, ref);
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
          // 16 rows: exponents, their maximum, weights
          auto part = [&](auto q_c) {
            constexpr int Q = decltype(q_c)::value;
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
              top = max3(top, e[j].x, e[j].y);
              pk[8 * Q + j] = dev::pack2<W>(dev::ex2(e[j].x), dev::ex2(e[j].y));
            }
          };
          part(std::integral_constant<int, 0>{});
          part(std::integral_constant<int, 1>{});
          if (words == 2) {
            part(std::integral_constant<int, 2>{});
            part(std::integral_constant<int, 3>{});
          }
          if (moved || !bar_or(bar, 128, top > kMove)) break;
          moved = true;
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.sfree(t, sb));  // the scores are read
#pragma unroll
        for (int j = 0; j < 16; ++j) add16x2<W>(l[j], pk[j]);  // l sums the rounded weights
        if (words == 2) {
#pragma unroll
          for (int j = 16; j < 32; ++j) add16x2<W>(l[j], pk[j]);
        }
        if constexpr (Q8) {  // times V's scale, which is the key's: rounded once more
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float2 w = dev::unpack2<W>(pk[j]), y = mul2(w, vsc);
            // (a weight of 0 must not meet a stale or NaN scale)
            pk[j] = masked ? dev::pack2<T>(w.x == 0.f ? 0.f : y.x, w.y == 0.f ? 0.f : y.y) : dev::pack2<T>(y.x, y.y);
          }
        }
        if (ok && n > 0) ok = wait_warp(sy.pdone(t), (n - 1) & 1);  // P^T's buffer is free
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(prow + ((j ^ (r & 7)) << 4)) =
              make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        if (words == 2) {
#pragma unroll
          for (int j = 4; j < 8; ++j)
            *reinterpret_cast<uint4*>(prow + ((j ^ (r & 7)) << 4)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        }
        if (masked) {
          const int vi = k.it0 + 2 * c + 1, vs = vi % NS;
          if (ok) ok = __all_sync(FULL, wait_issued(sy.issued(), vi)) && wait_warp(sy.ready(vs), (vi / NS) & 1);
          fence_after();
          guard<T, L>(x, gb, gb + L::RING + vs * L::SLOT, pbuf, (p.c0 + c) & 1, k.pair, jn, p.n, words, oc,
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
        pubs[64 * t + r] = make_float2(have && exists && seen ? ref : -INFINITY, sum);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.pub(t));
      // the warpgroup with the last chunk joins both accumulators; with half of
      // the rows each, each writes its own
      if (k.pair || ((k.ph + k.nc - 1) & 1) == t) {
        if (!k.pair && ok) ok = wait_warp(sy.pub(t ^ 1), k.i & 1);  // (after that tile's last product)
        named_bar(bar, 128);
        fence_after();
        write_rows<T, L>(a, x, p, pubs, x.tl + kColO + (k.pair ? 64 * t : 128 * pp), !k.pair, half, rows, exists);
      }
      if (ok) ok = wait_warp(sy.mfull(pp), (k.i >> 1) & 1);  // (every phase is seen in order)
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.ofree(pp));
    }
    if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  } else if (Q8) {
    fewer_registers<Q8>();
    convert<KT, T, L>(gb, sy);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (wid == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

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
  const int4 s0 = a.split[2 * k0], s1 = a.split[2 * k0 + 1];  // parts, first slot, first query row, item row | kv head, rows
  const int h = (s0.w + row) & ((1 << a.gl) - 1);
  if (s0.x == 0 || row >= s1.y || h >= a.G) return;
  auto slot_row = [&](int i) { return static_cast<size_t>(i == 0 ? s0.y : 2 * (k0 + i)) * kRows + row; };
  float M = -INFINITY, ls = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < s0.x; i0 += 32) {
    const int n = min(32, s0.x - i0);
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
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(FULL, w, i);
      const float* src = a.part_o + slot_row(i0 + i) * D + lane * V;
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const float2 f = *reinterpret_cast<const float2*>(src + v);
        acc[v] = fmaf(wi, f.x, acc[v]);
        acc[v + 1] = fmaf(wi, f.y, acc[v + 1]);
      }
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

// ---- launch ------------------------------------------------------------------
pa_status encode(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* p, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!fn) return fail(PA_ERR_CUDA, "pa_tree_attention: cuTensorMapEncodeTiled unavailable");
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(m, dt, rank, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(PA_ERR_CUDA, "pa_tree_attention: tensor map encode failed (%d)", static_cast<int>(r));
  return PA_OK;
}
// TMA map over a 16-bit cache of head_dim 128 whose box is one (block, kv
// head) tile, landing as [group of 8 tokens][span of 64 dims][8][128 B]: the
// 8-row groups of a span are evenly spaced over a run of tiles, as one UMMA
// operand of many tiles wants them.
pa_status make_group_map(CUtensorMap* m, const void* cache, int Hkv, int num_blocks, CUtensorMapDataType dt) {
  const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(2) * Hkv, static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[4] = {256, 128, 2048, static_cast<cuuint64_t>(4096) * Hkv};
  const cuuint32_t box[5] = {64, 8, 2, 2, 1};
  return encode(m, dt, 5, cache, dims, strides, box);
}
// TMA map over q [T][Hq][D] whose box is a 64-dim span of gp heads (a group,
// padded to a power of two) of as many nodes as make 32 rows.
pa_status make_q_map(CUtensorMap* m, const void* q, int D, int Hq, int T, int gp, CUtensorMapDataType dt) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(D) * 2 * Hq};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(gp), static_cast<cuuint32_t>(gp < 32 ? 32 / gp : 1)};
  return encode(m, dt, 3, q, dims, strides, box);
}

template <typename KT, typename T, int D>
pa_status launch_t(const TreeLaunch& l, CUtensorMapDataType dt, cudaStream_t stream) {
  using L = Lay<KT, D>;
  constexpr int EB = static_cast<int>(sizeof(KT));
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
  a.gl = 0;
  while ((1 << a.gl) < a.G) ++a.gl;
  const float mag = l.scale < 0.f ? -l.scale : l.scale;
  // a scale of 0 stays 0 for every finite score and leaves masked ones at -inf
  a.scale_log2 = mag * 1.4426950408889634f > 1e-30f ? mag * 1.4426950408889634f : 1e-30f;
  a.negate = l.scale < 0.f ? 1u : 0u;
  a.out_f32 = l.out_dtype == PA_DTYPE_F32;
  a.min_units = kItem + 2;
  const size_t rows = static_cast<size_t>(2) * a.n_cta * kRows;
  a.part_o = static_cast<float*>(l.workspace);
  a.part_m = a.part_o + rows * D;
  a.part_l = a.part_m + rows;
  a.split = reinterpret_cast<int4*>(a.part_l + rows);

  CUtensorMap tmK, tmV, tmQ;
  for (int v = 0; v < 2; ++v) {
    CUtensorMap* m = v ? &tmV : &tmK;
    const void* cache = v ? l.v_cache : l.k_cache;
    const pa_status st = D * EB == 256
                             ? make_group_map(m, cache, l.Hkv, l.num_blocks, dt)
                             : make_kv_map(m, cache, l.Hkv, l.num_blocks, D * EB, EB, dt, "pa_tree_attention");
    if (st != PA_OK) return st;
  }
  const pa_status sq = make_q_map(&tmQ, l.q, D, l.Hq, l.T, 1 << a.gl,
                                  std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
  if (sq != PA_OK) return sq;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices)
    return fail(PA_ERR_CUDA, "pa_tree_attention: no CUDA device");
  static std::once_flag once[kMaxDevices];
  static cudaError_t setup[kMaxDevices];
  std::call_once(once[dev], [dev] {
    setup[dev] = cudaFuncSetAttribute(tree_main<KT, T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  });
  if (setup[dev] != cudaSuccess)
    return fail(PA_ERR_CUDA, "pa_tree_attention: %s", cudaGetErrorString(setup[dev]));
  cudaError_t e = launch_dependent(tree_main<KT, T, D>, dim3(static_cast<unsigned>(a.n_cta)), dim3(L::THREADS),
                                   L::BYTES, stream, tmK, tmV, tmQ, a);
  if (e == cudaSuccess && l.max_context_len > kKeys)
    e = launch_dependent(tree_merge<T, D>, dim3(static_cast<unsigned>(a.n_cta), kRows / kMergeRows),
                         dim3(32 * kMergeRows), 0, stream, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_tree_attention launch: %s", cudaGetErrorString(e));
  return PA_OK;
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
