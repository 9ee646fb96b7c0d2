// Parts that both tree-attention kernels share: the batch's work and its planner
// warp, the ring of K and V chunks and its producer warp, the converters of
// 1-byte codes, bounded waits, tensor-memory access.
#pragma once

#include "device_common.cuh"
#include "tcgen05.cuh"

namespace pa {
namespace {

__device__ uint32_t g_tree_err;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kKeys = 128;  // keys per chunk
constexpr int kBlk = kKeys / 16;
constexpr uint32_t kTmemCols = 512;
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
  float* part_o;    // [2 * CTAs][slot_rows][D], then m and l [2 * CTAs][slot_rows]
  float* part_m;
  float* part_l;
  int4* split;      // [CTAs][2]: the item that CTA k leaves unfinished (Split), parts 0: none
  int32_t B, T, Hq, Hkv, G, max_blocks, num_blocks, max_context_len, max_q_len, words;
  int32_t gl;         // log2 of the rows of a node: its heads, up to a power of two
  int32_t min_units;  // units a CTA takes at least
  int32_t n_cta;
  int32_t item_rows;  // rows of an item at most
  int32_t slot_rows;  // rows of a set of partial rows
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
  s.tiles = ((s.n << a.gl) + a.item_rows - 1) / a.item_rows;
  s.nch = max(1, (s.L + kKeys - 1) / kKeys);  // a sequence without keys still owns its zero rows
  return s;
}
// An item's cost in units: its chunks, and kItem for its start and end (32
// sequences of 32 kv heads, mean context 1044: 124, 112, 105, 106 us at 2 .. 5).
constexpr int kItem = 4;
constexpr int kMaxUnits = INT32_MAX / 2;
__device__ __forceinline__ int units_of(const TreeArgs& a, const Seq& s) { return s.tiles * a.Hkv * (s.nch + kItem); }

// One item's run of chunks [c0, c1) for a CTA.
struct __align__(16) Piece {
  int qs, n, L, row0;    // the sequence; the item's first row
  int g, rows, c0, c1;   // kv head; the item's rows; chunks
  int b, slot, live, last;  // slot: its set of partial rows (-1: the whole item); live 0: no more pieces
};

// ---- shared memory -----------------------------------------------------------
// ROWS: the kernel with a thread per row (items of up to 256 rows), else the one
// with a thread per key (up to 64; with bf16 weights 32, whose low halves take the
// other 32 columns).
template <typename KT, typename T, int D_, bool ROWS_>
struct Lay {
  static constexpr bool Q8 = sizeof(KT) == 1, ROWS = ROWS_;
  // bf16 weights are the sum of two, which hold 16 bits.
  static constexpr bool SPLIT = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int D = D_;
  static constexpr int SPANS = D / 64;               // 128-byte spans of a 16-bit row
  // Q of pieces, places of HQ rows [span][HQ][128 B].  Two: a piece of up to HQ
  // rows takes one, in turns, a larger one both.  1-byte caches have one.
  static constexpr int HQ = ROWS ? 128 : 64;
  static constexpr int QP = Q8 ? 1 : 2;
  static constexpr int ITEM = ROWS ? QP * HQ : SPLIT ? HQ / 2 : HQ;  // rows of an item
  static constexpr int QTILE = HQ * D * 2;
  static constexpr int SLOT = kKeys * D * 2;         // one K or V chunk, 16-bit
  static constexpr int GRP = 1024 * SPANS;           // 8 keys of a slot: [span][8][128 B]
  static constexpr int P0 = QP * QTILE;              // P^T [tile][128 keys][128 B] (a thread per key)
  static constexpr int RING = P0 + (ROWS ? 0 : 2 * 16384);
  static constexpr int NS = D == 64 ? 10 : Q8 ? 4 : 5;
  // 1-byte caches: codes land in stages of their own, and are converted into the ring
  static constexpr int NL = Q8 ? (ROWS ? 3 : 2) : NS;  // places that chunks land in
  static constexpr int PRODUCERS = Q8 ? 2 : 1;
  static constexpr int STAGE = RING + NS * SLOT;
  static constexpr int SCALES = STAGE + (Q8 ? NL * kKeys * D : 0);  // [8 chunks][K 128, V 128] float
  static constexpr int BAR = SCALES + (Q8 ? 8 * 1024 : 0);
  static constexpr int NBAR = 2 * NL + 2 * NS + 23;
  static constexpr int MISC = (BAR + NBAR * 8 + 15) & ~15;  // tensor memory, items issued, force; at 64: bad keys
  static constexpr int PIECE = MISC + 128;           // Piece [4]
  static constexpr int PUB = PIECE + 4 * 48;         // float2 [2 tiles][HQ]
  static constexpr bool WORDS = !ROWS || Q8;         // the planner fetches mask words
  static constexpr int MASK = PUB + 16 * HQ;         // uint64 [2 pieces][64 nodes]
  static constexpr int BYTES = MASK + (WORDS ? 1024 : 0);
  static constexpr int THREADS = Q8 ? 512 : 384;
  // log2 of how far below its row's maximum a reference is set, and of how far that
  // maximum may outgrow it.  f16 weights: a row's largest is 2^7 .. 2^15, finite and as
  // far above what f16 drops as it goes, so that one of 2^-21 of it has all its bits.
  // bf16 drops nothing, and its values may be so large that a lift would overflow their
  // sum.  (1-byte caches: the maximum is of weight x V scale, which is what is rounded.
  // The weight itself is float32: 2^95 with scales of 2^-80, which smaller ones count as
  // here.)
  static constexpr float LIFT = SPLIT ? 0.f : 7.f, MOVE = SPLIT ? 8.f : 15.f;
  static constexpr int QREADY = 0;  // (Q is ready once it has landed)
  static constexpr int HIGH = Q8 ? 176 : 200, LOW = Q8 ? 80 : 104;  // registers: softmax threads', the others'
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// ---- waits -------------------------------------------------------------------
// Bounded, at about 2 s: a try that comes to nothing takes 3.8 us, whatever its
// hint.  (Inlined and without a clock, to keep the code small; a function call
// would tie every role to one register count.)
constexpr int kTries = 500000;
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
// Wait until ring item i is on its way into its slot (issued by the producer, or
// begun by the converters).  A slot's barrier tells one phase from the next by
// parity only; with the item under way, the slot's phase before it is over.
__device__ __forceinline__ bool wait_issued(uint32_t count, int item) {
#pragma unroll 1
  for (int i = 0; i < 16 * kTries; ++i) {  // (200 ns each)
    int v;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(count) : "memory");
    if (v > item) return true;
    __nanosleep(200);
  }
  return false;
}
__device__ __forceinline__ void publish(uint32_t count, int items) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(count), "r"(items) : "memory");
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
template <typename L>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::LOW));
}
template <typename L>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::HIGH));
}

// ---- tensor memory -----------------------------------------------------------
// Loads that have arrived when they return (load and wait in one statement, so
// no use of the registers can be scheduled between them).
#define PA_8(c, r, i) c(r[i]), c(r[i + 1]), c(r[i + 2]), c(r[i + 3]), c(r[i + 4]), c(r[i + 5]), c(r[i + 6]), c(r[i + 7])
#define PA_R8(r, i) PA_8("=r", r, i)
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
// 16 rows (lanes 16 h .. of the warp's 32) of 128 columns: thread 4 a + b has
// columns 8 i + 2 b and + 1 of row a in r[4 i], r[4 i + 1], of row a + 8 in the
// next two.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : PA_R8(r, 0), PA_R8(r, 8), PA_R8(r, 16), PA_R8(r, 24), PA_R8(r, 32), PA_R8(r, 40), PA_R8(r, 48), PA_R8(r, 56)
      : "r"(taddr)
      : "memory");
}
#undef PA_R8
#define PA_I8(r, i) PA_8("r", r, i)
// The same rows of 64 columns: thread 4 a + b gives column 4 i + b of rows a, a + 8
// in r[2 i], r[2 i + 1].
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      PA_I8(r, 0), PA_I8(r, 8), PA_I8(r, 16), PA_I8(r, 24)
      : "memory");
}
#undef PA_I8
#define PA_RW8(r, i) PA_8("+f", r, i)
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 128 columns under one wait.
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&f)[128]) {
#pragma unroll
  for (int i = 0; i < 128; i += 32) {
    uint32_t u[32];
    tcg::ld32(taddr + i, u);
#pragma unroll
    for (int j = 0; j < 32; ++j) f[i + j] = __uint_as_float(u[j]);
  }
  tcg::wait_ld();
#pragma unroll
  for (int j = 0; j < 128; j += 8) asm volatile("" : PA_RW8(f, j));  // no use of a register moves above the wait
}
#undef PA_RW8
#undef PA_8

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
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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
// What a pair of weights has beyond its bf16 halves, rounded to bf16 in turn.
__device__ __forceinline__ uint32_t low_half(float2 w, uint32_t pair) {
  const float2 h = dev::unpack2<__nv_bfloat16>(pair);
  return dev::pack2<__nv_bfloat16>(w.x - h.x, w.y - h.y);
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
// log2 of a V scale's size, for references.
__device__ __forceinline__ float log2_scale(float v) { return __log2f(fmaxf(fabsf(v), 0x1p-80f)); }
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
  __device__ __forceinline__ uint32_t full(int s) const { return at(s); }                // landing place s: landed
  __device__ __forceinline__ uint32_t taken(int s) const { return at(L::NL + s); }       // 1-byte: its codes are read
  __device__ __forceinline__ uint32_t conv(int s) const { return at(2 * L::NL + s); }    // and converted into slot s
  __device__ __forceinline__ uint32_t empty(int s) const { return at(2 * L::NL + L::NS + s); }  // slot used
  __device__ __forceinline__ uint32_t ready(int s) const { return L::Q8 ? conv(s) : full(s); }
  __device__ __forceinline__ uint32_t ext(int i) const { return at(2 * L::NL + 2 * L::NS + i); }
  __device__ __forceinline__ uint32_t sfull(int t) const { return ext(t); }         // scores of tile t
  __device__ __forceinline__ uint32_t sfree(int t) const { return ext(2 + t); }     // and read
  __device__ __forceinline__ uint32_t pfull(int t) const { return ext(4 + t); }     // weights of tile t written
  __device__ __forceinline__ uint32_t pdone(int t) const { return ext(6 + t); }     // their product with V ended
  __device__ __forceinline__ uint32_t qfull(int i) const { return ext(8 + i) ; }    // Q of a piece landed
  __device__ __forceinline__ uint32_t qfree(int i) const { return ext(10 + i); }    // its last scores are computed
  __device__ __forceinline__ uint32_t ofree(int i) const { return ext(12 + i); }    // piece parity i: all are done
  __device__ __forceinline__ uint32_t pub(int t) const { return ext(14 + t); }      // tile t's l and references
  __device__ __forceinline__ uint32_t mfull(int i) const { return ext(16 + i); }    // mask words of a piece
  __device__ __forceinline__ uint32_t pieces(int i) const { return ext(18 + i); }   // piece i % 4 published
  __device__ __forceinline__ uint32_t mdone() const { return ext(22); }             // after a timeout: no products
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
  // Sequences are read 32 at a time, a lane each, and once where that is the batch:
  // every read of them is a round trip to L2 at the start of the CTA.
  Seq mine;
  int group = -1;
  auto read = [&](int g, bool rep) {
    if (g == group) return;
    group = g;
    const int b = 32 * g + lane;
    mine = b < a.B ? seq_of(a, b, rep) : Seq{0, 0, 0, 0, 0};
  };
  auto seq = [&](int b) {
    read(b >> 5, false);
    return Seq{__shfl_sync(FULL, mine.qs, b & 31), __shfl_sync(FULL, mine.n, b & 31), __shfl_sync(FULL, mine.L, b & 31),
               __shfl_sync(FULL, mine.tiles, b & 31), __shfl_sync(FULL, mine.nch, b & 31)};
  };
  int64_t sum = 0;
  int most = 0, least = INT32_MAX;  // items per kv head, of sequences with rows
#pragma unroll 1
  for (int g = 0; 32 * g < a.B; ++g) {
    read(g, report);
    sum += units_of(a, mine);
    most = max(most, mine.tiles);
    if (mine.tiles > 0) least = min(least, mine.tiles);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL, sum, off);
  most = __reduce_max_sync(FULL, most);
  least = __reduce_min_sync(FULL, least);
  // Where every sequence has the same number of items per kv head, that many CTAs
  // side by side take the same chunks of one item each, at the same time, and all
  // but the first find them in L2 (unless that leaves many CTAs out).  512 rows,
  // 805 MB of K/V in all: 323 us for 330, repeated for seconds, at the power limit,
  // 340 for 359.
  const int side = L::ROWS && most == least && most > 1 && a.n_cta % most * 32 <= a.n_cta ? most : 1;
  const int groups = a.n_cta / side, me = static_cast<int>(blockIdx.x) / side;
  const int tile = static_cast<int>(blockIdx.x) - me * side;
  sum /= side;
  auto units = [&](const Seq& s) { return units_of(a, s) / side; };
  // more than the launch was checked for: q_start has ranges that overlap
  if (sum > kMaxUnits && report && lane == 0) flag(PA_DEVERR_QUERY_RANGE);
  const int total = sum > kMaxUnits ? 0 : static_cast<int>(sum);
  const int upc = max((total + groups - 1) / groups, a.min_units);
  const int start = me < groups ? min(me * upc, total) : total, end = min(start + upc, total);
  int b = 0, ub = 0;  // the sequence of unit `u`, and the units before it
#pragma unroll 1
  for (int b0 = 0; start < end; b0 += 32) {
    read(b0 >> 5, false);
    const int w = units(mine);
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
        Seq s = seq(b);
#pragma unroll 1
        while (u >= ub + units(s)) {
          ub += units(s);
          s = seq(++b);
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
        p.g = side > 1 ? item : item / s.tiles;
        p.row0 = (side > 1 ? tile : item - p.g * s.tiles) * a.item_rows;
        p.rows = min(a.item_rows, (s.n << a.gl) - p.row0);
        p.slot = p.c0 == 0 && p.c1 == s.nch ? -1 : 2 * static_cast<int>(blockIdx.x) + (i == 0 ? 0 : 1);
        if (p.c0 == 0 && p.c1 < s.nch) {  // the item goes on in the next CTAs: what tree_merge needs
          sp0 = make_int4((ub + (item + 1) * cost - 1) / upc - me + 1, p.slot, s.qs, p.row0);
          sp1 = make_int4(p.g, p.rows, side, 0);
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
    // (the first two pieces' words find their places free)
#pragma unroll 1
    for (int m = i == 1 ? 0 : max(i - 2, 2); m <= (i == 1 ? 1 : i - 2) && m < pieces; ++m) {
      const Piece& x = ring[m & 3];
      if (L::WORDS && x.n <= 64 && x.c1 * kKeys > x.L - x.n)
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

// The producer warps: each piece's Q rows, and its K and V chunks into the ring,
// one box per block.  1-byte caches have two of them, with half of each chunk's
// blocks (a single thread's issue rate would bound their 32 copies per chunk).
template <typename KT, typename L>
__device__ __forceinline__ void produce(const TreeArgs& a, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                     const CUtensorMap* tmQ, uint8_t* gb, Sync<L> sy, int part) {
  constexpr int NL = L::NL, D = L::D, kPart = kBlk / L::PRODUCERS;
  const int lane = static_cast<int>(threadIdx.x & 31);
  bool ok = true;
  int it = 0, q_issued = 0, q_free = 0;  // ring items, Qs of pieces, pieces done with theirs
  bool before_both = false;
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
  // place is free once `need` pieces have ended their last scores.
  auto load_q = [&](const Piece& x, int i, int need) {
    if (part > 0) return;
#pragma unroll 1
    for (; q_free < need; ++q_free)
      if (ok) ok = wait_warp(sy.qfree(q_free & 1), (q_free >> 1) & 1);
    if (!ok) return;
    ++q_issued;
    const bool both = x.rows > L::HQ;
    const int br = max(32, 1 << a.gl);
    const int sp = lane % L::SPANS, y = lane / L::SPANS * br;
    const bool mine = y < x.rows;
    const uint32_t n = static_cast<uint32_t>(__popc(__ballot_sync(FULL, mine)));
    if (lane == 0) dev::mbar_arrive_expect_tx(sy.qfull(i & 1), n * br * 128);
    __syncwarp();
    if (mine)
      dev::tma_load_3d(sy.base + (both ? y / L::HQ : i % L::QP) * L::QTILE + (sp * L::HQ + y % L::HQ) * 128, tmQ,
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
    // a piece in both places, and the one after it, wait for the piece before to
    // end: the first chunk then goes ahead
    const bool late = L::QP == 1 || p.rows > L::HQ || before_both;
    before_both = p.rows > L::HQ;
    if (!late) load_q(p, i - 1, i - 2);
#pragma unroll 1
    for (int c = p.c0; c < p.c1; ++c) {
      const int k4 = (c - p.c0) & 3;
      if (k4 == 0) {
        ids = ids_next;
        ids_next = c + 4 < p.c1 ? fetch(p, (c + 4) * kBlk) : ids_n;
      }
      int blk[kPart];  // the chunk's block ids
#pragma unroll
      for (int k = 0; k < kPart; ++k) blk[k] = __shfl_sync(FULL, ids, k4 * kBlk + kPart * part + k);
      const int live = max(0, min(kPart, nblk - c * kBlk - kPart * part));  // those that exist
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        const int s = it % NL;
        if (ok && it >= NL) ok = wait_warp(L::Q8 ? sy.taken(s) : sy.empty(s), (it / NL - 1) & 1);
        if (!ok) break;
        dev::fence_proxy_async_smem();  // the softmax's and converters' accesses precede the refill
        const uint32_t bar = sy.full(s);
        const uint32_t dst = sy.base + (L::Q8 ? L::STAGE + s * (L::SLOT / 2) + part * kPart * 2048
                                              : L::RING + s * L::SLOT + part * kPart * 32 * D);
        ++it;
        if (lane == 0) {
          const int bytes = L::Q8 ? 16 * D + (v ? 0 : 128) : 32 * D;  // (K's codes come with both scale rows)
          dev::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live * bytes));
          if (!L::Q8 && part == 0) publish(sy.issued(), it);
        }
        __syncwarp();
        const CUtensorMap* m = v ? tmV : tmK;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kPart; ++k) {
            if (k >= live) break;
            if constexpr (L::Q8) {
              dev::tma_load_3d(dst + k * 2048, m, bar, 0, p.g * 16, blk[k]);
              if (v == 0) {
                const uint32_t sc = sy.base + L::SCALES + (((it - 1) >> 1) & 7) * 1024 + (part * kPart + k) * 64;
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
  for (int i = max(0, it - NL); i < it; ++i) wait_thread(sy.full(i % NL), (i / NL) & 1);
  if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
  __syncwarp();
}

// A walk over the chunks of all pieces, in order.
template <typename L>
struct Cursor {
  Piece p;
  int i, c, nc, it0, ph;  // piece, chunk, its chunks, ring items before it, tile of its chunk 0
  bool live, both;        // both: each tile half of the rows; else alternate chunks
  __device__ __forceinline__ void open(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    live = sy.piece(gb, i, p, ok);
    c = 0;
    nc = p.c1 - p.c0;
    both = p.rows > L::HQ;
  }
  __device__ __forceinline__ void start(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    i = it0 = ph = 0;
    open(sy, gb, ok);
  }
  __device__ __forceinline__ void close() {
    it0 += 2 * nc;
    if (!both) ph ^= nc & 1;
    ++i;
  }
  // true: the next chunk is another piece's
  __device__ __forceinline__ bool next(const Sync<L>& sy, const uint8_t* gb, bool& ok) {
    if (++c < nc) return false;
    close();
    open(sy, gb, ok);
    return true;
  }
  __device__ __forceinline__ int tile() const { return (ph + c) & 1; }
};

// The converter warpgroup (1-byte caches): codes of a landed chunk -> 16-bit
// values in its slot of the ring, in the layout the MMAs read.  queries: what it does
// besides for a piece, behind the first chunk's codes.
struct AsLanded {
  __device__ __forceinline__ void operator()(const Piece&, int, bool&) const {}
};
template <typename KT, typename T, typename L, typename F = AsLanded>
__device__ __forceinline__ void convert(uint8_t* gb, Sync<L> sy, F queries = F{}) {
  constexpr int NS = L::NS, NL = L::NL;
  const int lane = static_cast<int>(threadIdx.x & 31), i0 = static_cast<int>(threadIdx.x) - 384;
  bool ok = true;
  int it = 0;
  Piece p;
#pragma unroll 1
  for (int i = 0; sy.piece(gb, i, p, ok); ++i) {
    const int n = 2 * (p.c1 - p.c0);
#pragma unroll 1
    for (int k = 0; k < n; ++k, ++it) {
      const int s = it % NL, to = it % NS;
      if (ok) ok = wait_warp(sy.full(s), (it / NL) & 1);
      const uint8_t* st = gb + L::STAGE + s * (L::SLOT / 2);
      uint4 w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // 16 codes: chunk c16 of row `key`
        const int x = i0 + 128 * j, key = x >> 3, c16 = x & 7;
        w[j] = *reinterpret_cast<const uint4*>(st + key * 128 + ((c16 ^ (key & 7)) << 4));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.taken(s));
      if (ok && it >= NS) ok = wait_warp(sy.empty(to), (it / NS - 1) & 1);
      if (i0 == 0) publish(sy.issued(), it + 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = i0 + 128 * j, key = x >> 3, c16 = x & 7, cc = 2 * (c16 & 3);
        uint32_t f[8];
        dev::code8x4_to<KT, T>(w[j].x, f[0], f[1]);
        dev::code8x4_to<KT, T>(w[j].y, f[2], f[3]);
        dev::code8x4_to<KT, T>(w[j].z, f[4], f[5]);
        dev::code8x4_to<KT, T>(w[j].w, f[6], f[7]);
        uint8_t* row = gb + L::RING + to * L::SLOT + (key >> 3) * L::GRP + (c16 >> 2) * 1024 + (key & 7) * 128;
        // (the two spans' threads store their halves in opposite order: no bank conflict)
        const bool up = c16 & 4;
        *reinterpret_cast<uint4*>(row + (((cc + up) ^ (key & 7)) << 4)) =
            make_uint4(up ? f[4] : f[0], up ? f[5] : f[1], up ? f[6] : f[2], up ? f[7] : f[3]);
        *reinterpret_cast<uint4*>(row + (((cc + !up) ^ (key & 7)) << 4)) =
            make_uint4(up ? f[0] : f[4], up ? f[1] : f[5], up ? f[2] : f[6], up ? f[3] : f[7]);
      }
      dev::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.conv(to));
      if (k == 1) queries(p, i, ok);
    }
  }
  if (!ok && lane == 0) flag(PA_DEVERR_TIMEOUT);
}

// Barriers, tensor memory (its address is returned), the kernel before this one.
template <typename L>
__device__ __forceinline__ uint32_t setup(uint8_t* gb, Sync<L> sy, int wid, const CUtensorMap* tmK,
                                          const CUtensorMap* tmV, const CUtensorMap* tmQ) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::NL; ++s) {
      dev::mbar_init(sy.full(s), L::PRODUCERS);
      dev::mbar_init(sy.taken(s), 4);
    }
    for (int s = 0; s < L::NS; ++s) {
      dev::mbar_init(sy.conv(s), 4);
      dev::mbar_init(sy.empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      dev::mbar_init(sy.sfull(t), 1);
      dev::mbar_init(sy.sfree(t), 4);
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
    dev::prefetch_tensormap(tmK);
    dev::prefetch_tensormap(tmV);
    dev::prefetch_tensormap(tmQ);
  }
  if (wid == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sy.base + L::MISC),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  dev::grid_dependency_wait();  // the cache write before this kernel is visible
  tcg::fence_before();
  __syncthreads();
  tcg::fence_after();
  return *reinterpret_cast<volatile uint32_t*>(gb + L::MISC);
}
__device__ __forceinline__ void teardown(int wid, uint32_t tmem) {
  __syncwarp();
  tcg::fence_before();
  __syncthreads();
  if (wid == 1) {
    tcg::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace
}  // namespace pa
