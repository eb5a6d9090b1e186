// The attention kernel: softmax(scale * q k^T) v on the tensor cores, over the
// paged cache (bf16 or e4m3) or packed prompts.
//
// For a row i of scores s_ij = scale * log2(e) * q_i.k_j one pass over the keys
// keeps a reference M_i (the running maximum), l_i = sum_j 2^(s_ij - M_i) and
// O_i = sum_j 2^(s_ij - M_i) v_j; the output is O_i / l_i and the log of the
// sum ln 2 * (M_i + log2 l_i).  M_i only has to be near the maximum: it is
// raised, and O_i and l_i rescaled, when a score passes it by 2^8, so most
// blocks leave O_i, which lives in tensor memory, alone.
//
// Rows.  The q_heads / kv_heads query heads of a group share their keys, so a
// tile of 128 rows holds floor(128 / group) tokens times the group and every
// key block is read once for all of them.
//
// Work.  An item is (sequence, key-value head, row tile); it costs a unit for
// each 128-key block that any of its rows sees, and SETUP units that stand for
// what an item costs besides (its query rows, its first scores, its output).
// The units of all items in order are cut into equal runs, one per CTA (one CTA
// per SM), so few long sequences fill the GPU as well as many short ones.  A cut
// within SNAP units of an item's end moves there: splitting an item has a price
// too.  An item that lies in several runs leaves partial (M, l, O) in the
// workspace and the last CTA to finish merges them, in order: nothing waits,
// and results do not depend on the order of arrival.
//
// Roles of a CTA's warps: one copies key and value blocks into shared memory
// (TMA), one issues the matrix products, two load the query rows of the next
// run, and eight per tile do the softmax, two threads a row (a warp reaches
// only the 32 tensor-memory lanes of its place in its warpgroup).  For an e4m3
// cache eight more turn the codes into f16 (see below).
//
// Tiles.  Two tiles of rows share a CTA's key blocks and take turns: the
// products of one (about 1,100 cycles a block) run under the softmax of the
// other.  With one tile two score buffers take turns instead.
//
// What bounds it, measured on GB300 (152 SMs, 6.70 TB/s, 1,937 TFLOP/s bf16):
//   one tile, bf16    memory: 64 sequences of 8 tokens over 500-8000 cached, 64
//                     query and 8 key-value heads of 128, 188 us, 6.1 TB/s
//   one tile, e4m3    shared memory and instruction issue: 64 sequences of 16 over
//                     1000-16000, 298 us, 3.5 TB/s and 847 TFLOP/s
//   two tiles         a tile's softmax, about 1,600 cycles, where the other's
//                     products take 1,100: 3 prompts of 4000-6450 tokens, 32 and 8
//                     heads of 128, 687 us, 1,363 TFLOP/s
//   few blocks        latency: a call of 3 prompts of up to 21 tokens takes 10.5 us
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "attn_plan.cuh"

namespace {

enum { KIND_BF16 = 0, KIND_E4M3 = 1, KIND_PACKED = 2 };

constexpr int HALF_BYTES = BN * 128;  // 64 of the D columns of a block: 128 rows of one swizzled 128-byte line
constexpr float LAZY = 8.0f;        // log2 of how far scores may pass the reference: f16 weights hold 2^15
constexpr float ABOVE = 1.0f + 1.0f / 65536.0f;   // see the weights in two parts
constexpr int POLLS = 1 << 18;      // of a bounded wait (about 1 s)
constexpr int SMEM_LIMIT = 232448;
constexpr int ODD_NONE = 0x7f7f7f7f;
// Least and largest exponent of a value block's reference (see the e4m3 conversion).  The sum of weights is
// taken in units of 2^-e, and a weight reaches 2^LAZY: at -97 the sum of 2^23 keys stays below 2^128 (at the
// -120 of a block of zero vectors 256 keys passed it), and at 126 its unit is still a normal number.
constexpr int EV_MIN = -97, EV_MAX = 126;
constexpr int BYTE_ZERO = 15;       // vectors of this scale (below 2^-103) and less count as zero beside others
constexpr int SPREAD = 14;          // exponents apart that a block's vectors may be to share one scale
constexpr float WIDE = 1.2676506e30f;   // 2^100, in place of the exponent of a block's values: vectors have their own

struct AttnParams {
  Batch B;
  Rows Q;
  const uint8_t *ks, *vs;           // scale bytes (e4m3)
  int q_heads, kv_heads, group;
  int tile_tokens;                  // floor(128 / group)
  int causal;
  float c;                          // scale * log2(e)
  __nv_bfloat16* out;
  float* lse;
  float* ws;                        // partials: [cta][2][MT] of PART floats
  int* counters;                    // [cta][MT], zero between calls
  int* odd;                         // [cta][4][3][D] first keys with values that are not finite (see note_odd), else ODD_NONE
};

// Floats of one partial: M, l and its correction per row, then O as [D / 4][128] float4
template <int D> __host__ __device__ constexpr int part_floats() { return 3 * BM + BM * D; }

// ------------------------------------------------------------------- PTX
__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t a, unsigned n) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a), "r"(n) : "memory"); }
__device__ __forceinline__ void bar_expect(uint32_t a, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(a), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t a) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory"); }
__device__ __forceinline__ bool bar_try(uint32_t a, unsigned parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(a), "r"(parity) : "memory");
  return ok != 0;
}
// Bounded wait of a whole warp: false (and the handle flagged) instead of a
// hang, in all lanes or in none.  Once one wait has given up the others see
// the flag and give up within 256 polls.
__device__ __forceinline__ bool bar_wait_slow(uint32_t a, unsigned parity, int* flags) {
  for (int it = 0; it < POLLS; ++it) {
    if (__all_sync(FULL, bar_try(a, parity))) return true;
    if ((it & 255) == 255 && __any_sync(FULL, *(volatile int*)&flags[1])) return false;
  }
  atomicExch(&flags[1], 1);
  return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t a, unsigned parity, int* flags) {
  return __all_sync(FULL, bar_try(a, parity)) || bar_wait_slow(a, parity, flags);
}
// The same for a thread on its own
__device__ __forceinline__ bool bar_wait_slow1(uint32_t a, unsigned parity, int* flags) {
  for (int it = 0; it < POLLS; ++it) {
    if (bar_try(a, parity)) return true;
    if ((it & 255) == 255 && *(volatile int*)&flags[1]) return false;
  }
  atomicExch(&flags[1], 1);
  return false;
}
__device__ __forceinline__ bool bar_wait1(uint32_t a, unsigned parity, int* flags) {
  return bar_try(a, parity) || bar_wait_slow1(a, parity, flags);
}
// One lane of a converged warp, the same one every time; the compiler knows that only one is active
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
#define R8(r, o) "=r"((r)[o]), "=r"((r)[o + 1]), "=r"((r)[o + 2]), "=r"((r)[o + 3]), "=r"((r)[o + 4]), "=r"((r)[o + 5]), "=r"((r)[o + 6]), "=r"((r)[o + 7])
#define I8(r, o) "r"((r)[o]), "r"((r)[o + 1]), "r"((r)[o + 2]), "r"((r)[o + 3]), "r"((r)[o + 4]), "r"((r)[o + 5]), "r"((r)[o + 6]), "r"((r)[o + 7])
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* m, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(m), "r"(x), "r"(y), "r"(z) : "memory");
}
// 32 bytes, a whole memory sector
__device__ __forceinline__ void st_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), I8(w, 0) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[smem] B[smem], and with A in tensor memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
#define P8(r, o) "+r"((r)[o]), "+r"((r)[o + 1]), "+r"((r)[o + 2]), "+r"((r)[o + 3]), "+r"((r)[o + 4]), "+r"((r)[o + 5]), "+r"((r)[o + 6]), "+r"((r)[o + 7])
// Waits for this thread's loads; the registers pass through, so that no use of them moves before it
__device__ __forceinline__ void tc_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : P8(r, 0), P8(r, 8), P8(r, 16), P8(r, 24)::"memory");
}
// 32 columns of this warp's 32 lanes; the loads complete at tc_wait_ld
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
               "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24) : "r"(a));
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : R8(r, 0), R8(r, 8) : "r"(a));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : P8(r, 0), P8(r, 8)::"memory");
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
               ::I8(r, 0), I8(r, 8), "r"(a) : "memory");
}
__device__ __forceinline__ float ex2(float x) { float y; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float max3(float a, float b, float c) { float y; asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c)); return y; }
typedef unsigned long long u64;
__device__ __forceinline__ u64 pk(float lo, float hi) { u64 r; asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi)); return r; }
__device__ __forceinline__ void upk(u64 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) { u64 d; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c)); return d; }
__device__ __forceinline__ u64 add2(u64 a, u64 b) { u64 d; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b)); return d; }
__device__ __forceinline__ void group_sync(int id, int n) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool group_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"(id), "r"(n), "r"((uint32_t)v) : "memory");
  return r != 0;
}

// Shared-memory operand descriptor, 128-byte swizzle.  Rows of 128 bytes, 8 of
// them (1024 bytes) a swizzle atom.  Query and key blocks are K-major (a row
// per query or key, 64 of D in its line); value blocks are MN-major (a row per
// key, 64 of D in its line), where the leading offset leads to the next 64 of D.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t leading_bytes) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(leading_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f16, M = 128, fp32 accumulators; A and B are both f16 or both bf16
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, int n, bool b_mn_major) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// ------------------------------------------------------------------ planning
__device__ __forceinline__ Seq load_seq(const Batch& B, int b, int tile_rows) {
  Seq s;
  const int a = __ldg(B.cu + b), e = __ldg(B.cu + b + 1);
  const bool range = a >= 0 && e >= a && e <= B.n_tokens;
  s.row0 = range ? a : 0;
  s.n = range ? e - a : 0;
  s.kv = B.kv_len ? __ldg(B.kv_len + b) : s.n;
  s.bad = B.kv_len && !len_valid(B, s.kv);
  if (s.bad) s.kv = 0;
  s.tiles = (s.n + tile_rows - 1) / tile_rows;
  s.bad |= !range;
  return s;
}
struct Segment {      // a run of blocks of one item
  int b, head;
  int row0, ntok;     // packed rows of the tile's tokens
  int kv;             // cached tokens
  int lim0;           // keys the tile's first token sees (causal) or kv
  int j0, j1, nblk;   // blocks of this run, of the item
  int bad, more;      // invalid sequence; another run of this CTA follows
  long long start;    // unit of the item's first block
};

// The second part has 2^-16 of every weight on top (see the softmax), which the sum of weights does not: 2^-8 of
// the output's own rounding.
// Rounding the weights to bf16 costs little where many keys share the error.
// An item of few blocks has its weights in two bf16 parts and takes the product
// with the values twice: up to 1152 keys where copies bound (one tile: 1% of the
// time over the range, 2% up to 2048), up to 128 where the products do (a block of
// two tiles takes 2.5 instead of 1.6 us).
template <int KIND, int MT> __device__ __forceinline__ bool two_parts(const Segment& g) { return KIND != KIND_E4M3 && g.nblk <= (MT == 1 ? 9 : 1); }

// Walks one CTA's run of units.  Every role walks on its own.
struct Walker {
  long long at, u0, u1;   // first unit of the item, the run
  int b, head, t;
  Seq s;
  __device__ bool any() const { return at < u1; }
  __device__ void advance(const AttnParams& A, int tile_rows) {
    if (++t == s.tiles) {
      t = 0;
      if (++head == A.kv_heads) {
        head = 0;
        do { s = load_seq(A.B, ++b, tile_rows); } while (s.tiles == 0 && b + 1 < A.B.n_seqs);
      }
    }
  }
  __device__ bool next(const AttnParams& A, int tile_rows, Segment& g) {
    if (at >= u1) return false;
    g.b = b; g.head = head;
    g.row0 = s.row0 + t * tile_rows;
    g.ntok = min(tile_rows, s.n - t * tile_rows);
    g.kv = s.kv;
    g.lim0 = A.causal ? s.kv - s.n + t * tile_rows + 1 : s.kv;
    g.nblk = tile_blocks(s, t, tile_rows, A.causal);
    g.start = at + SETUP;
    g.j0 = (int)max(0ll, u0 - g.start);
    g.j1 = (int)min((long long)g.nblk, u1 - g.start);
    g.bad = s.bad;
    at = g.start + g.nblk;
    g.more = at < u1;
    if (g.more) advance(A, tile_rows);
    return true;
  }
};

// --------------------------------------------- values that are not finite
// Causal rows see a prefix of the keys, so what such values do to a row follows
// from three keys per column: the first with NaN, +inf and -inf.  Only blocks
// that some rows see in part need this; elsewhere the products carry it.
template <int D, bool FP8, typename Piece>
__device__ __forceinline__ void note_odd(int* odd, int* flag, Piece piece, int half, int key) {
#pragma unroll 1
  for (int i = 0; i < D / 16; ++i) {
    uint16_t* const v = (uint16_t*)piece(i);
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = v[e], inf = FP8 ? 0x7c00u : 0x7f80u;
      if ((w & inf) != inf) continue;
      v[e] = 0;
      const int kind = (w & 0x7fffu) != inf ? 0 : w >> 15 ? 2 : 1;
      atomicMin(odd + kind * D + half * (D / 2) + 8 * i + e, key);
    }
  }
  __threadfence();
  *(volatile int*)flag = 1;
}
// A factor of scores: above 0, where a masked score's -inf would make NaN, and finite, where a score of 0 would
__device__ __forceinline__ float positive(float x) { return fminf(fmaxf(x, 1.17549435e-38f), 3.40282347e38f); }
// The scale bytes of a cached token's key and, in bits 8 to 15, value; 0 where there is none
__device__ __forceinline__ int scale_bytes(const AttnParams& A, const Segment& g, int p) {
  if (p >= g.kv) return 0;
  const int page = __ldg(A.B.table + (size_t)g.b * A.B.max_pages + (p >> A.B.page_shift));
  if ((unsigned)page >= (unsigned)A.B.num_pages) return 0;
  const size_t at = ((size_t)(page * A.kv_heads + g.head) << A.B.page_shift) + (p & ((1 << A.B.page_shift) - 1));
  const int k = __ldg(A.ks + at), v = __ldg(A.vs + at);
  return (k == BYTE_NAN ? EXP_BIAS : k) | (v == BYTE_NAN ? EXP_BIAS : v) << 8;
}
// Exponent, as the weights have it, of a value vector that has its own
__device__ __forceinline__ int value_exponent(int byte) { return min(max(byte - EXP_BIAS, EV_MIN), EV_MAX); }
// A sum of weights times 2^x, x <= 0.  That of an e4m3 cache may be as large as 2^126 (see EV_MIN), so that the
// product is a normal number where 2^x alone is not: two steps.
template <bool FP8> __device__ __forceinline__ float scaled(float l, float x) {
  if (!FP8) return ex2(x) * l;
  const float h = ex2(0.5f * x);
  return h * l * h;
}
// What a row that sees keys 0 .. lim-1 has in a column (0: nothing)
template <int D> __device__ __forceinline__ float odd_value(const int* odd, int col, int lim) {
  const bool nan = __ldcg(odd + col) < lim, pos = __ldcg(odd + D + col) < lim, neg = __ldcg(odd + 2 * D + col) < lim;
  return nan || (pos && neg) ? quiet_nan() : pos ? INFINITY : neg ? -INFINITY : 0.0f;
}

// -------------------------------------------------------------------- kernel
template <int D, int KIND, int MT>
struct Cfg {
  static constexpr bool FP8 = KIND == KIND_E4M3;
  static constexpr int HALVES = D / 64;
  static constexpr int BUF = HALVES * HALF_BYTES;             // a block of keys or values in 16 bits
  static constexpr int QBYTES = MT * BUF;
  static constexpr int RAW = BN * D;                          // a block of codes
  static constexpr int NRAW = FP8 ? (D == 128 ? 4 : 8) : 0;
  static constexpr int SMALL = 3072;                          // barriers and bookkeeping, behind the buffers
  static constexpr int NBUF = FP8 ? (D == 128 ? 4 : 6) : (SMEM_LIMIT - SMALL - QBYTES) / BUF;
  static constexpr int NK = (NBUF + 1) / 2, NV = NBUF / 2;
  static constexpr int SMEM = QBYTES + NBUF * BUF + NRAW * RAW + SMALL;
  static constexpr int Q_WARP0 = 2, Q_WARPS = 2;
  static constexpr int SOFT_WARP0 = 4, SOFT_WARPS = 8;        // per tile
  static constexpr int CONV_WARP0 = SOFT_WARP0 + SOFT_WARPS * MT;
  static constexpr int CONV_WARPS = FP8 ? 8 : 0;
  static constexpr int WARPS = CONV_WARP0 + CONV_WARPS;
  static constexpr int THREADS = WARPS * 32;
  // Registers: five warpgroups start with 96 each; the first one, which copies and issues, or for e4m3 the
  // converting ones give up what the softmax needs to hold half a row of scores (64 sequences of 16 tokens over
  // 1000-16000 e4m3: 327 us with 96 for all, 297 with 120 and 72, 299 with 112 and 80).
  static constexpr int REGS_SOFT = MT == 2 ? 104 : FP8 ? 120 : 0, REGS_WORK = FP8 ? 96 : 64, REGS_CONV = 72;
  static_assert(REGS_SOFT == 0 || 128 * REGS_WORK + SOFT_WARPS * MT * 32 * REGS_SOFT + CONV_WARPS * 32 * REGS_CONV <= THREADS * 96, "register split");
  static constexpr int INFO = 8;                              // ring of block references (more than NK + 1)
};
// named barriers: pairs of softmax warps of a quarter of a tile's rows, tiles, converting warps
enum { BAR_PAIR = 1, BAR_TILE = 9, BAR_CONV = 11 };      // the last: one for keys, one for values

template <int D, int KIND, int MT>
__global__ void __launch_bounds__(Cfg<D, KIND, MT>::THREADS, 1)
sa_attention_kernel(const __grid_constant__ AttnParams A, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D, KIND, MT>;
  constexpr int NK = C::NK, NV = C::NV, NT = C::THREADS;
  extern __shared__ __align__(1024) uint8_t gbase[];
  const uint32_t base = saddr(gbase);
  const uint32_t q_at = base, k_at = q_at + C::QBYTES, v_at = k_at + NK * C::BUF, raw_at = v_at + NV * C::BUF;
  uint8_t* const small = gbase + (raw_at - base) + C::NRAW * C::RAW;
  const uint32_t bars = saddr(small);
  // barriers, 8 bytes each
  const uint32_t k_full = bars, k_empty = k_full + 8 * NK, v_full = k_empty + 8 * NK, v_empty = v_full + 8 * NV,
                 raw_full = v_empty + 8 * NV, raw_empty = raw_full + 8 * C::NRAW, s_full = raw_empty + 8 * C::NRAW,
                 p_full = s_full + 16,
                 o_done = p_full + 16,   // a run's last product, per tile; with one tile, also every product (second barrier)
                 q_full = o_done + 16, q_empty = q_full + 8, drain = q_empty + 8;
  static_assert(C::WARPS <= 20, "planning sums");
  static_assert(8 * (2 * NK + 2 * NV + 2 * C::NRAW + 9) <= 320, "barrier area");
  int* const work = (int*)(small + 320);                  // tensor-memory base, plan, merge flags [16]
  int* const odd_flag = (int*)(small + 640);              // whether a run has values that are not finite in such a block [4]
  float2* const info = (float2*)(small + 384);            // block references of an e4m3 cache [INFO]
  int* const red = (int*)(small + 448);                   // planning (20 sums and 2 places of 8 bytes), then the converters' maxima
  Segment* const runs = (Segment*)(small + 768);          // runs as the query warps announce them [4]
  static_assert(sizeof(Segment) <= 64, "ring of runs");
  float* const swap = (float*)(small + 1024);             // [tile][half][row]: between the two threads of a row
  float* const q_scale = (float*)(small + 2048);          // [2][row]: powers of two taken out of query rows (e4m3)
  static_assert(!C::FP8 || MT == 1, "the second tile's part of swap lies over q_scale");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile_rows = MT * A.tile_tokens;
  int* const flags = A.B.flags;

  // ---- set-up: barriers, tensor memory, and this CTA's run of units
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) { bar_init(k_full + 8 * i, C::FP8 ? 4 : 1); bar_init(k_empty + 8 * i, 1); }
    for (int i = 0; i < NV; ++i) { bar_init(v_full + 8 * i, C::FP8 ? 4 : 1); bar_init(v_empty + 8 * i, 1); }
    for (int i = 0; i < C::NRAW; ++i) { bar_init(raw_full + 8 * i, 1); bar_init(raw_empty + 8 * i, 4); }
    for (int i = 0; i < 2; ++i) { bar_init(s_full + 8 * i, 1); bar_init(p_full + 8 * i, C::SOFT_WARPS); bar_init(o_done + 8 * i, 1); }
    bar_init(q_full, C::FP8 ? C::Q_WARPS : 1);
    bar_init(q_empty, 1);
    bar_init(drain, 1);
    for (int i = 0; i < 4; ++i) odd_flag[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(work)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  long long* const red64 = (long long*)red;
  long long mine = 0;
  for (int b = tid; b < A.B.n_seqs; b += NT) {
    const Seq s = load_seq(A.B, b, tile_rows);
    if (s.bad && blockIdx.x == 0) flags[0] = 1;
    mine += tiles_before(s, s.tiles, tile_rows, A.causal) * A.kv_heads;
  }
  long long sum = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  if (lane == 0) red64[warp] = sum;
  __syncthreads();
  long long units = 0;
  for (int w = 0; w < C::WARPS; ++w) units += red64[w];
  const long long ctas = min((long long)gridDim.x, max(1ll, units / MIN_RUN));
  Walker W;
  W.at = W.u1 = 0;                                        // an empty run
  W.b = W.head = W.t = 0;
  if (blockIdx.x < ctas && units > 0) {
    // the items that hold the run's two cuts; the last cut of all is the end
    const long long cut[2] = {cut_at(units, ctas, blockIdx.x), cut_at(units, ctas, blockIdx.x + 1)};
    long long before = 0;
    for (int b0 = 0; b0 < A.B.n_seqs && before <= cut[1]; b0 += NT) {   // their sequences
      const int b = b0 + tid;
      if (A.B.n_seqs > NT) {
        mine = 0;
        if (b < A.B.n_seqs) {
          const Seq s = load_seq(A.B, b, tile_rows);
          mine = tiles_before(s, s.tiles, tile_rows, A.causal) * A.kv_heads;
        }
      }
      long long scan = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(FULL, scan, o);
        if (lane >= o) scan += x;
      }
      __syncthreads();
      if (lane == 31) red64[warp] = scan;
      __syncthreads();
      long long chunk = 0, below = before;
      for (int w = 0; w < C::WARPS; ++w) {
        const long long x = red64[w];
        if (w < warp) below += x;
        chunk += x;
      }
      const long long end = below + scan, begin = end - mine;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (begin <= cut[e] && cut[e] < end) {
          const Spot at = locate(cut[e] - begin, mine / A.kv_heads);
          int* const found = work + 1 + 5 * e;            // sequence, head, tile, unit within the item
          found[0] = b;
          found[1] = at.head;
          red64[20 + e] = at.unit;
        }
      before += chunk;                                    // uniform
    }
    __syncthreads();
    // their tiles: half of the threads look for each
    const int mine_e = tid >= NT / 2;
    if (cut[mine_e] < units) {
      int* const found = work + 1 + 5 * mine_e;
      const Seq s = load_seq(A.B, found[0], tile_rows);
      const long long r = red64[20 + mine_e];
      for (int t = tid - mine_e * (NT / 2); t < s.tiles; t += NT / 2) {
        const long long lo = tiles_before(s, t, tile_rows, A.causal);
        if (lo <= r && r < lo + SETUP + tile_blocks(s, t, tile_rows, A.causal)) {
          found[2] = t;
          found[3] = (int)(r - lo);
        }
      }
    }
    __syncthreads();
    long long to[2], from = 0;
#pragma unroll
    for (int e = 1; e >= 0; --e) {
      const int* const found = work + 1 + 5 * e;
      to[e] = cut[e];
      if (cut[e] == units) continue;
      W.b = found[0]; W.head = found[1]; W.t = found[2];
      W.s = load_seq(A.B, W.b, tile_rows);
      const int in = found[3], size = SETUP + tile_blocks(W.s, W.t, tile_rows, A.causal);
      from = cut[e] - in;
      to[e] = moved_cut(cut[e], in, size);
    }
    W.u0 = to[0];
    W.u1 = to[1];
    W.at = from;
    if (W.u0 < W.u1 && W.u0 > from && to[0] != cut[0]) {  // moved to the end of that item
      W.at = W.u0;
      W.advance(A, tile_rows);
    }
    if (W.u0 >= W.u1) W.at = W.u1;
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = (uint32_t)work[0];
  const bool busy = W.any();
  // tensor memory: scores (and weights over them) at 0 and 128, outputs at 256 and 384
  const uint32_t S_COL = tmem, O_COL = tmem + 256;
  constexpr bool BF = !C::FP8;
  constexpr uint32_t ID_QK = instr_desc(BF, BN, false), ID_PV = instr_desc(BF, D, true);
  Segment g;

  if (warp < C::SOFT_WARP0) {
    if constexpr (C::REGS_SOFT > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_WORK));
    if (busy && warp == 0) {
    // ---------------------------------------------------------------- copies
    const int ps = 1 << A.B.page_shift, ppb = BN >> A.B.page_shift;
    const int nowhere = A.B.num_pages * A.kv_heads * ps;   // a row past the pool: the copy fills zeros
    unsigned nk = 0, nv = 0;                               // blocks issued
    bool ok = true;
    while (ok && W.next(A, tile_rows, g)) {
      const int32_t* const tab = KIND == KIND_PACKED ? nullptr : A.B.table + (size_t)g.b * A.B.max_pages;
      const int used = KIND == KIND_PACKED ? 0 : (g.kv + ps - 1) >> A.B.page_shift;
      auto row_of = [&](int j) {                           // this lane's page of block j
        const int p = j * ppb + lane;
        if (lane >= ppb || p >= used) return nowhere;
        const int page = __ldg(tab + p);
        return (unsigned)page < (unsigned)A.B.num_pages ? (page * A.kv_heads + g.head) * ps : nowhere;
      };
      int row = KIND == KIND_PACKED ? 0 : row_of(g.j0);
      for (int j = g.j0; j < g.j1; ++j) {
        const int cur = row;
        if (KIND != KIND_PACKED && j + 1 < g.j1) row = row_of(j + 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const CUtensorMap* const map = kv ? &map_v : &map_k;
          if constexpr (C::FP8) {
            const unsigned n = nk++, s = n % C::NRAW;
            if (!(ok = bar_wait(raw_empty + 8 * s, ((n / C::NRAW) & 1) ^ 1, flags))) break;
            if (lane == 0) bar_expect(raw_full + 8 * s, C::RAW);
            __syncwarp();
            if (lane < ppb) tma_2d(raw_at + s * C::RAW + lane * ps * D, map, 0, cur, raw_full + 8 * s);
          } else {
            const unsigned n = kv ? nv++ : nk++, ring = kv ? NV : NK, s = n % ring;
            const uint32_t full = (kv ? v_full : k_full) + 8 * s, empty = (kv ? v_empty : k_empty) + 8 * s;
            const uint32_t dst = (kv ? v_at : k_at) + s * C::BUF;
            if (!(ok = bar_wait(empty, ((n / ring) & 1) ^ 1, flags))) break;
            if (lane == 0) bar_expect(full, C::BUF);
            __syncwarp();
            if (KIND == KIND_PACKED) {
              if (lane < C::HALVES) tma_3d(dst + lane * HALF_BYTES, map, lane * 64, g.head, g.row0 - (g.lim0 - 1) + j * BN, full);
            } else if (lane < ppb) {
#pragma unroll
              for (int x = 0; x < C::HALVES; ++x) tma_2d(dst + x * HALF_BYTES + lane * ps * 128, map, x * 64, cur, full);
            }
          }
        }
        if (!ok) break;
      }
    }
    if (!ok) {                                             // let the copies in flight land
      const int rings = C::FP8 ? 1 : 2;
      for (int kv = 0; kv < rings; ++kv) {
        const unsigned n = kv ? nv : nk, ring = C::FP8 ? C::NRAW : kv ? NV : NK;
        for (unsigned i = n > ring ? n - ring : 0; i + 1 < n; ++i) {
          const uint32_t full = (C::FP8 ? raw_full : kv ? v_full : k_full) + 8 * (i % ring);
          for (int it = 0; it < 4096 && !bar_try(full, (i / ring) & 1); ++it) {}
        }
      }
    }
    } else if (busy && warp == 1) {
    // -------------------------------------------------------------- products
      if (elect_one()) {
        unsigned n = 0;                                    // blocks whose scores have been issued
        unsigned m = 0;                                    // blocks whose products with the values have been issued
        unsigned segs = 0;
        bool ok = true;
        auto scores = [&](int tile, uint32_t s_at, unsigned i) {   // S = Q K^T of block i
          const uint64_t kd = smem_desc(k_at + (i % NK) * C::BUF, 16), qd = smem_desc(q_at + tile * C::BUF, 16);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = ((x / 4) * HALF_BYTES + (x % 4) * 32) >> 4;
            mma_ss(s_at, qd + off, kd + off, ID_QK, x > 0);
          }
        };
        auto values = [&](int tile, uint32_t p_at, unsigned i, bool acc) {   // O (+)= P V of block i
          const uint64_t vd = smem_desc(v_at + (i % NV) * C::BUF, HALF_BYTES);
#pragma unroll
          for (int x = 0; x < BN / 16; ++x)
            mma_ts(O_COL + tile * 128, p_at + (x / 2) * 32 + (x % 2) * 8, vd + ((x * 16 * 128) >> 4), ID_PV, acc || x > 0);
        };
        auto wait_k = [&](unsigned i) { return bar_wait1(k_full + 8 * (i % NK), (i / NK) & 1, flags); };
        auto wait_v = [&](unsigned i) { return bar_wait1(v_full + 8 * (i % NV), (i / NV) & 1, flags); };
        while (ok && W.next(A, tile_rows, g)) {
          const int nb = g.j1 - g.j0;
          const bool split = two_parts<KIND, MT>(g);
          if (!(ok = bar_wait1(q_full, segs++ & 1, flags))) break;
          if constexpr (MT == 2) {
            if (!(ok = wait_k(n))) break;
            tc_after();
            for (int tile = 0; tile < 2; ++tile) {
              scores(tile, S_COL + tile * 128, n);
              tc_commit(s_full + 8 * tile);
            }
            tc_commit(k_empty + 8 * (n % NK));
            if (nb == 1) tc_commit(q_empty);
            ++n;
            for (int j = 0; j < nb && ok; ++j, ++m) {
              const bool more = j + 1 < nb;
              if (!(ok = wait_v(m) && (!more || wait_k(n)))) break;
#pragma unroll
              for (int tile = 0; tile < 2; ++tile) {
                if (!(ok = bar_wait1(p_full + 8 * tile, m & 1, flags))) break;
                tc_after();
                values(tile, S_COL + tile * 128, m, j > 0);
                if (split) values(tile, S_COL + tile * 128 + 16, m, true);
                if (more) {
                  scores(tile, S_COL + tile * 128, n);     // in order behind the product that reads its weights
                  tc_commit(s_full + 8 * tile);            // and so a sign that this product is done
                } else {
                  tc_commit(o_done + 8 * tile);
                }
              }
              if (!ok) break;
              if (j + 2 == nb) tc_commit(q_empty);
              tc_commit(v_empty + 8 * (m % NV));
              if (more) {
                tc_commit(k_empty + 8 * (n % NK));
                ++n;
              }
            }
          } else {
            int left = nb;
            auto issue = [&]() {
              if (!wait_k(n)) return false;
              tc_after();
              scores(0, S_COL + (n & 1) * 128, n);
              tc_commit(s_full + 8 * (n & 1));
              tc_commit(k_empty + 8 * (n % NK));
              if (--left == 0) tc_commit(q_empty);
              ++n;
              return true;
            };
            ok = issue() && (nb < 2 || issue());
            for (int j = 0; j < nb && ok; ++j, ++m) {
              if (!(ok = wait_v(m) && bar_wait1(p_full + 8 * (m & 1), (m >> 1) & 1, flags))) break;
              tc_after();
              values(0, S_COL + (m & 1) * 128, m, j > 0);
              if (split) values(0, S_COL + (m & 1) * 128 + 16, m, true);
              tc_commit(o_done + 8);
              if (j + 1 == nb) tc_commit(o_done);
              tc_commit(v_empty + 8 * (m % NV));
              if (j + 2 < nb) ok = issue();
            }
          }
        }
        tc_commit(drain);                                  // products and arrivals in flight end before the CTA does
        for (int it = 0; it < POLLS && !bar_try(drain, 0); ++it) {}
      }
      __syncwarp();
    } else if (busy) {
      // ------------------------------------------------------------ query rows
      // The rows of the next run, as soon as the scores of this one are all done.
      unsigned segs = 0;
      bool ok = true;
      if constexpr (!C::FP8) {
        const int used = A.tile_tokens * A.group;          // rows of a tile: floor(128 / group) tokens, the same box every time
        if (warp == C::Q_WARP0) {
          for (int i = lane; i < MT * C::HALVES * (BM - used) * 8; i += 32) {   // the rest never changes
            const int o = i % ((BM - used) * 8), x = i / ((BM - used) * 8);
            *(uint4*)(gbase + x * HALF_BYTES + used * 128 + o * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async();
          __syncwarp();
          if (elect_one()) {
            while (W.next(A, tile_rows, g)) {
#pragma unroll
              for (int i = 0; i < MT * C::HALVES; ++i)     // to L2 meanwhile
                prefetch_3d(&map_q, (i % C::HALVES) * 64, g.head * A.group, g.row0 + (i / C::HALVES) * A.tile_tokens);
              if (!bar_wait1(q_empty, (segs & 1) ^ 1, flags)) break;
              runs[segs & 3] = g;                          // the softmax is at most two runs behind
              bar_expect(q_full, MT * C::HALVES * used * 128);
#pragma unroll
              for (int i = 0; i < MT * C::HALVES; ++i)
                tma_3d(q_at + i * HALF_BYTES, &map_q, (i % C::HALVES) * 64, g.head * A.group, g.row0 + (i / C::HALVES) * A.tile_tokens, q_full);
              ++segs;
            }
            if (segs > 0 && *(volatile int*)&flags[1])     // given up somewhere: let the last copy land
              for (int it = 0; it < 4096 && !bar_try(q_full, (segs - 1) & 1); ++it) {}
          }
          __syncwarp();
        }
      } else {
        // as f16, normalised by a power of two: 16 bytes a thread, the threads of a row together
        constexpr int LR = D / 8, RP = C::Q_WARPS * 32 / LR;   // threads of a row, rows a pass
        const int t = tid - C::Q_WARP0 * 32, ch = t % LR;
        const unsigned over_group = 65536u / A.group + 1;  // r / group = r * over_group >> 16 for r < 128
        while (ok && W.next(A, tile_rows, g)) {
          const __nv_bfloat16* const rows = A.Q.ptr + g.row0 * A.Q.st + g.head * A.group * A.Q.sh;
          const int n_tok = min(A.tile_tokens, g.ntok);
          for (int r = t; r < BM; r += C::Q_WARPS * 32) {  // to L2 meanwhile
            const int tok = (int)(r * over_group >> 16);
            if (tok < n_tok) {
              const char* const line = (const char*)(rows + tok * A.Q.st + (r - tok * A.group) * A.Q.sh);
#pragma unroll
              for (int o = 0; o < 2 * D; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + o));
            }
          }
          if (!(ok = bar_wait(q_empty, (segs & 1) ^ 1, flags))) break;
          uint8_t* const q = gbase + (ch / 8) * HALF_BYTES;
          if (t == 0) runs[segs & 3] = g;                  // the softmax is at most two runs behind
          constexpr int U = 16;                            // loads of a thread in flight
#pragma unroll 1
          for (int r0 = t / LR; r0 < BM; r0 += U * RP) {
          uint4 xs[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int r = r0 + i * RP, tok = (int)(r * over_group >> 16);
            xs[i] = make_uint4(0, 0, 0, 0);
            if (tok < n_tok) xs[i] = __ldg((const uint4*)(rows + tok * A.Q.st + (r - tok * A.group) * A.Q.sh) + ch);
          }
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int r = r0 + i * RP;
            const uint4 x = xs[i];
            uint32_t w[4] = {x.x, x.y, x.z, x.w}, top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
            // largest magnitude in [1, 2): f16 holds it exactly, and what is 2^-14 of it or more
            const int e = top >= 0x7f80u ? 0 : min(max((int)(top >> 7), 7), 247) - EXP_BIAS;
            const float f = __int_as_float((EXP_BIAS - e) << 23);
            if (ch == 0) q_scale[(segs & 1) * BM + r] = __int_as_float((EXP_BIAS + e) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_f16(bf_lo(w[i]) * f, bf_hi(w[i]) * f);
            *(uint4*)(q + r * 128 + (((ch % 8) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          }
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(q_full);
          ++segs;
        }
      }
    }
  } else if (warp < C::CONV_WARP0) {
    if constexpr (C::REGS_SOFT > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFT));
    if (busy) {
    // --------------------------------------------------------------- softmax
    const int sw = warp - C::SOFT_WARP0, tile = MT == 2 ? sw >> 3 : 0, half = (sw >> 2) & 1;
    const int r = (warp & 3) * 32 + lane;                  // row of the tile, lane of tensor memory
    const uint32_t lane_at = (uint32_t)(warp & 3) << 21;   // 32 lanes a warp, lane number in bits 16..31
    const int pair = BAR_PAIR + tile * 4 + (warp & 3), group_bar = BAR_TILE + tile;
    constexpr int NS = C::SOFT_WARPS * 32;                 // threads of a tile
    const int ts = half * BM + r;                          // among them
    float* const to_pair = swap + (tile * 2 + half) * BM + r;
    const float* const from_pair = swap + (tile * 2 + (half ^ 1)) * BM + r;
    const int tok = r / A.group, head_in = r - tok * A.group;
    const int tk = tile * A.tile_tokens + tok;             // token of the item
    constexpr int DH = D / 2;                              // output columns of this thread
    const uint32_t o_at = O_COL + tile * 128 + lane_at + half * DH;
    unsigned n = 0, segs = 0;                              // blocks and runs done
    bool ok = true;
    do {
      auto wait_scores = [&]() {                           // a wait that gives up takes all to the exits below
        if (ok) ok = MT == 2 ? bar_wait(s_full + 8 * tile, n & 1, flags) : bar_wait(s_full + 8 * (n & 1), (n >> 1) & 1, flags);
        tc_after();
      };
      wait_scores();
      if (group_or(group_bar, NS, !ok)) break;             // all warps of the tile leave, or none
      const Segment& g = runs[segs & 3];                   // announced before its first scores
      const unsigned slot = segs & 3;
      const int j0 = g.j0, j1 = g.j1, lim = A.causal ? g.lim0 + tk : g.kv;
      float c = A.c;
      float M = -INFINITY, l = 0.0f, off = 0.0f;
      const bool split = two_parts<KIND, MT>(g);
      // Some rows do not see all of a block's keys, and a weight of 0 does not clear an infinity or NaN.
      auto care = [&](int j) {
        if (tile == 0 && (j + 1) * BN > (A.causal ? min(g.lim0, g.kv) : g.kv)) {
          // The threads of row r look after value row r: slots past the sequence's end, which may hold
          // anything, become 0, and so does what is not finite, after its key is noted in its column.
          if (ok) ok = bar_wait(v_full + 8 * (n % NV), (n / NV) & 1, flags);
          if (ok) {
            const int key = j * BN + r;
            uint8_t* const line = gbase + (v_at - base) + (n % NV) * C::BUF + r * 128;
            auto piece = [&](int i) {                      // 16-byte piece i of this half row, 8 values
              const int ch = half * (D / 16) + i;
              return (uint4*)(line + (ch / 8) * HALF_BYTES + (((ch % 8) ^ (r & 7)) << 4));
            };
            if (key >= g.kv) {
              if (!C::FP8)
#pragma unroll
                for (int i = 0; i < D / 16; ++i) *piece(i) = make_uint4(0, 0, 0, 0);
            } else {
              constexpr uint32_t EXP = C::FP8 ? 0x7c007c00u : 0x7f807f80u;
              uint32_t found = 0;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint4 w = *piece(i);
                found |= __vcmpeq2(w.x & EXP, EXP) | __vcmpeq2(w.y & EXP, EXP) | __vcmpeq2(w.z & EXP, EXP) | __vcmpeq2(w.w & EXP, EXP);
              }
              if (found) note_odd<D, C::FP8>(A.odd + (blockIdx.x * 4 + slot) * 3 * D, odd_flag + slot, piece, half, key);
            }
          }
          fence_async();
        }
      };
      for (int j = j0; j < j1; ++j, ++n) {
        const unsigned buf = MT == 2 ? tile : n & 1;
        const uint32_t s_at = S_COL + buf * 128 + lane_at + half * 64;
        if (j > j0) wait_scores();
        uint32_t x[64];
        tm_ld32(s_at, x);
        tm_ld32(s_at + 32, x + 32);
        float cb = c, ev = 0.0f;
        if constexpr (C::FP8) {
          const float2 t = info[n % C::INFO];
          if (j == j0) c *= q_scale[(segs & 1) * BM + r];
          cb = fmaxf(c * t.x, 1.17549435e-38f);              // a masked score's -inf times 0 would be NaN
          ev = t.y;
        }
        tc_wait_ld(x);
        tc_wait_ld(x + 32);
        const int rel = lim - j * BN - half * 64;          // keys of this half that the row sees
        if (rel < 64) {
#pragma unroll
          for (int i = 0; i < 64; ++i) x[i] = i < rel ? x[i] : 0xff800000u;
        }
        auto largest = [&]() {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(x[i + e]), __uint_as_float(x[i + 4 + e]));
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        };
        float best = largest(), top = fmaf(best, cb, ev);
        if (group_or(pair, 64, j == j0 || top > M + LAZY || !ok)) {
          // Set or raise the reference, the same for both threads of the row.
          float l_wide = 0.0f, m_wide = -INFINITY;         // sum of weights of a wide block, its reference
          if (C::FP8 && ev == WIDE) {
            // The block's vectors are too far apart for one scale (no score is so low that top misses WIDE):
            // s_ij + e_j, with each vector's own exponents, in place of the scores; the sum is without e_j.
            const float x_all = info[n % C::INFO].x;       // keys' factor if positive, else their own and maybe -256 - the values' exponent
#pragma unroll 1
            for (int i = 0; i < 64; i += 16) {
              uint32_t o[16];
              const int own = scale_bytes(A, g, j * BN + half * 64 + i + (lane & 15));
              tm_ld16(s_at + i, o);
              float m = m_wide;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int w = __shfl_sync(FULL, own, e);
                const float s = __uint_as_float(o[e]) * positive(c * (x_all > 0.0f ? x_all : scale_of(w & 255)));
                const float t = i + e < rel ? s + (x_all < -1.0f ? -256.0f - x_all : (float)value_exponent(w >> 8)) : -INFINITY;
                m = fmaxf(m, t);
                o[e] = __float_as_uint(t);
              }
              l_wide *= m == -INFINITY ? 0.0f : ex2(m_wide - m);
              m_wide = m;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int w = __shfl_sync(FULL, own, e);
                // the difference first: it is what the weight has, however large the scores
                l_wide += ex2(__uint_as_float(o[e]) - (m == -INFINITY ? 0.0f : m) - (x_all < -1.0f ? -256.0f - x_all : (float)value_exponent(w >> 8)));
              }
              tm_st16(s_at + i, o);
            }
            tc_wait_st();
            tm_ld32(s_at, x);
            tm_ld32(s_at + 32, x + 32);
            tc_wait_ld(x);
            tc_wait_ld(x + 32);
            cb = 1.0f;
            top = largest();
          }
          *to_pair = top;
          group_sync(pair, 64);
          const float up = fmaxf(fmaxf(M, top), *from_pair);
          if (j > j0) {
            // The block before must have been added to O; with two tiles its product was issued ahead of
            // these scores.
            if (MT == 1) {
              if (ok) ok = bar_wait(o_done + 8, (n - 1) & 1, flags);
              tc_after();
            }
            const float f = up == -INFINITY ? 1.0f : ex2(M - up);
            if (C::FP8 && f == 0.0f && l > 0.0f) l = scaled<true>(l, M - up);
            else l *= f;
            off *= f;
#pragma unroll 1
            for (int i = 0; i < DH; i += 16) {             // few at a time: the scores hold most registers
              uint32_t o[16];
              tm_ld16(o_at + i, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tm_st16(o_at + i, o);
            }
          }
          M = up;
          if (C::FP8 && ev == WIDE) {
            l += scaled<true>(l_wide, M == -INFINITY ? 0.0f : m_wide - M);
            ev = 0.0f;
          }
          if (group_or(pair, 64, !ok)) { ok = false; break; }   // both have read; both leave, or none
        }
        care(j);
        const float neg = ev - (M == -INFINITY ? 0.0f : M);
        const u64 c2 = pk(cb, cb), n2 = pk(neg, neg);
        u64 acc[2] = {0, 0};
        // exponentials, their sum, and the weights in 16 bits in place of their scores: 32 scores become 16
        // columns of weights and 16 of what rounding left of them
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            upk(fma2(pk(__uint_as_float(x[32 * h + 2 * i]), __uint_as_float(x[32 * h + 2 * i + 1])), c2, n2), a, b);
            a = ex2(a);
            b = ex2(b);
            acc[i & 1] = add2(acc[i & 1], pk(a, b));
            w[i] = C::FP8 ? pack_f16(a, b) : pack_bf16(a, b);
            if (!C::FP8) {
              x[32 * h + 2 * i] = __float_as_uint(a);
              x[32 * h + 2 * i + 1] = __float_as_uint(b);
            }
          }
          if (!C::FP8 && split) {
            // the first part rounded towards 0, the second with 2^-16 of the weight on top: it is positive
            // where the weight is, and an infinite value stays one
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t first = pack_bf16_down(__uint_as_float(x[32 * h + 2 * i]), __uint_as_float(x[32 * h + 2 * i + 1]));
              float a, b;
              upk(fma2(pk(__uint_as_float(x[32 * h + 2 * i]), __uint_as_float(x[32 * h + 2 * i + 1])), pk(ABOVE, ABOVE), pk(-bf_lo(first), -bf_hi(first))), a, b);
              w[i] = first;
              x[32 * h + i] = pack_bf16(a, b);
            }
            tm_st16(s_at + 32 * h + 16, x + 32 * h);
          }
          tm_st16(s_at + 32 * h, w);
        }
        float s0, s1, s2, s3;
        upk(acc[0], s0, s1);
        upk(acc[1], s2, s3);
        const float add = (s0 + s1) + (s2 + s3);
        l += C::FP8 ? add * ex2(-info[n % C::INFO].y) : add;   // 0 where it has been added already
        if (!C::FP8 && !split) {
          // what rounding to bf16 did to the largest of these weights (see the run's result)
          const float p = ex2(fmaf(best, cb, neg));
          off += __bfloat162float(__float2bfloat16(p)) - p;
        }
        tc_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(p_full + 8 * buf);
      }
      // -- the run's result.  Dividing by the sum of the rounded weights would cancel the rounding of a
      // key that dominates its row, where it does not average out; off corrects the sum for the largest
      // weight of each half block, which are the ones that can.
      bool bad = g.bad != 0;
      if (KIND != KIND_PACKED) {                           // pages of this run that do not exist
        const int used = (g.kv + (1 << A.B.page_shift) - 1) >> A.B.page_shift, ppb = BN >> A.B.page_shift;
        for (int p = g.j0 * ppb + ts; p < min(g.j1 * ppb, used); p += NS)
          bad |= (unsigned)__ldg(A.B.table + (size_t)g.b * A.B.max_pages + p) >= (unsigned)A.B.num_pages;
      }
      if (ok) ok = bar_wait(o_done + 8 * tile, segs & 1, flags);
      ++segs;
      if (group_or(group_bar, NS, !ok)) break;             // all warps of the tile leave, or none
      tc_after();
      *to_pair = l;
      bad = group_or(group_bar, NS, bad);
      l += *from_pair;
      group_sync(pair, 64);
      *to_pair = off;
      group_sync(pair, 64);
      off += *from_pair;
      group_sync(pair, 64);
      if (bad) {
        l = off = quiet_nan();
        if (ts == 0) flags[0] = 1;
      }
      const bool have = tok < A.tile_tokens && tk < g.ntok;
      if (g.j0 == 0 && g.j1 == g.nblk) {
        const size_t at = (size_t)(g.row0 + tk) * A.q_heads + g.head * A.group + head_in;
        const float inv = l == 0.0f ? 0.0f : 1.0f / (l + off);
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          uint32_t o[32];
          tm_ld32(o_at + 32 * i, o);
          tc_wait_ld(o);
          if (have) {
            __nv_bfloat16* const dst = A.out + at * D + half * DH + 32 * i;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w[8];
#pragma unroll
              for (int y = 0; y < 8; ++y)
                w[y] = pack_bf16(__uint_as_float(o[16 * e + 2 * y]) * inv, __uint_as_float(o[16 * e + 2 * y + 1]) * inv);
              st_32(dst + 16 * e, w);
            }
          }
        }
        if (*(volatile int*)(odd_flag + slot) && have) {
#pragma unroll 1
          for (int col = half * DH; col < half * DH + DH; ++col) {
            const float x = odd_value<D>(A.odd + (blockIdx.x * 4 + slot) * 3 * D, col, lim);
            if (x != 0.0f) A.out[at * D + col] = __float2bfloat16(x + 0.0f * l);   // NaN rows stay NaN
          }
        }
        if (A.lse && have && half == 0) A.lse[at] = (M + log2f(l)) * LN2_F;
      } else {
        // partial: slot 1 of this CTA holds an item's beginning, slot 0 a later part
        constexpr int PART = part_floats<D>();
        auto part = [&](int cta, int slot) { return A.ws + ((size_t)(cta * 2 + slot) * MT + tile) * PART; };
        float* const dst = part(blockIdx.x, g.j0 == 0 ? 1 : 0);
        if (have && half == 0) {
          __stcg(dst + r, M);
          __stcg(dst + BM + r, l);
          __stcg(dst + 2 * BM + r, off);
        }
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          uint32_t o[32];
          tm_ld32(o_at + 32 * i, o);
          tc_wait_ld(o);
          if (have) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              __stcg((float4*)(dst + 3 * BM) + (half * (DH / 4) + 8 * i + e) * BM + r,
                     make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3])));
          }
        }
        // runs that hold the item: cut x is at units x / ctas, or moved to the end of an item
        if (*(volatile int*)(odd_flag + slot) && have) {
#pragma unroll 1
          for (int col = half * DH; col < half * DH + DH; ++col) {
            const float x = odd_value<D>(A.odd + (blockIdx.x * 4 + slot) * 3 * D, col, lim);
            if (x != 0.0f) __stcg(dst + 3 * BM + (col / 4 * BM + r) * 4 + col % 4, x);
          }
        }
        const int c0 = first_run(g.start - SETUP, units, ctas), c1 = last_run(g.start - SETUP, SETUP + g.nblk, units, ctas);
        __threadfence();
        group_sync(group_bar, NS);
        if (ts == 0) work[14 + tile] = atomicAdd(A.counters + c0 * MT + tile, 1) == c1 - c0;
        group_sync(group_bar, NS);
        if (work[14 + tile]) {                              // the last to finish
          __threadfence();
          if (ts == 0) A.counters[c0 * MT + tile] = 0;
          const int rows = min(A.tile_tokens, max(0, g.ntok - tile * A.tile_tokens)) * A.group;
          if (c1 == c0 + 1) {
            // two partials: every thread merges a half of its row
            if (r < rows) {
              const float *const p = part(c0, 1), *const q = part(c1, 0);
              const float m0 = __ldcg(p + r), m1 = __ldcg(q + r), l0 = __ldcg(p + BM + r), l1 = __ldcg(q + BM + r),
                          d0 = __ldcg(p + 2 * BM + r), d1 = __ldcg(q + 2 * BM + r);
              const float4 *const po = (const float4*)(p + 3 * BM) + half * (DH / 4) * BM + r, *const qo = (const float4*)(q + 3 * BM) + half * (DH / 4) * BM + r;
              const float m_top = fmaxf(m0, m1), ref = m_top == -INFINITY ? 0.0f : m_top;
              const float f0 = ex2(m0 - ref), f1 = ex2(m1 - ref), sum = scaled<C::FP8>(l0, m0 - ref) + scaled<C::FP8>(l1, m1 - ref);
              const float inv = sum == 0.0f ? 0.0f : 1.0f / (sum + f0 * d0 + f1 * d1), w0 = f0 * inv, w1 = f1 * inv;
              const int rt = r / A.group;
              const size_t to = (size_t)(g.row0 + tile * A.tile_tokens + rt) * A.q_heads + g.head * A.group + r - rt * A.group;
#pragma unroll
              for (int i = 0; i < DH / 4; i += 4) {
                float4 x[4], y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  x[e] = __ldcg(po + (i + e) * BM);
                  y[e] = __ldcg(qo + (i + e) * BM);
                }
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  w[2 * e] = pack_bf16(w0 * x[e].x + w1 * y[e].x, w0 * x[e].y + w1 * y[e].y);
                  w[2 * e + 1] = pack_bf16(w0 * x[e].z + w1 * y[e].z, w0 * x[e].w + w1 * y[e].w);
                }
                st_32(A.out + to * D + half * DH + 4 * i, w);
              }
              if (A.lse && half == 0) A.lse[to] = (m_top + log2f(sum)) * LN2_F;
            }
          } else {
          // weight of every partial, left where its reference was
          if (ts < rows) {
            float m_top = -INFINITY, sum = 0.0f, fix = 0.0f;
            bool nan = false;
#pragma unroll 4
            for (int x = c0; x <= c1; ++x) {
              const float m = __ldcg(part(x, x == c0) + ts);
              nan |= isnan(m);
              m_top = fmaxf(m_top, m);
            }
            const float ref = m_top == -INFINITY ? 0.0f : m_top;
#pragma unroll 2
            for (int x = c0; x <= c1; ++x) {
              float* const p = part(x, x == c0);
              const float x2 = __ldcg(p + ts) - ref;
              sum += scaled<C::FP8>(__ldcg(p + BM + ts), x2);
              fix += ex2(x2) * __ldcg(p + 2 * BM + ts);
            }
            const float inv = nan ? quiet_nan() : sum == 0.0f ? 0.0f : 1.0f / (sum + fix);
#pragma unroll 4
            for (int x = c0; x <= c1; ++x) {
              float* const p = part(x, x == c0);
              __stcg(p + ts, ex2(__ldcg(p + ts) - ref) * inv);
            }
            const int rt = ts / A.group;
            if (A.lse)
              A.lse[(size_t)(g.row0 + tile * A.tile_tokens + rt) * A.q_heads + g.head * A.group + ts - rt * A.group] =
                  nan ? quiet_nan() : (m_top + log2f(sum)) * LN2_F;
          }
          group_sync(group_bar, NS);
          constexpr int U = 4;                             // quadruples of a thread in flight, of two partials
          const int all = rows * (D / 4);
          for (int i0 = ts; i0 < all; i0 += NS * U) {
            float4 o[U];
            int at[U], rr[U];
#pragma unroll
            for (int q = 0; q < U; ++q) {
              const int i = min(i0 + q * NS, all - 1), d4 = i / rows;
              rr[q] = i - d4 * rows;
              at[q] = d4 * BM + rr[q];
              o[q] = make_float4(0, 0, 0, 0);
            }
#pragma unroll 2
            for (int x = c0; x <= c1; ++x) {
              const float* const p = part(x, x == c0);
              float f[U];
              float4 y[U];
#pragma unroll
              for (int q = 0; q < U; ++q) {
                f[q] = __ldcg(p + rr[q]);
                y[q] = __ldcg((const float4*)(p + 3 * BM) + at[q]);
              }
#pragma unroll
              for (int q = 0; q < U; ++q) {
                o[q].x += f[q] * y[q].x; o[q].y += f[q] * y[q].y; o[q].z += f[q] * y[q].z; o[q].w += f[q] * y[q].w;
              }
            }
#pragma unroll
            for (int q = 0; q < U; ++q) {
              if (i0 + q * NS >= all) break;
              const int rt = rr[q] / A.group;
              const size_t to = (size_t)(g.row0 + tile * A.tile_tokens + rt) * A.q_heads + g.head * A.group + rr[q] - rt * A.group;
              *(uint2*)(A.out + to * D + 4 * (at[q] / BM)) = make_uint2(pack_bf16(o[q].x, o[q].y), pack_bf16(o[q].z, o[q].w));
            }
          }
          }
        }
      }
      const unsigned past = (slot + 2) & 3;                // the run before the last: both tiles are past it
      if (tile == 0 && *(volatile int*)(odd_flag + past)) {
        for (int i = ts; i < 3 * D; i += NS) __stcg(A.odd + (blockIdx.x * 4 + past) * 3 * D + i, ODD_NONE);
        __threadfence();
        group_sync(group_bar, NS);
        if (ts == 0) *(volatile int*)(odd_flag + past) = 0;
      }
      tc_before();
      if (!g.more) break;
    } while (true);
    }
  } else if constexpr (C::FP8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONV));
    if (busy) {
    // ---------------------------------------------- e4m3 codes to f16 blocks
    // A code is exact in f16, and so is its product with 2^(e_j - e), e the
    // largest exponent among the block's vectors, down to e - SPREAD.  The softmax
    // applies e once per block: key scores times 2^e, and for the values the
    // reference M covers s_ij + e, so a weight times a block value stays within
    // range whatever the vectors' sizes.  e of the values is kept within 2^64 of
    // the run's largest so that the weights do not vanish.  Where a vector is
    // smaller than that (a token of another size, which some rows may not even see)
    // the codes stay as they are and the softmax applies each vector's own
    // exponent, in the branch that raises the reference so that ordinary blocks pay
    // next to nothing.  Such a block takes five times as long (64 sequences of 16
    // over 1000-16000, all of them such: 1,560 instead of 297 us).  Vectors of scale
    // BYTE_ZERO and less, which zeros have, do not count for that.
    // Four warps convert the keys, four the values, a thread a vector.  Raw lines
    // are swizzled like the f16 ones, so that eight threads of eight keys reach
    // eight different 16-byte columns.
    const int key = tid & 127, kv = (warp - C::CONV_WARP0) >> 2, bar_id = BAR_CONV + kv;
    static_assert(C::CONV_WARPS == 8 && C::CONV_WARP0 % 4 == 0, "one converting thread per key and per value");
    int2* const wmax = (int2*)red + kv * 8;                // [2][4]: maxima per quarter of the keys
    const uint32_t full0 = kv ? v_full : k_full, empty0 = kv ? v_empty : k_empty;
    const unsigned ring = kv ? NV : NK;
    uint8_t* const out0 = gbase + ((kv ? v_at : k_at) - base) + key * 128;
    const uint8_t* const raw0 = gbase + (raw_at - base) + key * D;
    unsigned n = 0;
    bool ok = true, stop = false;
    while (!stop && W.next(A, tile_rows, g)) {
      const int32_t* const tab = A.B.table + (size_t)g.b * A.B.max_pages;
      int run = EV_MIN;
      // page of this thread's key in block j (loaded a block before its scale bytes, those a block before their use)
      auto page_of = [&](int j) {
        const int p = j * BN + key;
        return p < g.kv ? __ldg(tab + (p >> A.B.page_shift)) : -1;
      };
      auto load_bytes = [&](int j, int page) {             // scale bytes of this thread's key and value (0: none)
        if ((unsigned)page >= (unsigned)A.B.num_pages) return make_int2(0, 0);
        const size_t at = ((size_t)(page * A.kv_heads + g.head) << A.B.page_shift) + ((j * BN + key) & ((1 << A.B.page_shift) - 1));
        return make_int2(kv ? 0 : __ldg(A.ks + at), __ldg(A.vs + at));
      };
      // largest byte of a warp's vectors, and in the upper half 255 - the smallest that counts
      auto extremes = [&](int byte) {
        const int most = __reduce_max_sync(FULL, byte == BYTE_NAN ? 0 : byte);
        return most | __reduce_max_sync(FULL, byte == BYTE_NAN || byte <= BYTE_ZERO ? 0 : 255 - byte) << 16;
      };
      int2 nxt = load_bytes(g.j0, page_of(g.j0));
      int page = page_of(g.j0 + 1);
      for (int j = g.j0; j < g.j1; ++j, ++n) {
        const int2 cur = nxt;
        const int ka = kv ? 0 : extremes(cur.x), va = extremes(cur.y);
        int2* const wm = wmax + (n & 1) * 4;
        if (lane == 0) wm[warp & 3] = make_int2(ka, va);
        if ((stop = group_or(bar_id, BN, !ok))) break;     // all four warps leave, or none
        nxt = load_bytes(j + 1, page);
        page = page_of(j + 2);
        const unsigned kx = __vmaxu2(__vmaxu2(wm[0].x, wm[1].x), __vmaxu2(wm[2].x, wm[3].x));
        const unsigned vx = __vmaxu2(__vmaxu2(wm[0].y, wm[1].y), __vmaxu2(wm[2].y, wm[3].y));
        const int ek = max((int)(kx & 0xffff) - EXP_BIAS, EXP_MIN);
        const int ev = min(max((int)(vx & 0xffff) - EXP_BIAS, max(run - 64, EV_MIN)), EV_MAX);
        run = max(run, ev);
        const bool wide_k = ek - (255 - (int)(kx >> 16) - EXP_BIAS) > SPREAD, wide_v = ev - (255 - (int)(vx >> 16) - EXP_BIAS) > SPREAD;
        const bool valid = key < g.kv - j * BN;            // slots past the end may hold anything
        const int by = kv ? cur.y : cur.x;
        int d = by - EXP_BIAS - (kv ? ev : ek);            // <= 0 (1 above EV_MAX)
        if (kv ? wide_v : wide_k) d = kv ? by - EXP_BIAS - value_exponent(by) : 0;
        const uint32_t f1 = by == BYTE_NAN ? 0x7e00u : (uint32_t)max(15 + d, 0) << 10, f = f1 | (f1 << 16);   // NaN whatever the codes
        const unsigned raw = 2 * n + kv, rs = raw % C::NRAW, bs = n % ring;
        ok = bar_wait(raw_full + 8 * rs, (raw / C::NRAW) & 1, flags) && bar_wait(empty0 + 8 * bs, ((n / ring) & 1) ^ 1, flags);
        const uint8_t* const src = raw0 + rs * C::RAW;
        uint8_t* const dst = out0 + bs * C::BUF;
        if (ok) {
#pragma unroll 1
          for (int h = 0; h < D / 64; ++h) {               // 64 codes: one line of the f16 block
            uint4 xs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int ch = 4 * h + i;
              xs[i] = *(const uint4*)(src + ((D == 128 ? ch ^ (key & 7) : ch ^ ((key >> 1) & 3)) << 4));
              if (!valid) xs[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w[4] = {xs[i].x, xs[i].y, xs[i].z, xs[i].w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t hcode = e4m3_to_f16x2((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
                asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[e]) : "r"(hcode), "r"(f));
              }
              uint8_t* const line = dst + h * HALF_BYTES;
              *(uint4*)(line + (((2 * i) ^ (key & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
              *(uint4*)(line + (((2 * i + 1) ^ (key & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        // both for the softmax, ahead of the keys and so of the block's scores
        if (kv == 0 && key == 0) info[n % C::INFO] = make_float2(!wide_k ? __int_as_float((ek + EXP_BIAS) << 23) : wide_v ? -1.0f : -256.0f - ev, wide_k || wide_v ? WIDE : (float)ev);
        fence_async();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(raw_empty + 8 * rs);
          bar_arrive(full0 + 8 * bs);
        }
      }
    }
  }
  }
  tc_before();
  __syncthreads();
  for (int i = tid; i < 4 * 3 * D; i += NT)                // the last runs' notes
    if (odd_flag[i / (3 * D)]) A.odd[blockIdx.x * 4 * 3 * D + i] = ODD_NONE;
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

}  // namespace
