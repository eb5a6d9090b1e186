// Attention over a 4-bit cache for few rows: up to 16 rows (new tokens times the
// heads of a group) of a sequence and key-value head.
//
// With few rows nothing can take long but the reading of keys and values, 73
// bytes a vector of 128, so codes go from shared memory to the operand registers
// of warp-wide matrix instructions without being written anywhere as 16 bits.
// (The tensor-memory products of attn_tile.cuh have 128 rows whether they are
// used or not, and their operands pass shared memory three times as f16.)  The
// products are taken with keys and columns of values on the long side,
//
//     S^T [16 keys x 8 rows] = K [16 x D] Q^T [D x 8],
//     O^T [16 columns x 8 rows] += V^T [16 x 16 keys] P^T [16 keys x 8 rows],
//
// so 8 rows cost half of what the 16-row form would.  Within a product the order
// of the summed dimension is free, as long as both operands agree: a thread takes
// 32 neighbouring elements of its keys (D = 128), which are one 16-byte load and
// two scales, and 16 columns of four values, which share a scale each.  Scores
// leave the product with their keys along the registers' rows and turn into the
// weights' operand by a transposition of 8 x 8 (movmatrix).
//
// A warp takes slices of 32 keys in turn and keeps references, sums and outputs
// of its own; they meet once at the end of a run.  There are two references for
// a row: M of its scores (the running maximum, raised when a score passes it by
// LAZY), for the sum l, and N of scores plus the exponents of the values' vectors,
// for the output, since a weight and its vector's power of two go into the
// product as one f16 factor.  So vectors may differ in size as they like.
//
// Work is cut into runs as in attn_tile.cuh (the same schedule, with up to 16
// rows to a tile).  One warp announces the runs and lays out query rows as f16, a
// run ahead; the others, 15 or 11 for 8 or 16 rows, are as above.  Each copies its
// own slices, two or more ahead, into places of its own, so that none waits for
// another but at a run's end, where it has the next run's first slices on the way
// already.  (Three copying warps for all, in turns: a warp waited for its slice for
// 37% of the time, behind those that were late.)
//
// What bounds it, measured on GB300: 64 single tokens over 1000-16000, 64 query and
// 8 key-value heads of 128, take 174 us, 3.7 TB/s, where copies alone took 118.
// A slice is some 780 instructions, 128 each of them conversions of two codes and
// products of two elements with a scale, both at half rate; an SM issues half of
// its slots, with four warps to a quarter whose chains of products and conversions
// do not always cover one another.  16 rows: 225 us for 2 tokens each.  Rates that
// decided the form: f16 products of warps 1,024 multiply-adds a clock and SM, a
// quarter of the tensor-memory ones; conversions of two codes 64 lanes a clock.
// Small calls are a chain of latencies: 4 tokens over up to 700 take 12.1 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "attn_tile.cuh"

namespace {

template <int D, int NTILES>
struct Few {
  static constexpr int R = 8 * NTILES;                     // rows
  static constexpr int CONSUMERS = NTILES == 1 ? 15 : 11;        // and one for queries: 4 or 3 warps to a quarter of the registers
  static constexpr int WARPS = CONSUMERS + 1, THREADS = WARPS * 32, CT = CONSUMERS * 32;   // the last one: query rows
  static constexpr int SLICE = 32;                         // keys
  static constexpr int LINE = D / 2, NSC = D / 16;         // bytes of a vector's codes, its scales
  static constexpr int K_AT = 0, V_AT = SLICE * LINE, KB_AT = 2 * SLICE * LINE, VB_AT = KB_AT + SLICE * NSC, KS_AT = VB_AT + SLICE * NSC, VS_AT = KS_AT + SLICE;
  static constexpr int STAGE = VS_AT + SLICE;
  static constexpr int VEC = 2 * (LINE + NSC + 1);         // bytes of a cached token of a head
  static constexpr int DEPTH = D == 64 ? 4 : NTILES == 1 ? 2 : 3;   // stages of a warp
  static constexpr int NS = CONSUMERS * DEPTH;
  static constexpr int QBYTES = R * D * 2;
  static constexpr int CJ = D / 32;                        // words of codes of a key that a thread takes
  static constexpr int MT = D / 16;                        // 16-column tiles of the output
  static constexpr int CM = NTILES == 1 ? MT : 4;         // of them merged at a time
  static_assert(MT % CM == 0 && CM > 0, "merge passes");
  static constexpr int MERGE = CONSUMERS * CM * NTILES * 512;
  static constexpr int SMALL = 384;                        // barriers and bookkeeping
  static constexpr int OUT_AT = SMALL, OUT = R * D * 4;
  static constexpr int STAT_AT = OUT_AT + OUT, STAT = CONSUMERS * R * 16;      // (M, N, l, -) of every warp and row
  static constexpr int ROW_AT = STAT_AT + STAT, ROW = R * 16;                  // of the run
  static constexpr int Q_AT = ROW_AT + ROW, QS_AT = Q_AT + 2 * QBYTES;
  static constexpr int MERGE_AT = QS_AT + 2 * R * 4, RING_AT = (MERGE_AT + (MERGE > 152 * R * 4 ? MERGE : 152 * R * 4) + 127) / 128 * 128;
  static constexpr int SMEM = RING_AT + NS * STAGE;
  static_assert(SMEM <= SMEM_LIMIT, "shared memory");
  static_assert(STAGE % 16 == 0 && Q_AT % 16 == 0 && MERGE_AT % 16 == 0, "alignment");
};
constexpr int MAX_CTAS = 152;                              // weights of partials that fit the merge area

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// A reference before there is a score: -infinity would make NaN of differences.  Scores stay above -2^30, and 2 to the
// difference of a score that is not seen, or of two of these, is 0 and 1.
constexpr float NOTHING = -1e30f;
__device__ __forceinline__ float log_sum(const float4& t) { return (t.z == 0.0f ? -INFINITY : t.x + log2f(t.z)) * LN2_F; }
// eight e2m1 codes to f16 values
__device__ __forceinline__ void e2m1_raw(uint32_t c, uint32_t* y) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}" : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]) : "r"(c));
}
// 16 columns of a row: 2^(N - M) O / l, the power of two in two steps that stay within range
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const float* o, float M, float N, float l) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l, h = ex2(0.5f * (N - M));
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(o[2 * i] * inv * h * h, o[2 * i + 1] * inv * h * h);
  st_32(dst, w);
}

enum { BAR_ALL = 1 };              // the consuming warps

template <int D, int NTILES>
__global__ void __launch_bounds__(Few<D, NTILES>::THREADS, 1) sa_few_kernel(const __grid_constant__ AttnParams A, const uint8_t* kc, const uint8_t* vc) {
  using C = Few<D, NTILES>;
  constexpr int R = C::R, MT = C::MT, CT = C::CT;
  extern __shared__ __align__(1024) uint8_t mem[];
  const uint32_t base = saddr(mem), q_full = base, q_empty = q_full + 16;
  int* const work = (int*)(mem + 32);                     // plan [16]
  Segment* const runs = (Segment*)(mem + 96);             // as the query warp announces them [4]
  static_assert(96 + 4 * 64 <= C::SMALL && sizeof(Segment) <= 64, "bookkeeping");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* const flags = A.B.flags;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) { bar_init(q_full + 8 * i, 1); bar_init(q_empty + 8 * i, 1); }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  long long units, ctas;
  Walker W = plan_run<C::THREADS, true>(A, A.tile_tokens, (long long*)(mem + C::OUT_AT), work, units, ctas);
  __syncthreads();
  const bool busy = W.any();
  const int shift = A.B.page_shift, ps = 1 << shift;
  // slices of a run of an item's blocks
  auto slices = [&](const Segment& g) { return max(0, (min(g.kv, g.j1 * BN) - g.j0 * BN + C::SLICE - 1) / C::SLICE); };

  if (warp == C::CONSUMERS) {
    if (busy) {
      // ---------------------------------------------------------- query rows
      // As f16, normalised by a power of two, 8 elements a lane.  Element 8 ch + .. of row r goes where the product's
      // thread finds its D / 4 elements in 16-byte pieces, the pieces of a warp next to one another.
      constexpr int LR = D / 8, RP = 32 / LR, CJ = C::CJ;
      const int ch = lane % LR;
      const unsigned over_group = 65536u / A.group + 1;
      unsigned segs = 0;
      Segment g;
      while (W.next(A, A.tile_tokens, g)) {
        const unsigned buf = segs & 1;
        const __nv_bfloat16* const rows = A.Q.ptr + g.row0 * A.Q.st + g.head * A.group * A.Q.sh;
        const int n_tok = min(A.tile_tokens, g.ntok);
        constexpr int U = R / RP < 8 ? R / RP : 8;
        if (!bar_wait(q_empty + 8 * buf, ((segs >> 1) & 1) ^ 1, flags)) break;
        if (lane == 0) runs[segs & 3] = g;
#pragma unroll 1
        for (int r0 = lane / LR; r0 < R; r0 += U * RP) {
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
            uint32_t w[4] = {xs[i].x, xs[i].y, xs[i].z, xs[i].w}, top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
            const int e = top >= 0x7f80u ? 0 : min(max((int)(top >> 7), 7), 247) - EXP_BIAS;
            const float f = __int_as_float((EXP_BIAS - e) << 23);
            if (ch == 0) ((float*)(mem + C::QS_AT))[buf * R + r] = __int_as_float((EXP_BIAS + e) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_f16(bf_lo(w[j]) * f, bf_hi(w[j]) * f);
            *(uint4*)(mem + C::Q_AT + buf * C::QBYTES + (((ch % CJ) * R + r) * 4 + ch / CJ) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(q_full + 8 * buf);
        ++segs;
      }
    }
  } else {
    if (busy) {
      // ----------------------------------------------------- scores to outputs
      const int w = warp, ct = tid, gq = lane >> 2, t4 = lane & 3;   // row group and place in it of operand fragments
      constexpr int DV = D / 8;                            // columns of a value that a thread takes
      float4* const stat = (float4*)(mem + C::STAT_AT);    // [warp][row]
      float4* const row_stat = (float4*)(mem + C::ROW_AT); // [row]
      float* const merge = (float*)(mem + C::MERGE_AT);
      float* const res = (float*)(mem + C::OUT_AT);        // [row][D]
      unsigned n = 0, segs = 0;                            // slices of this warp, runs
      bool ok = true;
      // ---- copies.  The cursor: the run it is in, its next slice there, what has been asked for and not used, and the
      // page of the slice's first and second 16 keys (in lanes 0 and 1), loaded a slice ahead
      unsigned at_run = 0, asked = 0, pending = 0;
      int at = 0, at_count = 0, at_pos0 = 0, at_used = 0, at_head = 0, at_page = 0;
      const int32_t* at_tab = nullptr;
      constexpr int SC = C::NSC;                           // 16-byte pieces of 16 keys' scales
      const int sl = lane & (4 * SC - 1), sl_half = sl / SC & 1;               // this lane's piece of the scales
      const uint8_t *const kc_lane = kc + lane * 16, *const vc_lane = vc + lane * 16;
      const uint8_t* const sc_src = (sl < 2 * SC ? A.kb : A.vb) + (sl & (SC - 1)) * 16;
      const int sc_at = (sl < 2 * SC ? C::KB_AT : C::VB_AT) + sl % (2 * SC) * 16;
      const uint8_t* const ex_src = lane & 2 ? A.vs : A.ks;
      const int ex_at = (lane & 2 ? C::VS_AT : C::KS_AT) + (lane & 1) * 16;
      const uint32_t ring = base + C::RING_AT + w * C::DEPTH * C::STAGE;
      auto look_up = [&]() {                               // numbers of the pages of slice `at`; 0 where there is none: such a
        const int x = ((at_pos0 + at * C::SLICE) >> shift) + (ps == 16 ? lane & 1 : 0);   // page's slots are not used, or their rows NaN
        at_page = x < at_used && at < at_count ? __ldg(at_tab + x) : 0;
      };
      auto enter = [&](unsigned run) {                     // an announced run
        const Segment& g = runs[run & 3];
        at_run = run;
        at = w;
        at_count = slices(g);
        at_pos0 = g.j0 * BN;
        at_used = (g.kv + ps - 1) >> shift;
        at_head = g.head;
        at_tab = A.B.table + (size_t)g.b * A.B.max_pages;
        look_up();
      };
      auto ask = [&]() {                                   // asks for slice `at`
        const int page = (unsigned)at_page < (unsigned)A.B.num_pages ? at_page : 0, pos = at_pos0 + at * C::SLICE;
        const int page0 = __shfl_sync(FULL, page, 0), page1 = __shfl_sync(FULL, page, 1);
        at += C::CONSUMERS;
        look_up();
        // vectors of a pool are counted in 31 bits
        const unsigned v0 = ((unsigned)(page0 * A.kv_heads + at_head) << shift) + (pos & (ps - 1));
        const unsigned v1 = ps == 16 ? (unsigned)(page1 * A.kv_heads + at_head) << shift : v0 + 16;
        const uint32_t dst = ring + asked % C::DEPTH * C::STAGE, to = dst + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *const k = kc_lane + (size_t)(h ? v1 : v0) * C::LINE, *const v = vc_lane + (size_t)(h ? v1 : v0) * C::LINE;
#pragma unroll
          for (int x = 0; x < C::LINE / 32; ++x) {
            async16(to + C::K_AT + (h * (C::LINE / 32) + x) * 512, k + x * 512);
            async16(to + C::V_AT + (h * (C::LINE / 32) + x) * 512, v + x * 512);
          }
        }
        if (lane < 4 * SC) async16(dst + sc_at, sc_src + (size_t)(sl_half ? v1 : v0) * SC);
        if (lane < 4) async16(dst + ex_at, ex_src + (lane & 1 ? v1 : v0));
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++asked;
        ++pending;
      };
      do {
        const unsigned buf = segs & 1;
        ok = bar_wait(q_full + 8 * buf, (segs >> 1) & 1, flags);
        if (group_or(BAR_ALL, CT, !ok)) break;             // all of them leave, or none
        const Segment& g = runs[segs & 3];
        if (segs == 0 || at_run != segs) enter(segs);
        while (pending < C::DEPTH && at < at_count) ask();
        const bool more = g.more != 0;
        const int count = slices(g), kv = g.kv, pos0 = g.j0 * BN, lim0 = g.lim0;
        const int all_see = A.causal ? min(g.lim0, kv) : kv;       // keys that every row sees
        // Factors of scores stay far from the ends of their range.  (Not so with a row of zeros, as rows that pad a tile
        // are: 0.7% of the time of 256 single tokens with 4 of 8 rows used.)
        bool small_q = true;
        float cq[NTILES][2], M[NTILES][2], N[NTILES][2], l[NTILES][2], o[MT][NTILES][4];
#pragma unroll
        for (int nt = 0; nt < NTILES; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            cq[nt][c] = A.c * ((float*)(mem + C::QS_AT))[buf * R + nt * 8 + 2 * t4 + c];
            small_q &= cq[nt][c] > 1e-18f && cq[nt][c] < 1e18f;
            M[nt][c] = N[nt][c] = NOTHING;
            l[nt][c] = 0.0f;
#pragma unroll
            for (int m = 0; m < MT; ++m) o[m][nt][c] = o[m][nt][c + 2] = 0.0f;
          }
        small_q = __all_sync(FULL, small_q);
        for (int i = w; i < count; i += C::CONSUMERS, ++n) {
          if (pending == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");           // the oldest has to be there
          else if (pending == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
          else if (pending == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
          else asm volatile("cp.async.wait_group 3;" ::: "memory");
          __syncwarp();
          uint8_t* const st = mem + C::RING_AT + (w * C::DEPTH + n % C::DEPTH) * C::STAGE;
          const int pos = pos0 + i * C::SLICE;
          const bool edge = pos + C::SLICE > all_see;
          // ---- what is rare is put right in the slice itself, a lane a key: slots past the end, which may hold
          // anything, become 0; keys of NaN get scales of NaN; and where some rows do not see all keys, values of
          // NaN become 0 and are remembered (bit x: the 16 columns of scale x), for a weight of 0 would not hide them.
          uint32_t nan_blocks = 0;
          bool plain = small_q;
          {
            const int kb = st[C::KS_AT + lane], vb = st[C::VS_AT + lane];
            if (edge || __any_sync(FULL, (unsigned)(kb - 64) > 126 || vb == BYTE_NAN)) {
              plain = false;
              const bool valid = pos + lane < kv;
              uint8_t *const ks = st + C::KB_AT + lane * C::NSC, *const vs = st + C::VB_AT + lane * C::NSC;
#pragma unroll 1
              for (int x = 0; x < C::NSC; ++x) {
                if (kb == BYTE_NAN) ks[x] = 0x7f;
                if (vb == BYTE_NAN) vs[x] = 0x7f;
                if (!valid) ks[x] = vs[x] = 0;
                if (edge && (vs[x] & 0x7f) == 0x7f) {
                  nan_blocks |= 1u << x;
                  vs[x] = 0;
                }
              }
              if (kb == BYTE_NAN || !valid) st[C::KS_AT + lane] = EXP_BIAS;
              if (vb == BYTE_NAN || !valid) st[C::VS_AT + lane] = EXP_BIAS;
              __syncwarp();
            }
          }
          // ---- scores
          float S[2][NTILES][4], ev[2][2], kx[2][2];
          {
            uint32_t code[2][2][C::CJ], sc[2][2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = 16 * m + 8 * h + gq;
                uint32_t y;
                if constexpr (D == 128) {
                  const uint4 x = *(const uint4*)(st + C::K_AT + key * C::LINE + t4 * 16);
                  code[m][h][0] = x.x; code[m][h][1] = x.y; code[m][h][2] = x.z; code[m][h][3] = x.w;
                  y = e4m3_to_f16x2(*(const uint16_t*)(st + C::KB_AT + key * C::NSC + t4 * 2));
                  sc[m][h][1] = __byte_perm(y, y, 0x3232);
                } else {
                  const uint2 x = *(const uint2*)(st + C::K_AT + key * C::LINE + t4 * 8);
                  code[m][h][0] = x.x; code[m][h][1] = x.y;
                  y = e4m3_to_f16x2(st[C::KB_AT + key * C::NSC + t4]);
                }
                sc[m][h][0] = __byte_perm(y, y, 0x1010);
                kx[m][h] = __int_as_float(st[C::KS_AT + key] << 23);
                ev[m][h] = __int_as_float(0x4b000000 | st[C::VS_AT + key]) - (8388608.0f + EXP_BIAS);
              }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nt = 0; nt < NTILES; ++nt) S[m][nt][0] = S[m][nt][1] = S[m][nt][2] = S[m][nt][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < C::CJ; ++j) {
              uint32_t a[2][2][4];
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) e2m1_to_f16(code[m][h][j], sc[m][h][D == 128 ? j / 2 : 0], a[m][h]);
#pragma unroll
              for (int nt = 0; nt < NTILES; ++nt) {
                const uint4 q = *(const uint4*)(mem + C::Q_AT + buf * C::QBYTES + ((j * R + nt * 8 + gq) * 4 + t4) * 16);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  mma_f16(S[m][nt], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], q.x, q.y);
                  mma_f16(S[m][nt], a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], q.z, q.w);
                }
              }
            }
          }
          // ---- scores in units of log 2, those that are not seen -inf; whether one passes its reference
          bool raise = false;
#pragma unroll
          for (int nt = 0; nt < NTILES; ++nt) {
            if (plain) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < 4; ++c) S[m][nt][c] *= cq[nt][c & 1] * kx[m][c >> 1];
            } else {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < 4; ++c) S[m][nt][c] *= positive(cq[nt][c & 1] * kx[m][c >> 1]);
            }
            if (edge) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int row = nt * 8 + 2 * t4 + c, lim = (A.causal ? min(kv, lim0 + row / A.group) : kv) - pos - gq;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                  for (int h = 0; h < 2; ++h) S[m][nt][2 * h + c] = 16 * m + 8 * h < lim ? S[m][nt][2 * h + c] : -INFINITY;
              }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float a = fmaxf(max3(S[0][nt][c], S[0][nt][c + 2], S[1][nt][c]), S[1][nt][c + 2]);
              const float b = fmaxf(max3(S[0][nt][c] + ev[0][0], S[0][nt][c + 2] + ev[0][1], S[1][nt][c] + ev[1][0]), S[1][nt][c + 2] + ev[1][1]);
              raise |= a > M[nt][c] + LAZY || b > N[nt][c] + LAZY;
            }
          }
          if (__any_sync(FULL, raise)) {
#pragma unroll
            for (int nt = 0; nt < NTILES; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float a = M[nt][c], b = N[nt][c];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    a = fmaxf(a, S[m][nt][2 * h + c]);
                    b = fmaxf(b, S[m][nt][2 * h + c] + ev[m][h]);
                  }
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                  a = fmaxf(a, __shfl_xor_sync(FULL, a, x));
                  b = fmaxf(b, __shfl_xor_sync(FULL, b, x));
                }
                l[nt][c] *= ex2(M[nt][c] - a);
                const float f = ex2(N[nt][c] - b);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                  o[m][nt][c] *= f;
                  o[m][nt][c + 2] *= f;
                }
                M[nt][c] = a;
                N[nt][c] = b;
              }
          }
          // ---- weights: their sum, and in f16 with the values' powers of two, keys along the summed dimension.
          // In odd places of a row group the two keys of a pair change places (see the values).
          uint32_t p[2][NTILES][2];
          const uint32_t order = t4 & 1 ? 0x1032 : 0x3210;
#pragma unroll
          for (int nt = 0; nt < NTILES; ++nt) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float x0 = S[m][nt][2 * h], x1 = S[m][nt][2 * h + 1];
                l[nt][0] += ex2(x0 - M[nt][0]);
                l[nt][1] += ex2(x1 - M[nt][1]);
                const uint32_t y = transpose8(pack_f16(ex2(x0 + (ev[m][h] - N[nt][0])), ex2(x1 + (ev[m][h] - N[nt][1]))));
                p[m][nt][h] = __byte_perm(y, y, order);
              }
          }
          // ---- outputs
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            // This thread's four keys: 2 t4, 2 t4 + 1, and those 8 further, the odd one first in odd places, so that
            // two lines of keys share the banks and not four; its columns: DV from DV * gq on.
            uint32_t code[4][DV / 8], sc[4];
            const int key0 = 16 * m + 2 * t4;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = key0 + ((x ^ t4) & 1) + 4 * (x & 2);
              const uint8_t* const src = st + C::V_AT + key * C::LINE + gq * (DV / 2);
              if constexpr (D == 128) {
                const uint2 v = *(const uint2*)src;
                code[x][0] = v.x;
                code[x][1] = v.y;
              } else {
                code[x][0] = *(const uint32_t*)src;
              }
              sc[x] = st[C::VB_AT + key * C::NSC + (D == 128 ? gq : gq >> 1)];
            }
            const uint32_t s01 = e4m3_to_f16x2((uint16_t)(sc[0] | sc[1] << 8)), s23 = e4m3_to_f16x2((uint16_t)(sc[2] | sc[3] << 8));
#pragma unroll
            for (int y = 0; y < DV / 8; ++y) {
              uint32_t v[4][4];
#pragma unroll
              for (int x = 0; x < 4; ++x) e2m1_raw(code[x][y], v[x]);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const uint32_t a0 = mul2(__byte_perm(v[0][b], v[1][b], 0x5410), s01), a1 = mul2(__byte_perm(v[0][b], v[1][b], 0x7632), s01);
                const uint32_t a2 = mul2(__byte_perm(v[2][b], v[3][b], 0x5410), s23), a3 = mul2(__byte_perm(v[2][b], v[3][b], 0x7632), s23);
#pragma unroll
                for (int nt = 0; nt < NTILES; ++nt) mma_f16(o[4 * y + b][nt], a0, a1, a2, a3, p[m][nt][0], p[m][nt][1]);
              }
            }
            if (edge && __any_sync(FULL, nan_blocks != 0)) {
              // a product of 1 where a value is NaN and 1 where a row sees its key says where NaN belongs
              uint32_t bad[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                bad[x] = __shfl_sync(FULL, nan_blocks, key0 + (x & 1) + 4 * (x & 2)) >> (D == 128 ? gq : gq >> 1) & 1 ? 0x3c00u : 0;
              const uint32_t a0 = bad[0] | bad[1] << 16, a2 = bad[2] | bad[3] << 16;
#pragma unroll
              for (int nt = 0; nt < NTILES; ++nt) {
                float hit[4] = {0, 0, 0, 0};
                uint32_t see[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  see[h] = transpose8((S[m][nt][2 * h] == -INFINITY ? 0 : 0x3c00u) | (S[m][nt][2 * h + 1] == -INFINITY ? 0 : 0x3c00u) << 16);
                mma_f16(hit, a0, a0, a2, a2, see[0], see[1]);
#pragma unroll
                for (int x = 0; x < MT; ++x)
#pragma unroll
                  for (int c = 0; c < 4; ++c)
                    if (hit[c] > 0.0f) o[x][nt][c] = quiet_nan();
              }
            }
          }
          __syncwarp();
          --pending;
          if (at_run == segs && at >= at_count && more && ok && (ok = bar_wait(q_full + 8 * (buf ^ 1), ((segs + 1) >> 1) & 1, flags))) enter(segs + 1);
          if (at < at_count) ask();
        }
        // ---- the warps' results meet
        const int parts = min(count, C::CONSUMERS);
#pragma unroll
        for (int nt = 0; nt < NTILES; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(FULL, l[nt][c], x);
            if (gq == 0) stat[w * R + nt * 8 + 2 * t4 + c] = make_float4(M[nt][c], N[nt][c], l[nt][c], 0.0f);
          }
        bool bad = g.bad != 0;
        const int used = (kv + ps - 1) >> shift, ppb = BN >> shift;                        // pages of this run that do not exist
        for (int p = g.j0 * ppb + ct; p < min(g.j1 * ppb, used); p += CT)
          bad |= (unsigned)__ldg(A.B.table + (size_t)g.b * A.B.max_pages + p) >= (unsigned)A.B.num_pages;
        if (group_or(BAR_ALL, CT, !ok)) break;             // also: the statistics are there
        bad = group_or(BAR_ALL, CT, bad);
        if (bad && ct == 0) flags[0] = 1;
        if (ct == 0) bar_arrive(q_empty + 8 * buf);        // nobody reads this run's queries any more
        if (ct < R) {
          float m = NOTHING, v = NOTHING, sum = 0.0f;
          for (int x = 0; x < parts; ++x) {
            m = fmaxf(m, stat[x * R + ct].x);
            v = fmaxf(v, stat[x * R + ct].y);
          }
          for (int x = 0; x < parts; ++x) sum += stat[x * R + ct].z * ex2(stat[x * R + ct].x - m);
          row_stat[ct] = make_float4(m, v, bad ? quiet_nan() : sum, 0.0f);
        }
#pragma unroll
        for (int nt = 0; nt < NTILES; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = NOTHING;
            for (int x = 0; x < parts; ++x) v = fmaxf(v, stat[x * R + nt * 8 + 2 * t4 + c].y);
            const float f = ex2(N[nt][c] - v);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              o[m][nt][c] *= f;
              o[m][nt][c + 2] *= f;
            }
          }
        constexpr int PASS = C::CM * NTILES * 128;         // floats of a warp at a time
#pragma unroll
        for (int m0 = 0; m0 < MT; m0 += C::CM) {
          if (m0 > 0) group_sync(BAR_ALL, CT);
          if (w < parts)
#pragma unroll
            for (int m = 0; m < C::CM; ++m)
#pragma unroll
              for (int nt = 0; nt < NTILES; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) merge[w * PASS + (m * NTILES + nt) * 128 + c * 32 + lane] = o[m0 + m][nt][c];
          group_sync(BAR_ALL, CT);
          for (int x4 = ct; x4 < PASS / 4; x4 += CT) {
            float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll 4
            for (int y = 0; y < parts; ++y) {
              const float4 t = *(const float4*)(merge + y * PASS + 4 * x4);
              sum.x += t.x; sum.y += t.y; sum.z += t.z; sum.w += t.w;
            }
            // four lanes of a row group: the same columns of rows two apart
            const int x = 4 * x4, ln = x & 31, c = (x >> 5) & 3, nt = (x >> 7) % NTILES, m = m0 + (x >> 7) / NTILES;
            float* const to = res + (nt * 8 + (c & 1)) * D + DV * (ln >> 2) + 2 * m + (c >> 1);
            to[0] = sum.x; to[2 * D] = sum.y; to[4 * D] = sum.z; to[6 * D] = sum.w;
          }
        }
        group_sync(BAR_ALL, CT);
        // ---- to the output, or as a partial result
        const int rows = min(A.tile_tokens, g.ntok) * A.group;
        auto out_row = [&](int r) { return (size_t)(g.row0 + r / A.group) * A.q_heads + g.head * A.group + r % A.group; };
        if (g.j0 == 0 && g.j1 == g.nblk) {
          for (int x = ct; x < rows * (D / 16); x += CT) {
            const int r = x / (D / 16), d = x % (D / 16) * 16;
            const float4 t = row_stat[r];
            store_row(A.out + out_row(r) * D + d, res + r * D + d, t.x, t.y, t.z);
          }
          if (A.lse)
            for (int r = ct; r < rows; r += CT) A.lse[out_row(r)] = log_sum(row_stat[r]);
        } else {
          constexpr int PART = part_floats<D>();
          auto part = [&](int cta, int slot) { return A.ws + (size_t)(cta * 2 + slot) * 2 * PART; };
          float* const dst = part(blockIdx.x, g.j0 == 0 ? 1 : 0);
          for (int x = ct; x < rows * (D / 4); x += CT) __stcg((float4*)(dst + 4 * R) + x, ((const float4*)res)[x]);
          if (ct < rows) __stcg((float4*)dst + ct, row_stat[ct]);
          const int c0 = first_run(g.start - SETUP, units, ctas), c1 = last_run(g.start - SETUP, SETUP + g.nblk, units, ctas);
          __threadfence();
          group_sync(BAR_ALL, CT);
          if (ct == 0) work[15] = atomicAdd(A.counters + c0, 1) == c1 - c0;
          group_sync(BAR_ALL, CT);
          if (work[15]) {                                  // the last to finish merges, in order
            __threadfence();
            if (ct == 0) A.counters[c0] = 0;
            if (ct < rows) {
              float m = NOTHING, v = NOTHING, sum = 0.0f;
#pragma unroll 4
              for (int x = c0; x <= c1; ++x) {
                const float4 t = __ldcg((const float4*)part(x, x == c0) + ct);
                m = fmaxf(m, t.x);
                v = fmaxf(v, t.y);
              }
#pragma unroll 4
              for (int x = c0; x <= c1; ++x) {
                const float4 t = __ldcg((const float4*)part(x, x == c0) + ct);
                sum += t.z * ex2(t.x - m);
                merge[(x - c0) * R + ct] = ex2(t.y - v);
              }
              row_stat[ct] = make_float4(m, v, sum, 0.0f);
            }
            group_sync(BAR_ALL, CT);
            for (int x = ct; x < rows * (D / 4); x += CT) {
              const int r = x / (D / 4);
              float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll 4
              for (int y = c0; y <= c1; ++y) {
                const float4 t = __ldcg((const float4*)(part(y, y == c0) + 4 * R) + x);
                const float f = merge[(y - c0) * R + r];
                sum.x += f * t.x; sum.y += f * t.y; sum.z += f * t.z; sum.w += f * t.w;
              }
              ((float4*)res)[x] = sum;
            }
            group_sync(BAR_ALL, CT);
            for (int x = ct; x < rows * (D / 16); x += CT) {
              const int r = x / (D / 16), d = x % (D / 16) * 16;
              const float4 t = row_stat[r];
              store_row(A.out + out_row(r) * D + d, res + r * D + d, t.x, t.y, t.z);
            }
            if (A.lse && ct < rows) A.lse[out_row(ct)] = log_sum(row_stat[ct]);
          }
        }
        ++segs;
        group_sync(BAR_ALL, CT);                           // results and statistics are used again
        if (!more) break;
      } while (true);
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  }
}

}  // namespace
