// Where a token lives in the cache, and the append of rotated rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_common.cuh"

namespace {

// ------------------------------------------------------- where a token lives
// A warp works on one token at a time, all its heads: the search of its
// sequence and page is paid once for 2 * heads vectors, whose 16-byte pieces
// the lanes then hold, several in flight each.

// The sequence that holds packed token t, or -1: 32 probes a step.  cu need not
// be trusted: the search stays in range whatever it holds, and the result is
// checked.
__device__ __forceinline__ int find_seq(const Batch& B, int t, int lane) {
  int lo = 0, hi = B.n_seqs;                      // largest b with cu[b] <= t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, probe = lo + lane * step;
    const int below = __popc(__ballot_sync(FULL, probe < hi && __ldg(B.cu + min(probe, hi)) <= t));
    lo += max(0, below - 1) * step;
    hi = min(hi, lo + step);
    lo = min(lo, hi - 1);
  }
  const int a = __ldg(B.cu + lo), e = __ldg(B.cu + lo + 1);
  return (a >= 0 && a <= t && t < e && e <= B.n_tokens) ? lo : -1;
}
// Page of token t, its slot there and its position.  NO_ROW: in no sequence, as the rows that pad a batch are (a wrong cu
// is reported by flag_invalid_seqs); INVALID: in one whose length or page is not valid, which is reported;
// NO_SLOT: before the first position.
enum { NO_SLOT = -1, INVALID = -2, NO_ROW = -3 };
__device__ __forceinline__ int find_page(const Batch& B, int t, int lane, int& slot, int& pos) {
  const int b = find_seq(B, t, lane);
  int page = NO_ROW;
  if (b >= 0) {
    const int len = __ldg(B.kv_len + b);
    pos = len - __ldg(B.cu + b + 1) + t;
    if (!len_valid(B, len)) {
      page = INVALID;
    } else if (pos < 0) {
      page = NO_SLOT;
    } else {
      page = __ldg(B.table + (size_t)b * B.max_pages + (pos >> B.page_shift));
      if ((unsigned)page >= (unsigned)B.num_pages) page = INVALID;
      slot = pos & ((1 << B.page_shift) - 1);
    }
  }
  if (page == INVALID && lane == 0) B.flags[0] = 1;
  return page;
}

// ---------------------------------------------------------- rotated append
// A vector x at position p becomes, for every pair (a, b) of its first `rot`
// elements, (a c - b s, b c + a s) with the cosine and sine that the table holds
// for p: neighbours (2i, 2i+1) or halves (i, i + rot / 2).  The two products are
// rounded to 32 bits each and then their sum, so that the result is that of the
// formula's operations one by one; queries (and keys that are asked for) leave
// rounded once to bf16, cached keys and values are quantised from the 32 bits.
//
// Quantisation.  e4m3: x becomes round(x / 2^e), e the least exponent with
// max|x| <= 448 * 2^e.  e2m1: e is the least exponent with max|x| <= 2688 * 2^e,
// 16 values share s = round_e4m3(max|values| / 2^e / 6), and a code is
// round(x / 2^e / s).  That quotient is the correctly rounded one: s has 4
// significant bits, x often 8, so ties are common and a product with 1 / s would
// miss some (15 * fl(1 / 15) is above 1).  With r = fl(1 / s) and q = fl(x r) it
// is q + (x - q s) r in two fused steps (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990), which agrees with the
// division for every 24-bit x and 4-bit s.
//
// A warp works on some of the vectors of one token: queries, then keys, then
// values, 16 bytes a lane, so that a lane keeps the cosines and sines of its
// place in the vector and finds its partner's value by a shuffle.  The first
// vectors are loaded ahead of the search for the token's page, the next ones
// ahead of the work on these.
//
// Bound by memory where tokens are many: 35,894 tokens of 32 query and 8 key-value
// heads of 128 into a bf16 cache, with the rotated keys out too, take 158 us, 6.1
// TB/s (198 with twice as many loads at a time, none ahead, and 104 registers).
// 35,894 tokens with 32 query heads into 4 bits take 172 us where memory would
// need 115.  2,048 tokens with 64 query heads into an e4m3 cache take 18.4 us where
// L2 holds the outputs' memory already and 21.2 where not (memory: 11.8): a warp's
// chain of search, page and five loads.  Few tokens 3.3 us.
struct Turn {
  const float* table;              // [max_positions, rot]: cosines, then sines
  const int32_t* positions;        // of the tokens; null: their places in the cache
  int max_positions;
  int rot;
  int interleaved;
};
struct RowsOut {
  __nv_bfloat16* ptr;              // null: not wanted
  long long st, sh;
};
enum { POOL_BF16 = 0, POOL_E4M3 = 1, POOL_E2M1 = 2 };

// Least e >= EXP_MIN with x <= m * 2^(e + shift), x >= 0 and m = 1.f in [1, 2) by the bits of f
__device__ __forceinline__ int least_exponent(uint32_t x, int shift, uint32_t f) {
  return max(EXP_MIN, (int)(x >> 23) - EXP_BIAS - shift + ((x & 0x7fffffu) > f));
}
__device__ __forceinline__ uint4 ld_once(const void* p) {   // not through the read-only path: rows may be rotated in place
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

constexpr int UT = 2;              // 16-byte pieces that a lane loads at a time, while it works on as many before

// 1 / s of a scale of 4 significant bits, correctly rounded (the tests take every scale)
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return s > 0.0f ? __fmaf_rn(__fmaf_rn(-r, s, 1.0f), r, r) : 0.0f;
}
// x / s correctly rounded, r = fl(1 / s) (see above); two at once
__device__ __forceinline__ u64 quotient(u64 x, u64 s_neg, u64 r) {
  const u64 q = mul2f(x, r);
  return fma2(fma2(q, s_neg, x), r, q);
}

struct Four {
  uint8_t byte, scale;             // of the vector, of the block
};
// Quantises n elements y of a block of an e2m1 vector: to y / 2^e / scale.  top and block are the bits of the largest
// magnitude of the vector and of the block.
__device__ __forceinline__ Four four_scale(uint32_t top, uint32_t block, float* y, const int n) {
  const bool bad = top >= 0x7f800000u;            // an infinity or NaN
  int e = least_exponent(top, 11, 0x280000u);
  Four f;
  f.byte = (uint8_t)(bad ? BYTE_NAN : e + EXP_BIAS);
  float most = __uint_as_float(block);
  if (e < -64) {                                  // tiny vectors: away from the end of the exponents' range, exactly
    e += 64;
    most *= 18446744073709551616.0f;
#pragma unroll
    for (int i = 0; i < n; ++i) y[i] *= 18446744073709551616.0f;
  }
  // everything in units of 2^e: powers of two round nothing
  const float unit = __uint_as_float((uint32_t)(EXP_BIAS + e) << 23), inv = __uint_as_float((uint32_t)(EXP_BIAS - e) << 23);
  float sixth, ignored;
  upk(quotient(pk(most * inv, 0.0f), pk(-6.0f, -6.0f), pk(1.0f / 6.0f, 0.0f)), sixth, ignored);
  f.scale = bad ? 0x7f : (uint8_t)pack_e4m3(sixth, 0.0f, 0.0f, 0.0f);
  const float s = f16x2_to_f32(e4m3_to_f16x2(f.scale)).x, r = reciprocal(s) * inv, sn = -s * unit;
  const u64 r2 = pk(r, r), s2 = pk(sn, sn);
#pragma unroll
  for (int i = 0; i < n; i += 2) upk(quotient(pk(y[i], y[i + 1]), s2, r2), y[i], y[i + 1]);
  return f;
}

template <int D, int POOL>
__global__ void __launch_bounds__(128, POOL == POOL_E2M1 ? 8 : 7) sa_rotate_kernel(Batch B, Pool P, Turn T, Rows Q, Rows K, Rows V, RowsOut QO, RowsOut KO, int q_heads,
                                                        int heads, int splits, int per) {
  constexpr int U = UT;
  constexpr int LV = D / 8, VS = 32 / LV;         // lanes of a vector, vectors a step
  flag_invalid_seqs(B);
  const int lane = threadIdx.x & 31, piece = lane % LV, sub = lane / LV;
  const int unit = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = unit / splits, v0 = (unit - t * splits) * per, v1 = min(v0 + per, q_heads + 2 * heads);
  if (t >= B.n_tokens) return;
  uint4 x[U];
  auto load = [&](int v, uint4* x) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int vi = v + u * VS + sub;
      const __nv_bfloat16* src = Q.ptr + t * Q.st + vi * Q.sh;
      if (vi >= q_heads) src = K.ptr + t * K.st + (vi - q_heads) * K.sh;
      if (vi >= q_heads + heads) src = V.ptr + t * V.st + (vi - q_heads - heads) * V.sh;
      x[u] = vi < v1 ? ld_once(src + piece * 8) : make_uint4(0, 0, 0, 0);
    }
  };
  load(v0, x);
  int slot = 0, pos = 0, page = find_page(B, t, lane, slot, pos);
  if (page == NO_ROW) return;
  if (T.positions) pos = __ldg(T.positions + t);
  if (page >= 0 && (unsigned)pos >= (unsigned)T.max_positions) {
    page = INVALID;
    if (lane == 0) B.flags[0] = 1;
  }
  if (page < 0) {                                 // nothing for the cache; its rows are 0 or NaN
    const uint32_t f = page == INVALID ? 0x7fc07fc0u : 0;
    for (int v = v0; v < v1; v += VS) {
      const int vi = v + sub, h = vi - q_heads;
      if (vi < v1 && vi < q_heads) *(uint4*)(QO.ptr + t * QO.st + vi * QO.sh + piece * 8) = make_uint4(f, f, f, f);
      if (vi < v1 && h >= 0 && h < heads && KO.ptr) *(uint4*)(KO.ptr + t * KO.st + h * KO.sh + piece * 8) = make_uint4(f, f, f, f);
    }
    return;
  }
  // this lane's place in the rotation
  u64 C2[4], S2[4];                               // two elements' each: rounded one by one, two at a time
  int from = lane;
  const bool turns = piece * 8 < T.rot;
  if (turns) {
    const float* const row = T.table + (size_t)pos * T.rot;
    const int half = T.rot / 2;
    if (T.interleaved) {
      const float4 c = __ldg((const float4*)(row + piece * 4)), s = __ldg((const float4*)(row + half + piece * 4));
      C2[0] = pk(c.x, c.x); C2[1] = pk(c.y, c.y); C2[2] = pk(c.z, c.z); C2[3] = pk(c.w, c.w);
      S2[0] = pk(-s.x, s.x); S2[1] = pk(-s.y, s.y); S2[2] = pk(-s.z, s.z); S2[3] = pk(-s.w, s.w);
    } else {
      const bool first = piece * 8 < half;
      from = first ? lane + half / 8 : lane - half / 8;
      const float* const c = row + piece * 8 - (first ? 0 : half);
      const float sign = first ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 a = __ldg((const float4*)c + e), b = __ldg((const float4*)(c + half) + e);
        C2[2 * e] = pk(a.x, a.y);
        C2[2 * e + 1] = pk(a.z, a.w);
        S2[2 * e] = pk(sign * b.x, sign * b.y);
        S2[2 * e + 1] = pk(sign * b.z, sign * b.w);
      }
    }
  }
  const long long vec0 = (((long long)page * heads) << B.page_shift) + slot;
  for (int v = v0;;) {
    uint4 next[U];
    if (v + VS * U < v1) load(v + VS * U, next);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int vi = v + u * VS + sub, kh = vi - q_heads;
      if (v + u * VS >= v1) break;                // uniform
      const bool in = vi < v1, is_v = kh >= heads, turned = turns && !is_v;
      uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, o[4];
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf_lo(w[i]);
        y[2 * i + 1] = bf_hi(w[i]);
        o[i] = w[i];
      }
      if (v + u * VS < q_heads + heads) {        // uniform: some vector of the step is a query or a key
        if (!T.interleaved)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(FULL, w[i], from);
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = y[2 * i], b = y[2 * i + 1];
            const float pa = T.interleaved ? b : bf_lo(o[i]), pb = T.interleaved ? a : bf_hi(o[i]);
            float x0, x1, z0, z1;                 // sums one by one: a packed sum of packed products is fused
            upk(mul2f(pk(a, b), C2[i]), x0, x1);
            upk(mul2f(pk(pa, pb), S2[i]), z0, z1);
            y[2 * i] = __fadd_rn(x0, z0);
            y[2 * i + 1] = __fadd_rn(x1, z1);
            w[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
          }
        }
      }
      if (in && kh < 0) *(uint4*)(QO.ptr + t * QO.st + vi * QO.sh + piece * 8) = make_uint4(w[0], w[1], w[2], w[3]);
      if (in && kh >= 0 && !is_v && KO.ptr) *(uint4*)(KO.ptr + t * KO.st + kh * KO.sh + piece * 8) = make_uint4(w[0], w[1], w[2], w[3]);
      if (v + u * VS + VS <= q_heads) continue;   // uniform: queries only
      const long long vec = vec0 + ((long long)(is_v ? kh - heads : kh) << B.page_shift);
      char* const dst = (char*)(is_v ? P.v : P.k);
      if constexpr (POOL == POOL_BF16) {
        if (in && kh >= 0) *(uint4*)(dst + (vec * D + piece * 8) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        uint32_t top = 0;                         // magnitudes as bit patterns order like the values, NaN above all
        if (v + u * VS < q_heads + heads) {
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
        } else {                                  // bf16 as they came: two at once
          const uint32_t m = 0x7fff7fffu, z = __vmaxu2(__vmaxu2(w[0] & m, w[1] & m), __vmaxu2(w[2] & m, w[3] & m));
          top = max(z << 16, z & 0xffff0000u);
        }
        top = max(top, __shfl_xor_sync(FULL, top, 1));
        const uint32_t block = top;
#pragma unroll
        for (int s = LV / 2; s > 1; s >>= 1) top = max(top, __shfl_xor_sync(FULL, top, s));
        const bool bad = top >= 0x7f800000u;      // an infinity or NaN
        uint8_t byte;
        if constexpr (POOL == POOL_E4M3) {
          const int e = least_exponent(top, 8, 0x600000u);
          byte = (uint8_t)(bad ? BYTE_NAN : e + EXP_BIAS);
          const float inv = __uint_as_float((uint32_t)(EXP_BIAS - e) << 23);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= inv;
          uint2 c = make_uint2(pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7]));
          if (bad) c = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
          if (in && kh >= 0) *(uint2*)(dst + vec * D + piece * 8) = c;
        } else {
          const Four f = four_scale(top, block, y, 8);
          byte = f.byte;
          const uint32_t c = bad ? 0 : pack_e2m1(y);
          if (in && kh >= 0) {
            *(uint32_t*)(dst + vec * (D / 2) + piece * 4) = c;
            if (!(piece & 1)) (is_v ? P.vb : P.kb)[vec * (D / 16) + piece / 2] = f.scale;
          }
        }
        if (in && kh >= 0 && piece == 0) (is_v ? P.vs : P.ks)[vec] = byte;
      }
    }
    v += VS * U;
    if (v >= v1) return;
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = next[u];
  }
}

}  // namespace
