// Parameters and helpers shared by the cache and attention kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_plan.cuh"

// ---------------------------------------------------------------- parameters
namespace sv_attn {   // the same types in every translation unit
struct Batch {                     // spec_attn_batch, plus what follows from the handle
  const int32_t* cu;
  const int32_t* kv_len;           // null: packed prompts (a sequence holds its new tokens only)
  const int32_t* table;
  int n_seqs, n_tokens, max_pages;
  int page_shift;
  int num_pages;
  int* flags;                      // [0] invalid metadata, [1] wait timeout
};
struct Pool {
  void* k;
  void* v;
  uint8_t* ks;
  uint8_t* vs;
  uint8_t* kb;                     // e2m1: a scale for every 16 codes
  uint8_t* vb;
};
struct Rows {
  const __nv_bfloat16* ptr;
  long long st, sh;                // token and head strides, elements
};

}  // namespace sv_attn

namespace {

using namespace sv_attn;

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E_F = 1.44269504088896341f;
constexpr float LN2_F = 0.69314718055994531f;
constexpr int EXP_MIN = -120;      // least exponent of a cached vector's scale
constexpr int EXP_BIAS = 127;
constexpr int BYTE_NAN = 255;      // scale byte of a vector that holds an infinity or NaN

// ------------------------------------------------------------------- helpers
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }
// two floats in a 64-bit register, and arithmetic on both
typedef unsigned long long u64;
__device__ __forceinline__ u64 pk(float lo, float hi) { u64 r; asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi)); return r; }
__device__ __forceinline__ void upk(u64 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) { u64 d; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c)); return d; }
__device__ __forceinline__ u64 add2(u64 a, u64 b) { u64 d; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b)); return d; }
__device__ __forceinline__ u64 mul2f(u64 a, u64 b) { u64 d; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b)); return d; }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16_down(float lo, float hi) {   // towards 0
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// four floats to four e4m3 codes (nearest even, saturating; NaN stays NaN)
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// two e4m3 codes to two f16 values (exact)
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// eight e2m1 codes, the first in the lowest bits, to f16 values times f (both of a pair alike)
__device__ __forceinline__ void e2m1_to_f16(uint32_t c, uint32_t f, uint32_t* y) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}" : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]) : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y[i]) : "r"(f));
}
// eight floats to e2m1 codes (nearest even, saturating), the first in the lowest bits
__device__ __forceinline__ uint32_t pack_e2m1(const float* x) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
// 2^e for the exponents a scale byte can hold (0 for byte 0, see sa_read_kernel); NaN for BYTE_NAN
__device__ __forceinline__ float scale_of(int byte) { return byte == BYTE_NAN ? quiet_nan() : __int_as_float(byte << 23); }
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ bool len_valid(const Batch& B, int len) {
  return len >= 0 && len <= LEN_MAX && (long long)len <= ((long long)B.max_pages << B.page_shift);
}
// Whether sequence b's row range and length are within the call's limits.
__device__ __forceinline__ bool seq_valid(const Batch& B, int b) {
  const int a = __ldg(B.cu + b), e = __ldg(B.cu + b + 1);
  if (a < 0 || e < a || e > B.n_tokens) return false;
  return !B.kv_len || len_valid(B, __ldg(B.kv_len + b));
}
// The first block reports sequences that no token leads to (a decreasing cu).
__device__ __forceinline__ void flag_invalid_seqs(const Batch& B) {
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < B.n_seqs; b += blockDim.x)
      if (!seq_valid(B, b)) B.flags[0] = 1;
}

}  // namespace
