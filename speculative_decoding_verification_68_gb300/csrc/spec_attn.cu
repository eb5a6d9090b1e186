// spec_attn: paged key-value cache and attention around a verification step
// on one GB300 (sm_103a).  The C interface and the method are described in
// include/spec_attn.h; this file holds the kernels and the host side.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "spec_attn.h"

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E_F = 1.44269504088896341f;
constexpr float LN2_F = 0.69314718055994531f;
constexpr int EXP_MIN = -120;      // least exponent of a cached vector's scale
constexpr int EXP_BIAS = 127;
constexpr int BYTE_NAN = 255;      // scale byte of a vector that holds an infinity or NaN

// ---------------------------------------------------------------- parameters
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
};
struct Rows {
  const __nv_bfloat16* ptr;
  long long st, sh;                // token and head strides, elements
};

// ------------------------------------------------------------------- helpers
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
// 2^e for the exponents a scale byte can hold; NaN for BYTE_NAN
__device__ __forceinline__ float scale_of(int byte) {
  return byte == BYTE_NAN ? __int_as_float(0x7fc00000) : __int_as_float(byte << 23);
}
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The sequence that holds packed token t, or -1.  cu need not be trusted: the
// search stays in range whatever it holds, and the result is checked.
__device__ __forceinline__ int find_seq(const Batch& B, int t) {
  int lo = 0, hi = B.n_seqs;                      // largest b with cu[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(B.cu + mid) <= t) lo = mid; else hi = mid;
  }
  const int a = __ldg(B.cu + lo), e = __ldg(B.cu + lo + 1);
  return (a >= 0 && a <= t && t < e && e <= B.n_tokens) ? lo : -1;
}
// Slot index (page * page_size + slot, the head still to be added) of position
// pos; -1 where it has none, -2 where the metadata is invalid (flagged).
__device__ __forceinline__ long long find_slot(const Batch& B, int b, int pos) {
  if (pos < 0) return -1;
  const int page = __ldg(B.table + (size_t)b * B.max_pages + (pos >> B.page_shift));
  if ((unsigned)page >= (unsigned)B.num_pages) return -2;
  return ((long long)page << B.page_shift) | (pos & ((1 << B.page_shift) - 1));
}
// Position of packed token t; false where the sequence is invalid.
__device__ __forceinline__ bool token_place(const Batch& B, int t, int& b, int& pos) {
  b = find_seq(B, t);
  if (b < 0) return false;
  const int len = __ldg(B.kv_len + b);
  if (len < 0 || (long long)len > ((long long)B.max_pages << B.page_shift)) return false;
  pos = len - __ldg(B.cu + b + 1) + t;
  return true;
}
// element offset of the vector of (slot, head) in a pool [page, head, slot, D]
__device__ __forceinline__ long long vec_index(long long slot, int head, int heads, int page_shift) {
  const long long page = slot >> page_shift;
  return ((page * heads + head) << page_shift) + (slot & ((1 << page_shift) - 1));
}

// Whether sequence b's row range and length are within the call's limits.
__device__ __forceinline__ bool seq_valid(const Batch& B, int b) {
  const int a = __ldg(B.cu + b), e = __ldg(B.cu + b + 1);
  if (a < 0 || e < a || e > B.n_tokens) return false;
  if (!B.kv_len) return true;
  const int len = __ldg(B.kv_len + b);
  return len >= 0 && (long long)len <= ((long long)B.max_pages << B.page_shift);
}
// The first block reports sequences that no token leads to (a decreasing cu).
__device__ __forceinline__ void flag_invalid_seqs(const Batch& B) {
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < B.n_seqs; b += blockDim.x)
      if (!seq_valid(B, b)) B.flags[0] = 1;
}

// -------------------------------------------------------------------- append
// One 16-byte lane-load per 8 elements: D / 8 lanes hold one vector, so its
// largest magnitude is a few shuffles away and the codes leave as 8-byte
// stores.  Bound by memory: 2 D bytes read and D + 1 written per vector.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) sa_append_kernel(Batch B, Pool P, Rows K, Rows V, int heads) {
  constexpr int LV = D / 8;
  flag_invalid_seqs(B);
  const long long n = (long long)B.n_tokens * heads;
  const int lane = threadIdx.x % LV;
  const long long step = (long long)gridDim.x * (256 / LV);
  // every lane of a warp makes the same number of turns: the shuffles below are warp-wide
  for (long long base = (long long)blockIdx.x * (256 / LV); base < n; base += step) {
    const long long i = base + threadIdx.x / LV;
    const bool in = i < n;
    const int t = in ? (int)(i / heads) : 0, head = in ? (int)(i - (long long)t * heads) : 0;
    int b = -1, pos = -1;
    long long slot = -1;
    if (in) {
      if (token_place(B, t, b, pos)) slot = find_slot(B, b, pos);
      else slot = -2;
      if (slot == -2 && lane == 0) B.flags[0] = 1;
    }
    uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (slot >= 0) {
      x[0] = ldg_stream(K.ptr + t * K.st + head * K.sh + lane * 8);
      x[1] = ldg_stream(V.ptr + t * V.st + head * V.sh + lane * 8);
    }
    const long long vec = slot >= 0 ? vec_index(slot, head, heads, B.page_shift) : 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      char* dst = (char*)(s ? P.v : P.k);
      if constexpr (!FP8) {
        if (slot >= 0) *(uint4*)(dst + (vec * D + lane * 8) * 2) = x[s];
      } else {
        // magnitudes as bf16 bit patterns order like the values, infinities and NaN above all
        const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
#pragma unroll
        for (int o = LV / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
        // least e with max <= 448 * 2^e = 1.75 * 2^(e + 8)
        const int e = max(EXP_MIN, (int)(top >> 7) - EXP_BIAS - 8 + ((top & 0x7fu) > 0x60u));
        const bool bad = top >= 0x7f80u;
        const float inv = __int_as_float((EXP_BIAS - e) << 23);
        uint2 c;
        c.x = pack_e4m3(bf_lo(w[0]) * inv, bf_hi(w[0]) * inv, bf_lo(w[1]) * inv, bf_hi(w[1]) * inv);
        c.y = pack_e4m3(bf_lo(w[2]) * inv, bf_hi(w[2]) * inv, bf_lo(w[3]) * inv, bf_hi(w[3]) * inv);
        if (bad) c = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        if (slot >= 0) {
          *(uint2*)(dst + vec * D + lane * 8) = c;
          if (lane == 0) (s ? P.vs : P.ks)[vec] = (uint8_t)(bad ? BYTE_NAN : e + EXP_BIAS);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------- read
// The reverse of append, one 16-byte store per lane.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) sa_read_kernel(Batch B, Pool P, uint4* ko, uint4* vo, int heads) {
  constexpr int LV = D / 8;
  flag_invalid_seqs(B);
  const long long n = (long long)B.n_tokens * heads * LV;
  const uint32_t nan2 = 0x7fc07fc0u;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int lane = (int)(i % LV);
    const long long th = i / LV;
    const int t = (int)(th / heads), head = (int)(th - (long long)t * heads);
    int b, pos;
    if (!token_place(B, t, b, pos)) {
      if (lane == 0) B.flags[0] = 1;
      if (find_seq(B, t) >= 0) ko[i] = vo[i] = make_uint4(nan2, nan2, nan2, nan2);
      continue;
    }
    const long long slot = find_slot(B, b, pos);
    if (slot < 0) {
      if (slot == -2 && lane == 0) B.flags[0] = 1;
      const uint32_t f = slot == -2 ? nan2 : 0;
      ko[i] = vo[i] = make_uint4(f, f, f, f);
      continue;
    }
    const long long vec = vec_index(slot, head, heads, B.page_shift);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const char* src = (const char*)(s ? P.v : P.k);
      uint4 y;
      if constexpr (!FP8) {
        y = ldg_stream(src + (vec * D + lane * 8) * 2);
      } else {
        const uint2 c = __ldg((const uint2*)(src + vec * D + lane * 8));
        const float f = scale_of(__ldg((s ? P.vs : P.ks) + vec));
        const uint32_t w[2] = {c.x, c.y};
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 z = f16x2_to_f32(e4m3_to_f16x2((uint16_t)(w[j >> 1] >> (16 * (j & 1)))));
          r[j] = pack_bf16(z.x * f, z.y * f);
        }
        y = make_uint4(r[0], r[1], r[2], r[3]);
      }
      (s ? vo : ko)[i] = y;
    }
  }
}

// ----------------------------------------------------------------- attention
// One warp per row (token, query head).  32 keys at a time: each lane scores
// one key, the running maximum and sum are merged, then each lane adds the 32
// values of its D / 32 dimensions.  Everything in 32 bits.
template <int D, bool FP8, bool PACKED>
__global__ void __launch_bounds__(128) sa_attention_simple(Batch B, Pool P, Rows Q, Rows K, Rows V, int q_heads, int kv_heads,
                                                           int causal, float scale, __nv_bfloat16* out, float* lse) {
  constexpr int DL = D / 32;
  flag_invalid_seqs(B);
  __shared__ float qs[4][D];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + w;
  if (row >= (long long)B.n_tokens * q_heads) return;
  const int t = (int)(row / q_heads), hq = (int)(row % q_heads), head = hq / (q_heads / kv_heads);
  const int b = find_seq(B, t);
  if (b < 0) {
    if (lane == 0) B.flags[0] = 1;
    return;
  }
  const int first = __ldg(B.cu + b), n = __ldg(B.cu + b + 1) - first;
  int len = PACKED ? n : __ldg(B.kv_len + b);
  bool bad = !PACKED && (len < 0 || (long long)len > ((long long)B.max_pages << B.page_shift));
  const int seen = bad ? 0 : causal ? max(0, len - n + (t - first) + 1) : len;
  for (int d = lane; d < D; d += 32) qs[w][d] = __bfloat162float(Q.ptr[t * Q.st + hq * Q.sh + d]) * (scale * LOG2E_F);
  __syncwarp();
  float m = -INFINITY, l = 0.0f, o[DL];
#pragma unroll
  for (int i = 0; i < DL; ++i) o[i] = 0.0f;
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    long long vec = -1;
    if (j < seen) {
      if (PACKED) {
        vec = first + j;
      } else {
        const long long slot = find_slot(B, b, j);
        if (slot < 0) bad = true; else vec = vec_index(slot, head, kv_heads, B.page_shift);
      }
      if (vec >= 0) {
        s = 0.0f;
        if constexpr (FP8) {
          const uint2* p = (const uint2*)((const char*)P.k + vec * D);
          for (int c = 0; c < D / 8; ++c) {
            const uint2 x = __ldg(p + c);
            const uint32_t ww[2] = {x.x, x.y};
            for (int e = 0; e < 4; ++e) {
              const float2 z = f16x2_to_f32(e4m3_to_f16x2((uint16_t)(ww[e >> 1] >> (16 * (e & 1)))));
              s += z.x * qs[w][c * 8 + 2 * e];
              s += z.y * qs[w][c * 8 + 2 * e + 1];
            }
          }
          s *= scale_of(__ldg(P.ks + vec));
        } else {
          const uint4* p = (const uint4*)(PACKED ? K.ptr + vec * K.st + head * K.sh : (const __nv_bfloat16*)P.k + vec * D);
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = __ldg(p + c);
            const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
            for (int e = 0; e < 4; ++e) {
              s += bf_lo(ww[e]) * qs[w][c * 8 + 2 * e];
              s += bf_hi(ww[e]) * qs[w][c * 8 + 2 * e + 1];
            }
          }
        }
      }
    }
    float mx = s;
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, x));
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.0f : mn;
    const float p = exp2f(s - ref), f = exp2f(m - ref);
    float sum = p;
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(FULL, sum, x);
    l = l * f + sum;
    m = mn;
    for (int i = 0; i < DL; ++i) o[i] *= f;
    for (int k = 0; k < 32 && j0 + k < seen; ++k) {
      const float pk = __shfl_sync(FULL, p, k);
      const long long vk = __shfl_sync(FULL, vec, k);
      if (vk < 0) continue;
      if constexpr (FP8) {
        const float f2 = scale_of(__ldg(P.vs + vk)) * pk;
        const uint8_t* p8 = (const uint8_t*)P.v + vk * D + lane * DL;
        for (int i = 0; i < DL; ++i) o[i] += f2 * f16x2_to_f32(e4m3_to_f16x2(p8[i])).x;
      } else {
        const __nv_bfloat16* pv = (PACKED ? V.ptr + vk * V.st + head * V.sh : (const __nv_bfloat16*)P.v + vk * D) + lane * DL;
        for (int i = 0; i < DL; ++i) o[i] += pk * __bfloat162float(pv[i]);
      }
    }
  }
  bad = __any_sync(FULL, bad);
  if (bad && lane == 0) B.flags[0] = 1;
  const float inv = bad ? __int_as_float(0x7fc00000) : l == 0.0f ? 0.0f : 1.0f / l;
  for (int i = 0; i < DL; ++i) out[row * D + lane * DL + i] = __float2bfloat16(o[i] * inv);
  if (lse && lane == 0) lse[row] = bad ? inv : (m + log2f(l)) * LN2_F;
}

}  // namespace

// ---------------------------------------------------------------------- host
struct spec_attn_ctx {
  int device, q_heads, kv_heads, D, max_seqs;
  int n_sm;
  int* d_flags;
};

static void free_ctx(spec_attn_ctx* h) {
  if (!h) return;
  if (h->d_flags) cudaFree(h->d_flags);
  free(h);
}

extern "C" int spec_attn_init(spec_attn_t* out, int q_heads, int kv_heads, int head_dim, int max_seqs) {
  if (!out) return SV_ERR_ARG;
  *out = nullptr;
  if (q_heads < 1 || kv_heads < 1 || max_seqs < 1) return SV_ERR_ARG;
  if (q_heads % kv_heads || q_heads / kv_heads > 64 || q_heads > 1024 || max_seqs > 65536 || (head_dim != 64 && head_dim != 128))
    return SV_ERR_SIZE;
  spec_attn_ctx* h = (spec_attn_ctx*)calloc(1, sizeof(spec_attn_ctx));
  if (!h) return SV_ERR_ALLOC;
  h->q_heads = q_heads; h->kv_heads = kv_heads; h->D = head_dim; h->max_seqs = max_seqs;
  if (cudaGetDevice(&h->device) != cudaSuccess || cudaDeviceGetAttribute(&h->n_sm, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
    cudaGetLastError();
    free_ctx(h);
    return SV_ERR_CUDA;
  }
  if (cudaMalloc(&h->d_flags, 4 * sizeof(int)) != cudaSuccess || cudaMemset(h->d_flags, 0, 4 * sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    free_ctx(h);
    return SV_ERR_ALLOC;
  }
  *out = h;
  return SV_OK;
}

static bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

static int check_pool(const spec_attn_ctx* h, const spec_attn_pool* p) {
  if (!p || !p->k || !p->v || p->num_pages < 1 || !aligned16(p->k) || !aligned16(p->v)) return SV_ERR_ARG;
  if (p->dtype != SV_BF16 && p->dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (p->dtype == SV_E4M3 && (!p->k_scale || !p->v_scale)) return SV_ERR_ARG;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return SV_ERR_SIZE;
  if ((long long)p->num_pages * h->kv_heads * p->page_size >= (1ll << 31)) return SV_ERR_SIZE;
  return SV_OK;
}
static int check_batch(const spec_attn_ctx* h, const spec_attn_batch* b) {
  if (!b || b->n_seqs < 0 || b->n_tokens < 0 || b->max_pages < 0 || b->n_seqs > h->max_seqs) return SV_ERR_ARG;
  if (b->n_seqs > 0 && (!b->cu || !b->kv_len || (!b->page_table && b->max_pages > 0))) return SV_ERR_ARG;
  if ((long long)b->n_tokens * h->q_heads >= (1ll << 31)) return SV_ERR_SIZE;
  return SV_OK;
}
static int check_rows(const spec_attn_rows* r) {
  if (!r || !r->ptr || !aligned16(r->ptr) || r->token_stride % 8 || r->head_stride % 8 || r->token_stride < 0 || r->head_stride < 0)
    return SV_ERR_ARG;
  return SV_OK;
}
static int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}
static Batch batch_of(const spec_attn_ctx* h, const spec_attn_batch* b, const spec_attn_pool* p) {
  Batch r;
  r.cu = b->cu; r.kv_len = b->kv_len; r.table = b->page_table;
  r.n_seqs = b->n_seqs; r.n_tokens = b->n_tokens; r.max_pages = b->max_pages;
  r.page_shift = p ? log2_of(p->page_size) : 0;
  r.num_pages = p ? p->num_pages : 0;
  r.flags = h->d_flags;
  return r;
}
static Pool pool_of(const spec_attn_pool* p) { return Pool{p->k, p->v, p->k_scale, p->v_scale}; }
static Rows rows_of(const spec_attn_rows* r) { return Rows{(const __nv_bfloat16*)r->ptr, r->token_stride, r->head_stride}; }
static int launched() { return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

extern "C" int spec_attn_append(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                                const spec_attn_rows* k, const spec_attn_rows* v, void* cuda_stream) {
  if (!h) return SV_ERR_ARG;
  int rc;
  if ((rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return SV_OK;
  if ((rc = check_rows(k)) || (rc = check_rows(v))) return rc;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const Batch B = batch_of(h, batch, pool);
  const Pool P = pool_of(pool);
  const int per = 256 / (h->D / 8);
  const long long n = ((long long)B.n_tokens * h->kv_heads + per - 1) / per;
  const int grid = (int)(n < h->n_sm * 16 ? n : h->n_sm * 16);
  if (h->D == 128) {
    if (pool->dtype == SV_E4M3) sa_append_kernel<128, true><<<grid, 256, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else sa_append_kernel<128, false><<<grid, 256, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
  } else {
    if (pool->dtype == SV_E4M3) sa_append_kernel<64, true><<<grid, 256, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else sa_append_kernel<64, false><<<grid, 256, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
  }
  return launched();
}

extern "C" int spec_attn_read(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                              void* k_out, void* v_out, void* cuda_stream) {
  if (!h) return SV_ERR_ARG;
  int rc;
  if ((rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return SV_OK;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return SV_ERR_ARG;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const Batch B = batch_of(h, batch, pool);
  const Pool P = pool_of(pool);
  const long long n = ((long long)B.n_tokens * h->kv_heads * (h->D / 8) + 255) / 256;
  const int grid = (int)(n < h->n_sm * 16 ? n : h->n_sm * 16);
  uint4 *ko = (uint4*)k_out, *vo = (uint4*)v_out;
  if (h->D == 128) {
    if (pool->dtype == SV_E4M3) sa_read_kernel<128, true><<<grid, 256, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else sa_read_kernel<128, false><<<grid, 256, 0, s>>>(B, P, ko, vo, h->kv_heads);
  } else {
    if (pool->dtype == SV_E4M3) sa_read_kernel<64, true><<<grid, 256, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else sa_read_kernel<64, false><<<grid, 256, 0, s>>>(B, P, ko, vo, h->kv_heads);
  }
  return launched();
}

template <int D, bool FP8, bool PACKED>
static void launch_attention(spec_attn_ctx* h, const Batch& B, const Pool& P, const Rows& Q, const Rows& K, const Rows& V, int causal,
                             float scale, void* out, float* lse, cudaStream_t s) {
  const long long rows = (long long)B.n_tokens * h->q_heads;
  sa_attention_simple<D, FP8, PACKED><<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(B, P, Q, K, V, h->q_heads, h->kv_heads, causal, scale,
                                                                              (__nv_bfloat16*)out, lse);
}

extern "C" int spec_attn_chunk(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                               const spec_attn_rows* q, int causal, float scale, void* out, float* lse, void* cuda_stream) {
  if (!h || !(scale > 0.0f) || !isfinite(scale)) return SV_ERR_ARG;
  int rc;
  if ((rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return SV_OK;
  if ((rc = check_rows(q))) return rc;
  if (!out || !aligned16(out)) return SV_ERR_ARG;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const Batch B = batch_of(h, batch, pool);
  const Pool P = pool_of(pool);
  const Rows Q = rows_of(q), none{};
  if (h->D == 128) {
    if (pool->dtype == SV_E4M3) launch_attention<128, true, false>(h, B, P, Q, none, none, causal, scale, out, lse, s);
    else launch_attention<128, false, false>(h, B, P, Q, none, none, causal, scale, out, lse, s);
  } else {
    if (pool->dtype == SV_E4M3) launch_attention<64, true, false>(h, B, P, Q, none, none, causal, scale, out, lse, s);
    else launch_attention<64, false, false>(h, B, P, Q, none, none, causal, scale, out, lse, s);
  }
  return launched();
}

extern "C" int spec_attn_prompt(spec_attn_t h, int n_seqs, int n_tokens, const int32_t* cu,
                                const spec_attn_rows* q, const spec_attn_rows* k, const spec_attn_rows* v,
                                float scale, void* out, float* lse, void* cuda_stream) {
  if (!h || !(scale > 0.0f) || !isfinite(scale) || n_seqs < 0 || n_tokens < 0 || n_seqs > h->max_seqs) return SV_ERR_ARG;
  if ((long long)n_tokens * h->q_heads >= (1ll << 31)) return SV_ERR_SIZE;
  if (n_seqs == 0 || n_tokens == 0) return SV_OK;
  int rc;
  if (!cu) return SV_ERR_ARG;
  if ((rc = check_rows(q)) || (rc = check_rows(k)) || (rc = check_rows(v))) return rc;
  if (!out || !aligned16(out)) return SV_ERR_ARG;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const spec_attn_batch batch = {cu, nullptr, nullptr, n_seqs, n_tokens, 0};
  const Batch B = batch_of(h, &batch, nullptr);
  if (h->D == 128) launch_attention<128, false, true>(h, B, Pool{}, rows_of(q), rows_of(k), rows_of(v), 1, scale, out, lse, s);
  else launch_attention<64, false, true>(h, B, Pool{}, rows_of(q), rows_of(k), rows_of(v), 1, scale, out, lse, s);
  return launched();
}

extern "C" int spec_attn_get_error(spec_attn_t h) {
  if (!h) return SV_ERR_ARG;
  int f[2] = {0, 0};
  if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(f, h->d_flags, sizeof f, cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(h->d_flags, 0, sizeof f) != cudaSuccess) {
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return f[1] ? SV_ERR_TIMEOUT : f[0] ? SV_ERR_DATA : SV_OK;
}

extern "C" void spec_attn_destroy(spec_attn_t h) { free_ctx(h); }
