// spec_attn: paged key-value cache and attention around a verification step
// on one GB300 (sm_103a).  The C interface and the method are described in
// include/spec_attn.h; this file holds the kernels and the host side.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "attn_common.cuh"
#include "attn_tile.cuh"
#include "spec_attn.h"

namespace {

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

}  // namespace

// ---------------------------------------------------------------------- host
struct spec_attn_ctx {
  int device, q_heads, kv_heads, D, max_seqs;
  int n_sm;
  int* d_flags;
  float* ws;                         // partial results of the split attention
  int* counters;
};

static void free_ctx(spec_attn_ctx* h) {
  if (!h) return;
  void* ptrs[] = {h->d_flags, h->ws, h->counters};
  for (void* p : ptrs)
    if (p) cudaFree(p);
  free(h);
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

// ---- attention launches
constexpr int MT_MAX = 2;
static size_t ws_bytes(int n_sm, int D) { return (size_t)n_sm * 2 * MT_MAX * (D == 128 ? part_floats<128>() : part_floats<64>()) * sizeof(float); }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return (EncodeTiled)p;
  }();
  return f;
}
// Pool pages as rows of D elements, one page and head a box (64 columns of it for 16-bit elements, which swizzled lines hold)
static bool map_pool(CUtensorMap* m, const spec_attn_ctx* h, const spec_attn_pool* p, void* base) {
  const bool e4m3 = p->dtype == SV_E4M3;
  const cuuint64_t dims[2] = {(cuuint64_t)h->D, (cuuint64_t)p->num_pages * h->kv_heads * p->page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)h->D * (e4m3 ? 1 : 2)};
  const cuuint32_t box[2] = {(cuuint32_t)(e4m3 ? h->D : 64), (cuuint32_t)p->page_size}, step[2] = {1, 1};
  return encode_tiled()(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, e4m3 && h->D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Packed rows [token, head, D]; a box of `tokens` tokens of `box_heads` heads and 64 columns
static bool map_rows(CUtensorMap* m, int D, int heads, const Rows& r, int n_tokens, int box_heads, int tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)n_tokens};
  // a dimension of one element has no stride worth the name
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? r.sh : D) * 2, (cuuint64_t)(n_tokens > 1 ? r.st : (long long)D * heads) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)tokens}, step[3] = {1, 1, 1};
  return encode_tiled()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)r.ptr, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
static bool map_queries(CUtensorMap* m, const spec_attn_ctx* h, const AttnParams& A) {
  return map_rows(m, h->D, h->q_heads, A.Q, A.B.n_tokens, A.group, A.tile_tokens);
}
template <int D, int KIND, int MT>
static bool allow_smem() {
  return cudaFuncSetAttribute(sa_attention_kernel<D, KIND, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, KIND, MT>::SMEM) == cudaSuccess;
}
template <int D>
static bool allow_smem_all() {
  return allow_smem<D, KIND_BF16, 1>() && allow_smem<D, KIND_BF16, 2>() && allow_smem<D, KIND_E4M3, 1>() && allow_smem<D, KIND_PACKED, 2>();
}
template <int D, int KIND, int MT>
static int launch_attention(const spec_attn_ctx* h, const AttnParams& A, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  sa_attention_kernel<D, KIND, MT><<<h->n_sm, Cfg<D, KIND, MT>::THREADS, Cfg<D, KIND, MT>::SMEM, s>>>(A, mq, mk, mv);
  return launched();
}
static AttnParams attn_params(const spec_attn_ctx* h, const Batch& B, const Rows& Q, int causal, float scale, void* out, float* lse) {
  AttnParams A;
  A.B = B; A.Q = Q;
  A.ks = A.vs = nullptr;
  A.q_heads = h->q_heads; A.kv_heads = h->kv_heads; A.group = h->q_heads / h->kv_heads;
  A.tile_tokens = BM / A.group;
  A.causal = causal != 0;
  A.c = fmaxf(scale * LOG2E_F, 1.17549435e-38f);
  A.out = (__nv_bfloat16*)out; A.lse = lse;
  A.ws = h->ws; A.counters = h->counters;
  return A;
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
  if (!encode_tiled() || !(head_dim == 128 ? allow_smem_all<128>() : allow_smem_all<64>())) {
    cudaGetLastError();
    free_ctx(h);
    return SV_ERR_CUDA;
  }
  const size_t counters = (size_t)h->n_sm * MT_MAX * sizeof(int);
  if (cudaMalloc(&h->d_flags, 4 * sizeof(int)) != cudaSuccess || cudaMemset(h->d_flags, 0, 4 * sizeof(int)) != cudaSuccess ||
      cudaMalloc(&h->counters, counters) != cudaSuccess || cudaMemset(h->counters, 0, counters) != cudaSuccess ||
      cudaMalloc(&h->ws, ws_bytes(h->n_sm, head_dim)) != cudaSuccess) {
    cudaGetLastError();
    free_ctx(h);
    return SV_ERR_ALLOC;
  }
  *out = h;
  return SV_OK;
}

extern "C" int spec_attn_chunk(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                               const spec_attn_rows* q, int causal, float scale, void* out, float* lse, void* cuda_stream) {
  if (!h || !(scale > 0.0f) || !isfinite(scale)) return SV_ERR_ARG;
  int rc;
  if ((rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return SV_OK;
  if ((rc = check_rows(q))) return rc;
  if (!out || ((uintptr_t)out & 31)) return SV_ERR_ARG;   // rows leave in 32-byte stores
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const Batch B = batch_of(h, batch, pool);
  AttnParams A = attn_params(h, B, rows_of(q), causal, scale, out, lse);
  CUtensorMap mq, mk, mv;
  if (!map_queries(&mq, h, A)) return SV_ERR_ARG;
  if (!map_pool(&mk, h, pool, pool->k) || !map_pool(&mv, h, pool, pool->v)) return SV_ERR_CUDA;
  if (pool->dtype == SV_E4M3) {
    A.ks = pool->k_scale; A.vs = pool->v_scale;
    return h->D == 128 ? launch_attention<128, KIND_E4M3, 1>(h, A, mq, mk, mv, s) : launch_attention<64, KIND_E4M3, 1>(h, A, mq, mk, mv, s);
  }
  const bool two = (long long)B.n_tokens * A.group > (long long)B.n_seqs * BM;   // more rows per sequence and head than one tile holds
  if (h->D == 128) return two ? launch_attention<128, KIND_BF16, 2>(h, A, mq, mk, mv, s) : launch_attention<128, KIND_BF16, 1>(h, A, mq, mk, mv, s);
  return two ? launch_attention<64, KIND_BF16, 2>(h, A, mq, mk, mv, s) : launch_attention<64, KIND_BF16, 1>(h, A, mq, mk, mv, s);
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
  if (!out || ((uintptr_t)out & 31)) return SV_ERR_ARG;   // rows leave in 32-byte stores
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const spec_attn_batch batch = {cu, nullptr, nullptr, n_seqs, n_tokens, 0};
  const Batch B = batch_of(h, &batch, nullptr);
  const AttnParams A = attn_params(h, B, rows_of(q), 1, scale, out, lse);
  CUtensorMap mq, mk, mv;
  if (!map_queries(&mq, h, A) || !map_rows(&mk, h->D, h->kv_heads, rows_of(k), n_tokens, 1, BN) ||
      !map_rows(&mv, h->D, h->kv_heads, rows_of(v), n_tokens, 1, BN))
    return SV_ERR_ARG;
  return h->D == 128 ? launch_attention<128, KIND_PACKED, 2>(h, A, mq, mk, mv, s) : launch_attention<64, KIND_PACKED, 2>(h, A, mq, mk, mv, s);
}

extern "C" int spec_attn_get_error(spec_attn_t h) {
  if (!h) return SV_ERR_ARG;
  int f[2] = {0, 0};
  if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(f, h->d_flags, sizeof f, cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(h->d_flags, 0, sizeof f) != cudaSuccess ||
      // a call whose wait expired may have left its merge counters behind
      (f[1] && cudaMemset(h->counters, 0, (size_t)h->n_sm * MT_MAX * sizeof(int)) != cudaSuccess)) {
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return f[1] ? SV_ERR_TIMEOUT : f[0] ? SV_ERR_DATA : SV_OK;
}

extern "C" void spec_attn_destroy(spec_attn_t h) { free_ctx(h); }
