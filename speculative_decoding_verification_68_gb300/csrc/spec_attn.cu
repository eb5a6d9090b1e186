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
// Page of token t, and its slot there.  NO_ROW: in no sequence, as the rows that pad a batch are (a wrong cu
// is reported by flag_invalid_seqs); INVALID: in one whose length or page is not valid, which is reported;
// NO_SLOT: before the first position.
enum { NO_SLOT = -1, INVALID = -2, NO_ROW = -3 };
__device__ __forceinline__ int find_page(const Batch& B, int t, int lane, int& slot) {
  const int b = find_seq(B, t, lane);
  int page = NO_ROW;
  if (b >= 0) {
    const int len = __ldg(B.kv_len + b), pos = len - __ldg(B.cu + b + 1) + t;
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
// Pieces of a lane in flight, and warps of a block.  36K tokens appended to e4m3 pools take 40.1 us with 2
// pieces, 47.3 with 4, 40.9 with 1 (8 tokens of 256 sequences 4.8, 5.0, 5.0); 39.1 us with 4 warps a block, 40.8
// with 8, 42.2 with 16.  More loads in flight spread the stores over more pages at once.
constexpr int U = 2;
// A piece is 16 bytes of the pool: 8 bf16 values or 16 codes, D / piece of them a vector.
template <bool FP8> constexpr int piece_of = FP8 ? 16 : 8;

// -------------------------------------------------------------------- append
// x becomes round(x / 2^e) in e4m3, e the least exponent with max|x| <= 448 * 2^e.
// The lanes of a vector find its largest magnitude by a few shuffles.  Bound by
// memory, 2 D bytes read and D + 1 (e4m3) or 2 D written per vector: 35,894
// tokens of 8 heads of 128 to e4m3 take 39.1 us, 5.65 TB/s; a few tokens 2.7 us,
// a launch and the chain of search, page, vector and store.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) sa_append_kernel(Batch B, Pool P, Rows K, Rows V, int heads) {
  constexpr int E = piece_of<FP8>, LV = D / E, NL = E / 8;
  flag_invalid_seqs(B);
  const int lane = threadIdx.x & 31, piece = lane % LV;
  const int pieces = 2 * heads * LV;              // keys, then values
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t < B.n_tokens) {
    int slot = 0;
    const int page = find_page(B, t, lane, slot);
    if (page < 0) return;
    const __nv_bfloat16 *const k = K.ptr + t * K.st + piece * E, *const v = V.ptr + t * V.st + piece * E;
    const long long vec0 = (((long long)page * heads) << B.page_shift) + slot;
    for (int c0 = lane; c0 - lane < pieces; c0 += 32 * U) {   // as often in every lane: the shuffles are warp-wide
      uint4 x[U][NL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vi = (c0 + 32 * u) / LV;
        const __nv_bfloat16* const src = vi < heads ? k + vi * K.sh : v + (vi - heads) * V.sh;
#pragma unroll
        for (int i = 0; i < NL; ++i) x[u][i] = vi < 2 * heads ? ldg_stream(src + 8 * i) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vi = (c0 + 32 * u) / LV;
        const bool in = vi < 2 * heads, is_v = vi >= heads;
        const long long vec = vec0 + ((long long)(is_v ? vi - heads : vi) << B.page_shift);
        char* const dst = (char*)(is_v ? P.v : P.k);
        if constexpr (!FP8) {
          if (in) *(uint4*)(dst + (vec * D + piece * E) * 2) = x[u][0];
        } else {
          // magnitudes as bf16 bit patterns order like the values, infinities and NaN above all
          uint32_t top = 0, c[4];
#pragma unroll
          for (int i = 0; i < NL; ++i) {
            const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
          }
#pragma unroll
          for (int o = LV / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
          // least e with max <= 448 * 2^e = 1.75 * 2^(e + 8)
          const int e = max(EXP_MIN, (int)(top >> 7) - EXP_BIAS - 8 + ((top & 0x7fu) > 0x60u));
          const bool bad = top >= 0x7f80u;
          const float inv = __int_as_float((EXP_BIAS - e) << 23);
#pragma unroll
          for (int i = 0; i < NL; ++i) {
            const uint4 w = x[u][i];
            c[2 * i] = pack_e4m3(bf_lo(w.x) * inv, bf_hi(w.x) * inv, bf_lo(w.y) * inv, bf_hi(w.y) * inv);
            c[2 * i + 1] = pack_e4m3(bf_lo(w.z) * inv, bf_hi(w.z) * inv, bf_lo(w.w) * inv, bf_hi(w.w) * inv);
          }
          if (bad) c[0] = c[1] = c[2] = c[3] = 0x7f7f7f7fu;
          if (in) {
            *(uint4*)(dst + vec * D + piece * E) = make_uint4(c[0], c[1], c[2], c[3]);
            if (piece == 0) (is_v ? P.vs : P.ks)[vec] = (uint8_t)(bad ? BYTE_NAN : e + EXP_BIAS);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------- read
// The reverse of append: code * 2^e, exact in bf16 but below its normal range.
// Bound by memory: 42,403 tokens of 8 heads of 128 from e4m3 take 45.4 us,
// 5.75 TB/s.  A lane's 16 codes leave as one 32-byte store: as two of 16 bytes,
// which fill half a sector each, the same call took 60 us.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) sa_read_kernel(Batch B, Pool P, __nv_bfloat16* ko, __nv_bfloat16* vo, int heads) {
  constexpr int E = piece_of<FP8>, LV = D / E;
  flag_invalid_seqs(B);
  const int lane = threadIdx.x & 31, piece = lane % LV;
  const int pieces = 2 * heads * LV;              // keys, then values
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t < B.n_tokens) {
    int slot = 0;
    const int page = find_page(B, t, lane, slot);
    if (page == NO_ROW) return;
    __nv_bfloat16 *const kt = ko + (size_t)t * heads * D, *const vt = vo + (size_t)t * heads * D;
    if (page < 0) {
      const uint32_t f = page == INVALID ? 0x7fc07fc0u : 0;
      for (int c = lane; c < heads * (D / 8); c += 32) ((uint4*)kt)[c] = ((uint4*)vt)[c] = make_uint4(f, f, f, f);
      return;
    }
    const long long vec0 = (((long long)page * heads) << B.page_shift) + slot;
    for (int c0 = lane; c0 < pieces; c0 += 32 * U) {
      uint4 x[U];
      float f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vi = (c0 + 32 * u) / LV;
        const bool is_v = vi >= heads;
        const long long vec = vec0 + ((long long)(is_v ? vi - heads : vi) << B.page_shift);
        if (vi >= 2 * heads) continue;
        x[u] = ldg_stream((const char*)(is_v ? P.v : P.k) + (vec * D + piece * E) * (FP8 ? 1 : 2));
        if constexpr (FP8) {
          const int byte = __ldg((is_v ? P.vs : P.ks) + vec);
          f[u] = byte == 0 ? __int_as_float(1 << 22) : scale_of(byte);   // 2^-127 is subnormal
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vi = (c0 + 32 * u) / LV;
        if (vi >= 2 * heads) continue;
        uint4* const dst = (uint4*)((vi < heads ? kt + vi * D : vt + (vi - heads) * D) + piece * E);
        if constexpr (!FP8) {
          *dst = x[u];
        } else {
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint32_t r[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 z = f16x2_to_f32(e4m3_to_f16x2((uint16_t)(w[j >> 1] >> (16 * (j & 1)))));
            r[j] = pack_bf16(z.x * f[u], z.y * f[u]);
          }
          st_32(dst, r);
        }
      }
    }
  }
}

}  // namespace

// ---------------------------------------------------------------------- host
struct spec_attn_ctx {
  int device, q_heads, kv_heads, D, max_seqs;
  int n_sm;
  char* memory;                      // one allocation, of
  int* odd;                          // notes on values that are not finite
  int* d_flags;
  int* counters;                     // of the merges
  float* ws;                         // partial results of the split attention
};

static void free_ctx(spec_attn_ctx* h) {
  if (!h) return;
  if (h->memory) cudaFree(h->memory);
  free(h);
}

// Launches, maps and streams are the current device's, the buffers the handle's: the two have to be the same.
static int check_device(const spec_attn_ctx* h) {
  int device;
  if (!h) return SV_ERR_ARG;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return device == h->device ? SV_OK : SV_ERR_ARG;
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
  if (!b || b->n_seqs < 0 || b->n_tokens < 0 || b->max_pages < 0 || b->max_kv < 0 || b->n_seqs > h->max_seqs) return SV_ERR_ARG;
  if (b->n_seqs > 0 && (!b->cu || !b->kv_len || (!b->page_table && b->max_pages > 0))) return SV_ERR_ARG;
  if (b->n_tokens > LEN_MAX || (long long)b->n_tokens * h->q_heads >= (1ll << 31)) return SV_ERR_SIZE;
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
  int rc;
  if ((rc = check_device(h)) || (rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return SV_OK;
  if ((rc = check_rows(k)) || (rc = check_rows(v))) return rc;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const Batch B = batch_of(h, batch, pool);
  const Pool P = pool_of(pool);
  const int grid = (B.n_tokens + 3) / 4;           // four warps a block, a token each
  if (h->D == 128) {
    if (pool->dtype == SV_E4M3) sa_append_kernel<128, true><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else sa_append_kernel<128, false><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
  } else {
    if (pool->dtype == SV_E4M3) sa_append_kernel<64, true><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else sa_append_kernel<64, false><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
  }
  return launched();
}

extern "C" int spec_attn_read(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                              void* k_out, void* v_out, void* cuda_stream) {
  int rc;
  if ((rc = check_device(h)) || (rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return SV_OK;
  if (!k_out || !v_out || ((uintptr_t)k_out | (uintptr_t)v_out) & 31) return SV_ERR_ARG;   // 32-byte stores
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const Batch B = batch_of(h, batch, pool);
  const Pool P = pool_of(pool);
  const int grid = (B.n_tokens + 3) / 4;           // four warps a block, a token each
  __nv_bfloat16 *ko = (__nv_bfloat16*)k_out, *vo = (__nv_bfloat16*)v_out;
  if (h->D == 128) {
    if (pool->dtype == SV_E4M3) sa_read_kernel<128, true><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else sa_read_kernel<128, false><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
  } else {
    if (pool->dtype == SV_E4M3) sa_read_kernel<64, true><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else sa_read_kernel<64, false><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
  }
  return launched();
}

// ---- attention launches
constexpr int MT_MAX = 2;
static size_t ws_bytes(int n_sm, int D) { return (size_t)n_sm * 2 * MT_MAX * (D == 128 ? part_floats<128>() : part_floats<64>()) * sizeof(float); }

static size_t odd_bytes(const spec_attn_ctx* h) { return (size_t)h->n_sm * 4 * 3 * h->D * sizeof(int); }
static size_t small_bytes(const spec_attn_ctx* h) { return 256 + ((size_t)h->n_sm * MT_MAX * sizeof(int) + 255) / 256 * 256; }   // flags, counters

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
  return allow_smem<D, KIND_BF16, 1>() && allow_smem<D, KIND_BF16, 2>() && allow_smem<D, KIND_E4M3, 1>() && allow_smem<D, KIND_PACKED, 1>() && allow_smem<D, KIND_PACKED, 2>();
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
  A.c = fminf(fmaxf(scale * LOG2E_F, 1.17549435e-38f), 3.40282347e38f);   // above 0 and finite, as scale is
  A.out = (__nv_bfloat16*)out; A.lse = lse;
  A.ws = h->ws; A.counters = h->counters; A.odd = h->odd;
  return A;
}

// Two tiles of rows per CTA share every key block, which pays where rows are many and the products bound; one
// tile makes twice as many items.  Measured, one tile against two: 4 chunks of 300-512 tokens over 6000-16000
// cached 298 against 244 us; 8 prompts of 100-2048 tokens 89 against 79 us; but 64 sequences of 8 tokens over
// 500-8000 188 against 230 us, one chunk of 113 over 6096 39 against 51 us, prompts of 25 and 15 tokens 10.6
// against 13.8 us.  The rule: more rows per sequence and head than one tile holds, and at least 12 blocks of two
// tiles for every SM (between 9, where one tile still won, and 14).  `keys`: how many a row sees, about.
constexpr int TWO_TILE_UNITS = 12;
static bool two_tiles(const spec_attn_ctx* h, const AttnParams& A, long long keys) {
  const long long rows = ((long long)A.B.n_tokens * A.group + A.B.n_seqs - 1) / A.B.n_seqs;   // of a sequence and head
  const long long units = A.B.n_seqs * A.kv_heads * ((rows + 2 * BM - 1) / (2 * BM)) * (keys / BN + 1);
  return rows > BM && units >= (long long)TWO_TILE_UNITS * h->n_sm;
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
  // notes at ODD_NONE, flags and counters at 0, both multiples of 256 bytes; the partials need no initial value
  const size_t odd = odd_bytes(h), small = small_bytes(h);
  if (cudaMalloc(&h->memory, odd + small + ws_bytes(h->n_sm, head_dim)) != cudaSuccess || cudaMemset(h->memory, ODD_NONE & 0xff, odd) != cudaSuccess ||
      cudaMemset(h->memory + odd, 0, small) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    free_ctx(h);
    return SV_ERR_ALLOC;
  }
  h->odd = (int*)h->memory;
  h->d_flags = (int*)(h->memory + odd);
  h->counters = h->d_flags + 64;
  h->ws = (float*)(h->memory + odd + small);
  *out = h;
  return SV_OK;
}

extern "C" int spec_attn_chunk(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch,
                               const spec_attn_rows* q, int causal, float scale, void* out, float* lse, void* cuda_stream) {
  if (!h || !(scale > 0.0f) || !isfinite(scale)) return SV_ERR_ARG;
  int rc;
  if ((rc = check_device(h)) || (rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
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
  // The table's width is a poor bound where it has room for the longest sequence of all: a chunk of 113 tokens over
  // 6096 with 64/8 heads of 128 and a table for 131,072 takes 51 us on two tiles, 39 with max_kv given.
  const long long room = (long long)B.max_pages << B.page_shift;
  const bool two = two_tiles(h, A, batch->max_kv > 0 && batch->max_kv < room ? batch->max_kv : room);
  if (h->D == 128) return two ? launch_attention<128, KIND_BF16, 2>(h, A, mq, mk, mv, s) : launch_attention<128, KIND_BF16, 1>(h, A, mq, mk, mv, s);
  return two ? launch_attention<64, KIND_BF16, 2>(h, A, mq, mk, mv, s) : launch_attention<64, KIND_BF16, 1>(h, A, mq, mk, mv, s);
}

extern "C" int spec_attn_prompt(spec_attn_t h, int n_seqs, int n_tokens, const int32_t* cu,
                                const spec_attn_rows* q, const spec_attn_rows* k, const spec_attn_rows* v,
                                float scale, void* out, float* lse, void* cuda_stream) {
  if (!h || !(scale > 0.0f) || !isfinite(scale) || n_seqs < 0 || n_tokens < 0 || n_seqs > h->max_seqs) return SV_ERR_ARG;
  if (n_tokens > LEN_MAX || (long long)n_tokens * h->q_heads >= (1ll << 31)) return SV_ERR_SIZE;
  int rc;
  if ((rc = check_device(h))) return rc;
  if (n_seqs == 0 || n_tokens == 0) return SV_OK;
  if (!cu) return SV_ERR_ARG;
  if ((rc = check_rows(q)) || (rc = check_rows(k)) || (rc = check_rows(v))) return rc;
  if (!out || ((uintptr_t)out & 31)) return SV_ERR_ARG;   // rows leave in 32-byte stores
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const spec_attn_batch batch = {cu, nullptr, nullptr, n_seqs, n_tokens, 0, 0};
  const Batch B = batch_of(h, &batch, nullptr);
  const AttnParams A = attn_params(h, B, rows_of(q), 1, scale, out, lse);
  CUtensorMap mq, mk, mv;
  if (!map_queries(&mq, h, A) || !map_rows(&mk, h->D, h->kv_heads, rows_of(k), n_tokens, 1, BN) ||
      !map_rows(&mv, h->D, h->kv_heads, rows_of(v), n_tokens, 1, BN))
    return SV_ERR_ARG;
  const bool two = two_tiles(h, A, n_tokens / n_seqs / 2);
  if (h->D == 128) return two ? launch_attention<128, KIND_PACKED, 2>(h, A, mq, mk, mv, s) : launch_attention<128, KIND_PACKED, 1>(h, A, mq, mk, mv, s);
  return two ? launch_attention<64, KIND_PACKED, 2>(h, A, mq, mk, mv, s) : launch_attention<64, KIND_PACKED, 1>(h, A, mq, mk, mv, s);
}

extern "C" int spec_attn_get_error(spec_attn_t h) {
  int rc, f[2] = {0, 0};
  if ((rc = check_device(h))) return rc;
  if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(f, h->d_flags, sizeof f, cudaMemcpyDeviceToHost) != cudaSuccess ||
      // a call whose wait expired may have left its merge counters and notes behind
      ((f[0] || f[1]) && cudaMemset(h->d_flags, 0, f[1] ? small_bytes(h) : sizeof f) != cudaSuccess) ||
      (f[1] && cudaMemset(h->odd, ODD_NONE & 0xff, odd_bytes(h)) != cudaSuccess) ||
      cudaDeviceSynchronize() != cudaSuccess) {           // streams that do not wait for the default one may follow
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return f[1] ? SV_ERR_TIMEOUT : f[0] ? SV_ERR_DATA : SV_OK;
}

extern "C" void spec_attn_destroy(spec_attn_t h) { free_ctx(h); }
