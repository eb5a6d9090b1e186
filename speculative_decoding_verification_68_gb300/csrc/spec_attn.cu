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
#include "attn_rotate.cuh"
#include "attn_tile.cuh"
#include "spec_attn.h"

namespace sv_attn {   // spec_attn_few.cu
bool few_init(int D);
int few_launch(const AttnParams& A, const Pool& P, int D, int rows, int n_sm, cudaStream_t s);
}  // namespace sv_attn

namespace {

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
// a launch and the chain of search, page, vector and store.  To e2m1 (attn_rotate.cuh
// has the quantiser) 39.1 us too, 4.8 TB/s: bound by issue, 0.74 of the slots.  A
// lane's 16 elements are a block of one scale; with 8 a lane, and the blocks' and
// vectors' extremes by more shuffles, the same call took 75 us.
template <int D, int POOL>
__global__ void __launch_bounds__(128) sa_append_kernel(Batch B, Pool P, Rows K, Rows V, int heads) {
  constexpr int E = piece_of<POOL != POOL_BF16>, LV = D / E, NL = E / 8;
  flag_invalid_seqs(B);
  const int lane = threadIdx.x & 31, piece = lane % LV;
  const int pieces = 2 * heads * LV;              // keys, then values
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t < B.n_tokens) {
    int slot = 0, pos;
    const int page = find_page(B, t, lane, slot, pos);
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
        if constexpr (POOL == POOL_BF16) {
          if (in) *(uint4*)(dst + (vec * D + piece * E) * 2) = x[u][0];
        } else if constexpr (POOL == POOL_E2M1) {          // a lane's 16 elements share a scale
          uint32_t w[8], z = 0;
          float y[16];
#pragma unroll
          for (int i = 0; i < NL; ++i) {
            w[4 * i] = x[u][i].x; w[4 * i + 1] = x[u][i].y; w[4 * i + 2] = x[u][i].z; w[4 * i + 3] = x[u][i].w;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            z = __vmaxu2(z, w[i] & 0x7fff7fffu);           // magnitudes as bit patterns order like the values
            y[2 * i] = bf_lo(w[i]);
            y[2 * i + 1] = bf_hi(w[i]);
          }
          const uint32_t block = max(z << 16, z & 0xffff0000u);
          uint32_t top = block;
#pragma unroll
          for (int o = LV / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
          const Four f = four_scale(top, block, y, 16);
          if (in) {
            *(uint2*)(dst + vec * (D / 2) + piece * 8) = f.byte == BYTE_NAN ? make_uint2(0, 0) : make_uint2(pack_e2m1(y), pack_e2m1(y + 8));
            (is_v ? P.vb : P.kb)[vec * (D / 16) + piece] = f.scale;
            if (piece == 0) (is_v ? P.vs : P.ks)[vec] = f.byte;
          }
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
// which fill half a sector each, the same call took 60 us.  From e2m1 a lane reads
// 8 bytes and their scale: 35,894 tokens 36.5 us, 5.2 TB/s.
template <int D, int POOL>
__global__ void __launch_bounds__(128) sa_read_kernel(Batch B, Pool P, __nv_bfloat16* ko, __nv_bfloat16* vo, int heads) {
  constexpr bool FP8 = POOL == POOL_E4M3;
  constexpr int E = piece_of<POOL != POOL_BF16>, LV = D / E;
  flag_invalid_seqs(B);
  const int lane = threadIdx.x & 31, piece = lane % LV;
  const int pieces = 2 * heads * LV;              // keys, then values
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t < B.n_tokens) {
    int slot = 0, pos;
    const int page = find_page(B, t, lane, slot, pos);
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
        if constexpr (POOL == POOL_E2M1) {                 // 8 bytes and their scale
          const uint2 c = __ldg((const uint2*)((const char*)(is_v ? P.v : P.k) + vec * (D / 2)) + piece);
          x[u] = make_uint4(c.x, c.y, __ldg((is_v ? P.vb : P.kb) + vec * (D / 16) + piece), 0);
        } else {
          x[u] = ldg_stream((const char*)(is_v ? P.v : P.k) + (vec * D + piece * E) * (FP8 ? 1 : 2));
        }
        if constexpr (POOL != POOL_BF16) {
          const int byte = __ldg((is_v ? P.vs : P.ks) + vec);
          f[u] = byte == 0 ? __int_as_float(1 << 22) : scale_of(byte);   // 2^-127 is subnormal
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vi = (c0 + 32 * u) / LV;
        if (vi >= 2 * heads) continue;
        uint4* const dst = (uint4*)((vi < heads ? kt + vi * D : vt + (vi - heads) * D) + piece * E);
        if constexpr (POOL == POOL_BF16) {
          *dst = x[u];
        } else {
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint32_t r[8], h[8];
          if constexpr (POOL == POOL_E2M1) {               // a code times its scale is exact in f16
            const uint32_t s = e4m3_to_f16x2((uint16_t)(x[u].z | x[u].z << 8));
            e2m1_to_f16(x[u].x, s, h);
            e2m1_to_f16(x[u].y, s, h + 4);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 z = f16x2_to_f32(FP8 ? e4m3_to_f16x2((uint16_t)(w[j >> 1] >> (16 * (j & 1)))) : h[j]);
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
  if (p->dtype != SV_BF16 && p->dtype != SV_E4M3 && p->dtype != SV_E2M1) return SV_ERR_DTYPE;
  if (p->dtype != SV_BF16 && (!p->k_scale || !p->v_scale)) return SV_ERR_ARG;
  if (p->dtype == SV_E2M1 && (!p->k_block || !p->v_block || !aligned16(p->k_block) ||
                              !aligned16(p->v_block) || !aligned16(p->k_scale) || !aligned16(p->v_scale))) return SV_ERR_ARG;
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
// Whether rows that a call writes lie apart: those of the closer stride do, and the other stride steps over all of them.
static bool rows_apart(const spec_attn_rows* r, int D, int n_tokens, int heads) {
  long long near = n_tokens > 1 ? r->token_stride : 0, far = heads > 1 ? r->head_stride : 0, few = n_tokens, many = heads;
  if (near > far) {
    long long x = near; near = far; far = x;
    x = few; few = many; many = x;
  }
  if (few > 1 && near < D) return false;
  return many == 1 || (far >= D && (few == 1 || (far - D) / (few - 1) >= near));
}
// Whether rows that a call writes are other than those it reads from, or the same ones in the same places.
static bool apart_or_in_place(const spec_attn_rows* to, const spec_attn_rows* from, int n_tokens, int heads) {
  return to->ptr != from->ptr || ((n_tokens == 1 || to->token_stride == from->token_stride) && (heads == 1 || to->head_stride == from->head_stride));
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
static Pool pool_of(const spec_attn_pool* p) {
  const bool blocks = p->dtype == SV_E2M1;
  return Pool{p->k, p->v, p->k_scale, p->v_scale, blocks ? p->k_block : nullptr, blocks ? p->v_block : nullptr};
}
static Rows rows_of(const spec_attn_rows* r) { return Rows{(const __nv_bfloat16*)r->ptr, r->token_stride, r->head_stride}; }
static RowsOut out_rows_of(const spec_attn_rows* r) { return RowsOut{(__nv_bfloat16*)r->ptr, r->token_stride, r->head_stride}; }
static int launched() { return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

// Vectors of a token for a warp: all of them where there are tokens enough to fill the GPU, else fewer, a step of
// loads at least.  More warps repeat the search for the page: 2,048 tokens with 64 query heads into an e4m3 cache take
// 18.4 us with 16 warps per SM, 25.7 with 8, 20.9 with 32, 21.7 with 64, and with outputs that L2 does not hold 21.2,
// 28.8, 23.6 and 24.0 (each within 0.1 over repeats in turn; 36K tokens have one split whatever the figure).
constexpr int WARPS_PER_SM = 16;
template <int D, int POOL>
static int launch_rotate(const spec_attn_ctx* h, const Batch& B, const Pool& P, const Turn& T, const Rows& Q, const Rows& K, const Rows& V,
                         const RowsOut& QO, const RowsOut& KO, cudaStream_t s) {
  const int step = 256 / D * UT;
  const int q_heads = QO.ptr ? h->q_heads : 0, all = q_heads + 2 * h->kv_heads, steps = (all + step - 1) / step;
  const long long want = ((long long)h->n_sm * WARPS_PER_SM + B.n_tokens - 1) / B.n_tokens;
  const int per = (steps + (int)(want < steps ? want : steps) - 1) / (int)(want < steps ? want : steps) * step, splits = (all + per - 1) / per;
  const long long warps = (long long)B.n_tokens * splits;
  if (warps > 0x7fffffffll) return SV_ERR_SIZE;
  sa_rotate_kernel<D, POOL><<<(unsigned)((warps + 3) / 4), 128, 0, s>>>(B, P, T, Q, K, V, QO, KO, q_heads, h->kv_heads, splits, per);
  return launched();
}
template <int D>
static int launch_turned(const spec_attn_ctx* h, int dtype, const Batch& B, const Pool& P, const Turn& T, const Rows& Q, const Rows& K, const Rows& V,
                         const RowsOut& QO, const RowsOut& KO, cudaStream_t s) {
  return dtype == SV_E2M1   ? launch_rotate<D, POOL_E2M1>(h, B, P, T, Q, K, V, QO, KO, s)
         : dtype == SV_E4M3 ? launch_rotate<D, POOL_E4M3>(h, B, P, T, Q, K, V, QO, KO, s)
                            : launch_rotate<D, POOL_BF16>(h, B, P, T, Q, K, V, QO, KO, s);
}

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
    if (pool->dtype == SV_E2M1) sa_append_kernel<128, POOL_E2M1><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else if (pool->dtype == SV_E4M3) sa_append_kernel<128, POOL_E4M3><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else sa_append_kernel<128, POOL_BF16><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
  } else {
    if (pool->dtype == SV_E2M1) sa_append_kernel<64, POOL_E2M1><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else if (pool->dtype == SV_E4M3) sa_append_kernel<64, POOL_E4M3><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
    else sa_append_kernel<64, POOL_BF16><<<grid, 128, 0, s>>>(B, P, rows_of(k), rows_of(v), h->kv_heads);
  }
  return launched();
}

extern "C" int spec_attn_append_rotated(spec_attn_t h, const spec_attn_pool* pool, const spec_attn_batch* batch, const spec_attn_rope* rope,
                                        const spec_attn_rows* q, const spec_attn_rows* k, const spec_attn_rows* v,
                                        const spec_attn_rows* q_out, const spec_attn_rows* k_out, void* cuda_stream) {
  int rc;
  if ((rc = check_device(h)) || (rc = check_pool(h, pool)) || (rc = check_batch(h, batch))) return rc;
  if (!rope || !rope->table || !aligned16(rope->table) || rope->max_positions < 1 || !q != !q_out) return SV_ERR_ARG;
  if (rope->rot_dim < 16 || rope->rot_dim > h->D || rope->rot_dim % 16) return SV_ERR_SIZE;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return SV_OK;
  if ((rc = check_rows(k)) || (rc = check_rows(v)) || (q && ((rc = check_rows(q)) || (rc = check_rows(q_out)))) || (k_out && (rc = check_rows(k_out))))
    return rc;
  const int n = batch->n_tokens;
  if (q_out && (!rows_apart(q_out, h->D, n, h->q_heads) || !apart_or_in_place(q_out, q, n, h->q_heads) || q_out->ptr == k->ptr || q_out->ptr == v->ptr))
    return SV_ERR_ARG;
  if (k_out && (!rows_apart(k_out, h->D, n, h->kv_heads) || !apart_or_in_place(k_out, k, n, h->kv_heads) || k_out->ptr == v->ptr ||
                (q && (k_out->ptr == q->ptr || k_out->ptr == q_out->ptr))))
    return SV_ERR_ARG;
  const Turn T = {rope->table, rope->positions, rope->max_positions, rope->rot_dim, rope->interleaved != 0};
  const RowsOut none = {nullptr, 0, 0};
  const Rows Q = q ? rows_of(q) : rows_of(k);
  const RowsOut QO = q ? out_rows_of(q_out) : none, KO = k_out ? out_rows_of(k_out) : none;
  return (h->D == 128 ? launch_turned<128> : launch_turned<64>)(h, pool->dtype, batch_of(h, batch, pool), pool_of(pool), T, Q, rows_of(k), rows_of(v),
                                                                QO, KO, (cudaStream_t)cuda_stream);
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
    if (pool->dtype == SV_E2M1) sa_read_kernel<128, POOL_E2M1><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else if (pool->dtype == SV_E4M3) sa_read_kernel<128, POOL_E4M3><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else sa_read_kernel<128, POOL_BF16><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
  } else {
    if (pool->dtype == SV_E2M1) sa_read_kernel<64, POOL_E2M1><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else if (pool->dtype == SV_E4M3) sa_read_kernel<64, POOL_E4M3><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
    else sa_read_kernel<64, POOL_BF16><<<grid, 128, 0, s>>>(B, P, ko, vo, h->kv_heads);
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
// Pool pages as rows of D elements, one page and head a box (64 columns of it for 16-bit elements, which swizzled
// lines hold); codes go as bytes, in lines of 128, 64 or 32 that are swizzled by their length
static bool map_pool(CUtensorMap* m, const spec_attn_ctx* h, const spec_attn_pool* p, void* base) {
  const bool coded = p->dtype != SV_BF16;
  const cuuint64_t line = p->dtype == SV_E2M1 ? h->D / 2 : h->D;                      // elements of a row
  const cuuint64_t dims[2] = {line, (cuuint64_t)p->num_pages * h->kv_heads * p->page_size};
  const cuuint64_t strides[1] = {line * (coded ? 1 : 2)};
  const cuuint32_t box[2] = {(cuuint32_t)(coded ? line : 64), (cuuint32_t)p->page_size}, step[2] = {1, 1};
  const CUtensorMapSwizzle swizzle = !coded || line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : line == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  return encode_tiled()(m, coded ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  return allow_smem<D, KIND_BF16, 1>() && allow_smem<D, KIND_BF16, 2>() && allow_smem<D, KIND_E4M3, 1>() && allow_smem<D, KIND_E2M1, 1>() && allow_smem<D, KIND_PACKED, 1>() && allow_smem<D, KIND_PACKED, 2>();
}
template <int D, int KIND, int MT>
static int launch_attention(const spec_attn_ctx* h, const AttnParams& A, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  sa_attention_kernel<D, KIND, MT><<<h->n_sm, Cfg<D, KIND, MT>::THREADS, Cfg<D, KIND, MT>::SMEM, s>>>(A, mq, mk, mv);
  return launched();
}
static AttnParams attn_params(const spec_attn_ctx* h, const Batch& B, const Rows& Q, int causal, float scale, void* out, float* lse) {
  AttnParams A;
  A.B = B; A.Q = Q;
  A.ks = A.vs = A.kb = A.vb = nullptr;
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

// Rows of a tile of the kernel for few rows (attn_few.cuh), 0: not for this call.  The mean number of rows of a
// sequence and head decides, and a tile holds a group at least.  Measured, that kernel against the other: 64 single
// tokens over 1000-16000 (8 rows) 174 against 271 us, 2 tokens each (16 rows) 225 against 268; with tiles of 24 and 32
// rows 93 against 70 us for 32 sequences of 3 tokens over 300-5000, 108 against 70 for 4, and in two tiles of 16 longer
// still (32 of 4 over 500-2000: 69 against 45), but for calls of next to nothing (2 of 8 over 500-3000: 18 against 23).
// A batch gets one kernel, whatever its longest sequence: 63 single tokens over 500-8000 and a chunk of 60, 150 or 512
// over 4000 take 149, 211 or 209 us with 32/8 heads and 202, 195 or 245 with 64/8, where two calls, one for the chunk,
// take 164, 162 or 183 and 160, 170 or 218.
static int few_rows(const AttnParams& A) {
  const long long mean = ((long long)A.B.n_tokens * A.group + A.B.n_seqs - 1) / A.B.n_seqs, rows = mean > A.group ? mean : A.group;
  return rows > 16 ? 0 : rows <= 8 ? 8 : 16;
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
  if (!encode_tiled() || !few_init(head_dim) || !(head_dim == 128 ? allow_smem_all<128>() : allow_smem_all<64>())) {
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
  if (!map_queries(&mq, h, A)) return SV_ERR_ARG;     // whatever kernel it is, the same calls are refused
  if (pool->dtype != SV_BF16) {
    A.ks = pool->k_scale; A.vs = pool->v_scale;
  }
  if (pool->dtype == SV_E2M1) {
    A.kb = pool->k_block; A.vb = pool->v_block;
    const int few = few_rows(A);
    if (few) return few_launch(A, pool_of(pool), h->D, few, h->n_sm, s);
  }
  if (!map_pool(&mk, h, pool, pool->k) || !map_pool(&mv, h, pool, pool->v)) return SV_ERR_CUDA;
  if (pool->dtype == SV_E2M1)
    return h->D == 128 ? launch_attention<128, KIND_E2M1, 1>(h, A, mq, mk, mv, s) : launch_attention<64, KIND_E2M1, 1>(h, A, mq, mk, mv, s);
  if (pool->dtype == SV_E4M3)
    return h->D == 128 ? launch_attention<128, KIND_E4M3, 1>(h, A, mq, mk, mv, s) : launch_attention<64, KIND_E4M3, 1>(h, A, mq, mk, mv, s);
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
