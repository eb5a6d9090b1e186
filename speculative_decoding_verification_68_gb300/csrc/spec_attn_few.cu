// Launches of the attention kernel for few rows (attn_few.cuh).
#include <cuda_runtime.h>

#include "attn_few.cuh"
#include "spec_attn.h"

namespace sv_attn {

template <int D, int NTILES>
static bool allow() {
  return cudaFuncSetAttribute(sa_few_kernel<D, NTILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<D, NTILES>::SMEM) == cudaSuccess;
}
bool few_init(int D) {
  return D == 128 ? allow<128, 1>() && allow<128, 2>() : allow<64, 1>() && allow<64, 2>();
}

template <int D, int NTILES>
static int launch(AttnParams A, const Pool& P, int n_sm, cudaStream_t s) {
  A.tile_tokens = 8 * NTILES / A.group;
  const int grid = n_sm < MAX_CTAS ? n_sm : MAX_CTAS;
  sa_few_kernel<D, NTILES><<<grid, Few<D, NTILES>::THREADS, Few<D, NTILES>::SMEM, s>>>(A, (const uint8_t*)P.k, (const uint8_t*)P.v);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
// rows: 8 or 16 that a tile holds, at least a group
int few_launch(const AttnParams& A, const Pool& P, int D, int rows, int n_sm, cudaStream_t s) {
  if (D == 128) return rows == 8 ? launch<128, 1>(A, P, n_sm, s) : launch<128, 2>(A, P, n_sm, s);
  return rows == 8 ? launch<64, 1>(A, P, n_sm, s) : launch<64, 2>(A, P, n_sm, s);
}

}  // namespace sv_attn
