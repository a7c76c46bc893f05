// Argument checks shared by the entry points' translation units (host code).
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/sgqa.h"

namespace sgqa {

extern int g_test_stall_cta;  // sgqa_test_stall_decode_cta (failure-detection tests only)

inline bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_dims(const sgqa_dims* d) {
  if (!d) return SGQA_ERR_INVALID_ARG;
  if (d->batch <= 0 || d->T <= 0 || d->Hq <= 0 || d->G <= 0 || d->d <= 0 || d->d_idx <= 0 || d->B <= 0 ||
      d->k <= 0)
    return SGQA_ERR_INVALID_ARG;
  if (d->T >= (1 << 28) || d->batch > 65535) return SGQA_ERR_UNSUPPORTED;
  // row indices of q, gate, out and q_idx (and TMA coordinates) are 32-bit
  if ((long)d->batch * d->T * (d->Hq > d->G ? d->Hq : d->G) >= (1L << 31)) return SGQA_ERR_UNSUPPORTED;
  if (d->d != 64 && d->d != 128) return SGQA_ERR_UNSUPPORTED;
  if (d->d_idx != 32 && d->d_idx != 64) return SGQA_ERR_UNSUPPORTED;
  if (d->B != 1 && d->B != 2 && d->B != 4 && d->B != 8 && d->B != 16) return SGQA_ERR_UNSUPPORTED;
  if (d->k % d->B != 0) return SGQA_ERR_UNSUPPORTED;
  if (d->Hq % d->G != 0 || d->Hq / d->G > 16 || 128 % d->G != 0) return SGQA_ERR_UNSUPPORTED;
  if (d->k / d->B > 16384) return SGQA_ERR_UNSUPPORTED;
  return SGQA_OK;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA; }

}  // namespace sgqa
