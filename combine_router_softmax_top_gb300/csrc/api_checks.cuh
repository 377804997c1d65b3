// Argument checks of the C entry points (api.cu, fp8_api.cu, fp4_api.cu, norm.cu).
#pragma once

#include "moe_internal.cuh"

#define MOE_CHECK(x)                  \
  do {                                \
    moe_status_t _s = (x);            \
    if (_s != MOE_OK) return _s;      \
  } while (0)

#define MOE_ALIGNED(p, n)                                         \
  do {                                                            \
    if (reinterpret_cast<uintptr_t>(p) & ((n) - 1)) {             \
      moe::set_error("%s is not %d-byte aligned", #p, (int)(n));  \
      return MOE_ERR_INVALID_ARG;                                 \
    }                                                             \
  } while (0)

#define MOE_PTR_N(p, n)                      \
  do {                                       \
    if (!(p)) {                              \
      moe::set_error("%s is NULL", #p);      \
      return MOE_ERR_INVALID_ARG;            \
    }                                        \
    MOE_ALIGNED(p, n);                       \
  } while (0)

#define MOE_PTR(p) MOE_PTR_N(p, 16)
#define MOE_PTR_OPT(p) MOE_ALIGNED(p, 16)
// rows that the expert products move in whole 32-byte sectors
#define MOE_PTR32(p) MOE_PTR_N(p, 32)
#define MOE_PTR32_OPT(p) MOE_ALIGNED(p, 32)
