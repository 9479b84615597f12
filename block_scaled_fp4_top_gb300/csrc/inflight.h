// The loads that one thread has asked for on an mbarrier, one a phase: which phase the last of them completes. (host code
// too, so that it can be tested without a GPU)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FP4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FP4_HOST_DEVICE inline
#endif

namespace fp4moe {

struct InFlight {
  uint32_t issued = 0;
  FP4_HOST_DEVICE void issue() { ++issued; }
  FP4_HOST_DEVICE bool any() const { return issued != 0; }
  // Parity of the last load's phase: of the (n + 1)-th load on a barrier it is n & 1.
  FP4_HOST_DEVICE uint32_t last() const { return (issued - 1) & 1u; }
};

}  // namespace fp4moe
