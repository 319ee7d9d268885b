// Arguments shared by the kernels of the adapter projection (adapter.cu).
#pragma once

#include <stdint.h>

namespace moe {

struct AdapterArgs {
  const uint16_t* x;   // [T, K]
  const uint16_t* w;   // [N, K]
  const uint16_t* a;   // [adapters, R, K]
  const uint16_t* b;   // [adapters, N, R]
  const int32_t* ids;  // [T]
  const float* scale;  // [adapters] or null
  int T, K, N, R, adapters;
  int slices;         // K slices of the partial low-rank vectors
  const float* part;  // [slices, T, R]: x A^T of each token's adapter
  uint16_t* y;        // [T, N]
};

}  // namespace moe
