// Shared by the kernels of the adapter projection (adapter.cu, adapter_shrink.cu,
// adapter_tile.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

struct AdapterArgs {
  const uint16_t* x;   // [T, K]
  const uint16_t* w;   // [N, K]
  const uint16_t* a;   // [adapters, R, K]
  const uint16_t* b;   // [adapters, N, R]
  const int32_t* ids;  // [T]
  const float* scale;  // [adapters] or null
  int T, K, N, R, adapters;
  float* low;   // [T, R]: scale x A^T of each token's adapter
  uint16_t* y;  // [T, N]
};

constexpr int kSplitTokens = 256;  // up to here adapter_split_kernel, one block of tokens

// low from x, a and scale (adapter_shrink.cu).  Triggers its dependents at once.
int launch_adapter_shrink(const AdapterArgs& a, int* status, cudaStream_t st);

// The projection with its low-rank term for many tokens (adapter_tile.cu),
// launched as a programmatic dependent of the shrink.
int launch_adapter_tile(const AdapterArgs& a, int* status, cudaStream_t st);

// Tensor map of [rows][cols] bf16: boxes of 64 columns and box_rows rows, with
// the 128-byte swizzle.
inline bool adapter_map_rows(CUtensorMap* m, const uint16_t* base, int rows, int cols,
                             int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(cols) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

// Programmatic dependent launch: the dependents may start now; wait until the
// kernel this one depends on has finished and its writes are visible.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// An id outside [0, adapters) selects none.
__device__ __forceinline__ int checked_id(int id, int adapters) {
  return id >= 0 && id < adapters ? id : -1;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

}  // namespace moe
