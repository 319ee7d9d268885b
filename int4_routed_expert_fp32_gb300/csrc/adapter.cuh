// Shared by the kernels of the adapter projection (adapter.cu, adapter_shrink.cu,
// adapter_tile.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "tcgen05.cuh"

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

constexpr int kSplitTokens = 256;  // up to here adapter_split_kernel
constexpr int kTileSmemLeast = 168 * 1024;  // above: a CTA of adapter_tile_kernel takes more

// Whether the two kernels of a call with few tokens are laid out to share the SMs
// (T <= kSplitTokens).  Low-rank work that is small beside W: 128 tokens of rank
// 32 with an adapter each take 30 us so and 34 one after the other, 256 of rank 16
// 38 and 50; 256 of rank 32 43 and 38, 128 of rank 64 58 and 45 (K 7168, N 2048 or
// 3584), because little shared memory means few adapters to a pass over x.
inline bool adapter_beside(int T, int R) { return T <= 64 || T * R <= 4096; }

// For tests of the exit paths: the kernel whose copies stop (by a build of its own),
// the stage before which they do, counted per CTA, and the limit of every wait.
struct AdapterStall {
  int kernel;  // 0: the shrink; 1: the projection; 2: the split kernel's copies of B
  int stage;
  long long wait_ns;
};

// low from x, a and scale (adapter_shrink.cu).  Triggers its dependents at once.
int launch_adapter_shrink(const AdapterArgs& a, int* status, cudaStream_t st,
                          const AdapterStall* stall = nullptr);

// The projection with its low-rank term for many tokens (adapter_tile.cu),
// launched as a programmatic dependent of the shrink.
int launch_adapter_tile(const AdapterArgs& a, int* status, cudaStream_t st,
                        const AdapterStall* stall = nullptr);

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

// Dynamic shared memory for a kernel, and all of an SM's L1 as shared memory while it
// runs: the split in force is the first kernel's, and a CTA of the next one that
// wants more of it waits until the SM is empty.
inline cudaError_t adapter_smem(const void* kernel) {
  const cudaError_t e = allow_most_smem(kernel);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

// *size: the largest cluster (at most `most` CTAs) of which the device holds
// `clusters` at a time, or 1: one cluster too many would wait for a whole other one
// to finish.  After adapter_smem.
cudaError_t adapter_cluster(const void* kernel, int threads, int smem, int clusters, int most,
                            int* size);

// Launch attributes: clusters of `ranks` CTAs, programmatic dependent of the
// kernel before it in the stream.
inline void set_adapter_attrs(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int ranks) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = ranks > 0 ? 2 : 1;
}

// Programmatic dependent launch: the dependents may start now; wait until the
// kernel this one depends on has finished and its writes are visible.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A tile of a tensor map on its way to L2.
__device__ __forceinline__ void prefetch_tile_2d(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(c0),
               "r"(c1)
               : "memory");
}

// An id outside [0, adapters) selects none.
__device__ __forceinline__ int checked_id(int id, int adapters) {
  return id >= 0 && id < adapters ? id : -1;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ float ld_cluster_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// hi and lo of v = hi + lo + remainder, both bf16 bits.
__device__ __forceinline__ void split_bf16(float v, uint32_t& hi, uint32_t& lo) {
  hi = f32_to_bf16_bits(v);
  const float h = bf16_bits_to_f32(hi);
  lo = fabsf(h) < INFINITY ? f32_to_bf16_bits(v - h) : 0u;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// By one warp, over the columns [k0, k1): out[j] = x A[j]^T for j < R <= 16 MT.  The
// rows of A are the M side of m16n8k16 MMAs, x the first of the N columns.  A lane's
// 16-byte loads (columns 8 (lane % 4) .. + 7 of a 32-column step) feed two MMAs, of
// which each takes the same columns of both operands, in an order of its own that the
// sum does not see.
template <int MT>
__device__ __forceinline__ void shrink_token(const uint16_t* x, const uint16_t* A, int K, int R,
                                             int k0, int k1, float* out) {
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  float acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
  const uint16_t* ap = A + static_cast<size_t>(g) * K + 8 * q;
  const uint16_t* xp = x + 8 * q;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr int kUnroll = MT == 1 ? 8 : 2;  // ~100 registers of loads
#pragma unroll kUnroll
  for (int k = k0; k < k1; k += 32) {
    uint4 av[MT][2];
    const uint4 xv = g == 0 ? ldg16(xp + k) : zero;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * m + 8 * h;  // R % 8 == 0: all eight rows or none
        av[m][h] = r < R ? ldg16(ap + static_cast<size_t>(r) * K + k) : zero;
      }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mma_bf16(acc[m], av[m][0].x, av[m][1].x, av[m][0].y, av[m][1].y, xv.x, xv.y);
      mma_bf16(acc[m], av[m][0].z, av[m][1].z, av[m][0].w, av[m][1].w, xv.z, xv.w);
    }
  }
  if (q == 0) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (16 * m + 8 * h < R) out[16 * m + 8 * h + g] = acc[m][2 * h];
  }
  __syncwarp();  // whole again for the next token's MMAs
}

}  // namespace moe
