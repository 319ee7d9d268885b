// A shared projection with the low-rank adapters of many requests:
//   y[t] = x[t] W^T + s_a (x[t] A_a^T) B_a^T,  a = ids[t]  (-1: no adapter),
// x bf16 [T, K], W bf16 [N, K], A bf16 [adapters, R, K], B bf16 [adapters, N,
// R], y bf16 [T, N]; fp32 accumulation, one rounding of the sum.  The
// projections it stands beside are the latent ones and the shared expert's
// ("Kimi K3 latent up-projection" page, KimiSparseMoeBlock listing); no page
// has adapters.
//
// Two launches.  The shrink (adapter_shrink.cu) forms p = s x A^T for each
// token's own adapter, in fp32.  A projection kernel forms x W^T on the tensor cores and
// adds p B^T before its one rounding.  It is launched as a programmatic
// dependent: it streams W while the shrink still runs and waits for p only
// when it needs it.
//
// A few tokens of low rank take one launch: there the shrink is a small part of
// the projection kernel's own K ranges, done by warps that are idle meanwhile.
// Each kernel lets the next call's first kernel start early, and waits for its
// predecessor before it reads anything.
//
//  - adapter_split_kernel, few tokens: bound by reading W.  128 rows of W are
//    the MMA's M side and up to 256 tokens its N side; the K range is split
//    over the CTAs of a cluster, which add their accumulators through
//    distributed shared memory in the order of their ranks, so that 100 and
//    more SMs stream W whatever N is.  The low-rank term is a dot product of
//    length R per output, with each token's own rows of B.
//  - adapter_tile_kernel (adapter_tile.cu), many tokens: bound by the tensor
//    cores; the low-rank term is R more columns of K for each adapter that
//    occurs in an output tile's rows.
#include <math.h>

#include <algorithm>

#include "adapter.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kMaxRank = 128;

constexpr int kSpThreads = 256;  // warp 0: TMA, 1: MMA + TMEM, 2-5: TMEM -> smem; all: the sums
constexpr int kSpWBytes = 128 * 64 * 2;
constexpr int kSpMaxCluster = 8;

// Up to here the split kernel does the shrink itself: every output tile reads the
// adapters' A again (T R of them in place of 128 rows of W a tile).
constexpr int kFusedLow = 64;  // T R
constexpr int kLowWarps = 6;   // warps 2-7

struct SplitShape {
  int tb;      // tokens to a block (the MMA's N), a multiple of 16
  int stages;
  int cluster;  // CTAs that share an output tile, each with its K range
  uint32_t cols;  // TMEM columns
  size_t smem;
};

}  // namespace

// FUSED: the low-rank vectors too (T R <= kFusedLow, one block of tokens).
// Cluster (x = rank, y, z): rows 128 y of W, tokens tb z; rank j takes the
// K steps [j n / cluster, (j + 1) n / cluster) of n = ceil(K / 64).
template <bool FUSED>
__global__ void __launch_bounds__(kSpThreads, 1)
    adapter_split_kernel(const __grid_constant__ CUtensorMap mw,
                         const __grid_constant__ CUtensorMap mx, const AdapterArgs a, int tb,
                         int stages, uint32_t cols, int* status, long long wait_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[8], empty[8], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int cta_abort;
  __shared__ float lowp[kLowWarps + 1][kFusedLow];  // FUSED: the warps' sums, and the CTA's
  __shared__ __align__(16) float lowv[kFusedLow];   // FUSED: scaled, of all ranks
  __shared__ int16_t low_rows[8];
  const Waiter wt{&cta_abort, status, wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = kSpWBytes + tb * 128;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    cta_abort = 0;
    fence_mbarrier_init();
  }
  if (FUSED && threadIdx.x < 8) low_rows[threadIdx.x] = 0;
  if (warp == 1) {
    tmem_alloc(&tmem_slot, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;
  if (FUSED) grid_wait();
  grid_launch_dependents();
  const int ranks = gridDim.x, rank = blockIdx.x;
  const int n0 = blockIdx.y * 128, t0 = blockIdx.z * tb;
  const int tokens = min(tb, a.T - t0);
  const int steps = (a.K + 63) / 64;
  const int s0 = steps * rank / ranks, s1 = steps * (rank + 1) / ranks;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensor_map(&mw);
      prefetch_tensor_map(&mx);
      uint32_t it = 0;
      for (int k = s0; k < s1; ++k, ++it) {
        const int s = it % stages;
        if (!mbar_wait(&empty[s], ((it / stages) & 1u) ^ 1u, wt)) break;
        uint8_t* st = smem + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        tma_g2s_2d(st, &mw, &full[s], k * 64, n0);
        tma_g2s_2d(st + kSpWBytes, &mx, &full[s], k * 64, t0);
      }
      drain_ring(full, it, stages, status);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16(128, tb);
    uint32_t it = 0;
    for (int k = s0; k < s1; ++k, ++it) {
      const int s = it % stages;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (it / stages) & 1u, wt))) break;
      tc_fence_after();
      const uint8_t* st = smem + s * stage_bytes;
      const uint64_t da = smem_desc_sw128(st);
      const uint64_t db = smem_desc_sw128(st + kSpWBytes);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_f16_warp(tbase, da + 2 * kk, db + 2 * kk, idesc, (it | kk) != 0);
      umma_commit_warp(&empty[s]);
    }
    umma_commit_warp(&done);
    mbar_drain(&done, 0, status);
  } else {
    // B of this rank's tokens on its way to L2 while W streams
    const int rows = min(128, a.N - n0);
    for (int j = warp - 2; j * ranks + rank < tokens; j += kLowWarps) {
      const int id = checked_id(a.ids[t0 + j * ranks + rank], a.adapters);
      if (id < 0) continue;
      const uint16_t* b = a.b + (static_cast<size_t>(id) * a.N + n0) * a.R;
      for (int e = lane * 64; e < rows * a.R; e += 32 * 64)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(b + e));
    }
    if (FUSED) {
      // this rank's columns, dealt to the warps in whole 32-column steps
      const int k0 = s0 * 2, k1 = min(s1 * 2, a.K / 32);
      const int w = warp - 2;
      const int a0 = (k0 + (k1 - k0) * w / kLowWarps) * 32;
      const int a1 = (k0 + (k1 - k0) * (w + 1) / kLowWarps) * 32;
      for (int t = 0; t < tokens; ++t) {
        const int id = checked_id(a.ids[t], a.adapters);
        if (id != a.ids[t] && a.ids[t] != -1) record_status(status, MOE_ERR_INVALID);
        if (id < 0) continue;
        const uint16_t* A = a.a + static_cast<size_t>(id) * a.R * a.K;
        const uint16_t* x = a.x + static_cast<size_t>(t) * a.K;
        float* out = &lowp[w][t * a.R];
        if (a.R <= 16)
          shrink_item<1, 1>(x, A, a.K, a.R, low_rows, 1, a0, a1, out);
        else
          shrink_item<4, 1>(x, A, a.K, a.R, low_rows, 1, a0, a1, out);
      }
    }
  }
  // every copy has landed and every MMA is done: the ring becomes the fp32
  // tile [tokens][128 columns of y]
  __syncthreads();
  mbar_drain(&done, 0, status);  // complete: each reader observes it for itself
  tc_fence_after();
  float* red = reinterpret_cast<float*>(smem);
  if (warp >= 2 && warp < 6) {
    const int q = warp & 3;
    for (int c0 = 0; c0 < tb; c0 += 16) {
      uint32_t r[16];
      tmem_ld16(tbase + (static_cast<uint32_t>(32 * q) << 16) + c0, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) red[(c0 + i) * 128 + 32 * q + lane] = __uint_as_float(r[i]);
    }
  }
  if (FUSED && threadIdx.x < tokens * a.R) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kLowWarps; ++w) v += lowp[w][threadIdx.x];
    lowp[kLowWarps][threadIdx.x] = v;
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, cols);
  }
  if (FUSED) {
    if (threadIdx.x < tokens * a.R) {
      const int id = checked_id(a.ids[threadIdx.x / a.R], a.adapters);
      float v = 0.f;
      if (id >= 0) {
        for (int r = 0; r < ranks; ++r)
          v += ld_cluster_f1(mapa_shared(&lowp[kLowWarps][threadIdx.x], r));
        if (a.scale) v *= a.scale[id];
      }
      lowv[threadIdx.x] = v;
    }
    __syncthreads();
  } else {
    grid_wait();  // the low-rank vectors are complete
  }
  // token by token: rank r takes tokens r, r + ranks, ... in turn with its
  // warps; a lane sums four columns over the cluster, in the order of the ranks
  const int n = n0 + 4 * lane;
  const bool on = n < a.N;  // N % 8 == 0: all four columns or none
  constexpr int kStep = kSpThreads / 32;
  int id = -1, next = -1;
  if (warp * ranks + rank < tokens) next = checked_id(a.ids[t0 + warp * ranks + rank], a.adapters);
  for (int i = warp * ranks + rank; i < tokens; i += ranks * kStep) {
    id = next;
    if (i + ranks * kStep < tokens) next = checked_id(a.ids[t0 + i + ranks * kStep], a.adapters);
    float4 o[kSpMaxCluster];
#pragma unroll
    for (int r = 0; r < kSpMaxCluster; ++r)
      if (r < ranks) o[r] = ld_cluster_f4(mapa_shared(red + i * 128 + 4 * lane, r));
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (id >= 0 && on) {
      const uint16_t* b = a.b + (static_cast<size_t>(id) * a.N + n) * a.R;
      const float* l = FUSED ? lowv + i * a.R : a.low + static_cast<size_t>(t0 + i) * a.R;
#pragma unroll 2
      for (int j = 0; j < a.R; j += 8) {
        const float4 l0 = *reinterpret_cast<const float4*>(l + j);
        const float4 l1 = *reinterpret_cast<const float4*>(l + j + 4);
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = ldg16(b + c * a.R + j);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[c] = fmaf(__uint_as_float(w[c].x << 16), l0.x, s[c]);
          s[c] = fmaf(__uint_as_float(w[c].x & 0xffff0000u), l0.y, s[c]);
          s[c] = fmaf(__uint_as_float(w[c].y << 16), l0.z, s[c]);
          s[c] = fmaf(__uint_as_float(w[c].y & 0xffff0000u), l0.w, s[c]);
          s[c] = fmaf(__uint_as_float(w[c].z << 16), l1.x, s[c]);
          s[c] = fmaf(__uint_as_float(w[c].z & 0xffff0000u), l1.y, s[c]);
          s[c] = fmaf(__uint_as_float(w[c].w << 16), l1.z, s[c]);
          s[c] = fmaf(__uint_as_float(w[c].w & 0xffff0000u), l1.w, s[c]);
        }
      }
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kSpMaxCluster; ++r)
      if (r < ranks) {
        v.x += o[r].x; v.y += o[r].y; v.z += o[r].z; v.w += o[r].w;
      }
    if (on) {
      uint2 q;
      q.x = f32_to_bf16_bits(v.x + s[0]) |
            (static_cast<uint32_t>(f32_to_bf16_bits(v.y + s[1])) << 16);
      q.y = f32_to_bf16_bits(v.z + s[2]) |
            (static_cast<uint32_t>(f32_to_bf16_bits(v.w + s[3])) << 16);
      *reinterpret_cast<uint2*>(a.y + static_cast<size_t>(t0 + i) * a.N + n) = q;
    }
  }
  cluster_sync_all();  // no CTA leaves while another reads its tile
}

namespace {

SplitShape split_shape(int T, int K, int N) {
  SplitShape s;
  const int blocks = (T + 255) / 256;
  s.tb = ((T + blocks - 1) / blocks + 15) / 16 * 16;
  const int tiles = (N + 127) / 128 * blocks;
  const int steps = (K + 63) / 64;
  // at most one CTA to an SM: a second one on some would take twice the time
  s.cluster = std::min(std::max(1, std::min(kSpMaxCluster, num_sms() / tiles)), steps);
  const int stage = kSpWBytes + s.tb * 128;
  const int budget = s.tb <= 64 ? 104 * 1024 : 204 * 1024;
  s.stages = std::min(8, budget / stage);
  s.cols = 32;
  while (s.cols < static_cast<uint32_t>(s.tb)) s.cols *= 2;
  s.smem = std::max<size_t>(static_cast<size_t>(s.stages) * stage, static_cast<size_t>(s.tb) * 512) +
           1024;
  return s;
}

template <bool FUSED>
int launch_split(const AdapterArgs& a, int* status, cudaStream_t st) {
  const SplitShape sh = split_shape(a.T, a.K, a.N);
  CUtensorMap mw, mx;
  if (!adapter_map_rows(&mw, a.w, a.N, a.K, 128) || !adapter_map_rows(&mx, a.x, a.T, a.K, sh.tb)) return MOE_ERR_CUDA;
  auto kern = adapter_split_kernel<FUSED>;
  MOE_TRY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(sh.smem)));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sh.cluster, (a.N + 127) / 128, (a.T + sh.tb - 1) / sh.tb);
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = sh.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  set_adapter_attrs(&cfg, attr, sh.cluster);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kern, mw, mx, a, sh.tb, sh.stages, sh.cols, status,
                                  static_cast<long long>(kDefaultWaitNs)));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_adapter_linear_workspace_size(int T, int K, int N, int R) {
  (void)K;
  (void)N;
  if (T <= 0 || R <= 0) return 256;
  return align_up(static_cast<size_t>(T) * R * sizeof(float), 256);
}

extern "C" int moe_adapter_linear(const uint16_t* x, const uint16_t* w, const uint16_t* lora_a,
                                  const uint16_t* lora_b, const int32_t* ids, const float* scale,
                                  int T, int K, int N, int R, int adapters, uint16_t* y, void* ws,
                                  size_t ws_bytes, void* stream) {
  moe::Range range_("moe_adapter_linear");
  if (T < 0 || K <= 0 || N <= 0 || R <= 0 || adapters <= 0) return MOE_ERR_INVALID;
  if (K % 32 != 0 || N % 8 != 0 || R % 8 != 0 || R > kMaxRank) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w || !lora_a || !lora_b || !ids || !y || !ws) return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16) ||
      !aligned(ids, 4) || !aligned(scale, 4) || !aligned(y, 16) || !aligned(ws, 256))
    return MOE_ERR_INVALID;
  if (ws_bytes < moe_adapter_linear_workspace_size(T, K, N, R)) return MOE_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return MOE_ERR_CUDA;
  AdapterArgs a{};
  a.x = x;
  a.w = w;
  a.a = lora_a;
  a.b = lora_b;
  a.ids = ids;
  a.scale = scale;
  a.T = T;
  a.K = K;
  a.N = N;
  a.R = R;
  a.adapters = adapters;
  a.low = static_cast<float*>(ws);
  a.y = y;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T * R <= kFusedLow && T <= 8) return launch_split<true>(a, status, st);
  const int rc = launch_adapter_shrink(a, status, st);
  if (rc) return rc;
  return T > kSplitTokens ? launch_adapter_tile(a, status, st) : launch_split<false>(a, status, st);
}
