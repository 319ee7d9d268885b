// A shared projection with the low-rank adapters of many requests:
//   y[t] = x[t] W^T + s_a (x[t] A_a^T) B_a^T,  a = ids[t]  (-1: no adapter),
// x bf16 [T, K], W bf16 [N, K], A bf16 [adapters, R, K], B bf16 [adapters, N,
// R], y bf16 [T, N]; fp32 accumulation, one rounding of the sum.  The
// projections it stands beside are the latent ones and the shared expert's
// ("Kimi K3 latent up-projection" page, KimiSparseMoeBlock listing); no page
// has adapters.
//
// Two launches.  adapter_shrink_kernel forms p = x A^T for each token's own
// adapter, as fp32 partial sums over slices of K.  A projection kernel forms
// x W^T on the tensor cores and adds s p B^T before its one rounding.  It is
// launched as a programmatic dependent: it streams W while the shrink still
// runs and waits for the partials only when it needs them.
//
//  - adapter_split_kernel, few tokens: bound by reading W.  128 rows of W are
//    the MMA's M side and up to 256 tokens its N side; the K range is split
//    over the CTAs of a cluster, which add their accumulators through
//    distributed shared memory in the order of their ranks, so that 100 and
//    more SMs stream W whatever N is.  The low-rank term is a dot product of
//    length R per output, with each token's own rows of B.
//  - adapter_tile_kernel, many tokens: bound by the tensor cores.  Persistent
//    128 x 256 output tiles; the low-rank term is R more columns of K: for
//    each adapter that occurs in the tile's 128 rows, an A operand of the rows
//    that use it (zero elsewhere) and its rows of B.
#include <math.h>

#include <algorithm>

#include "adapter.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kAdTile = 128;    // tokens to a shrink CTA, and rows of an output tile
constexpr int kMaxRank = 128;

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

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

// ------------------------------------------------------------------- shrink

constexpr int kShWarps = 8;

struct ShrinkArgs {
  const uint16_t* x;
  const uint16_t* a;
  const int32_t* ids;
  int T, K, R, adapters;
  int slices;  // K slices, of whole 32-column steps
  float* part;  // [slices, T, R]
  int* status;
};

// The rows of a tile, grouped by adapter: unit u holds rows
// row[start[u]] .. row[start[u + 1] - 1], all of adapter id[u].
struct Units {
  int32_t ids[kAdTile];
  int16_t row[kAdTile];
  int16_t start[kAdTile + 1];
  int32_t id[kAdTile];
  int n;
};

// Groups the tile's rows (threads 0 .. 127, all threads call): a row's place
// is counted against the other 127 rows, in their order.
__device__ void group_rows(Units& u, const int32_t* ids, int t0, int rows, int adapters,
                           int* status, bool report) {
  const int i = threadIdx.x;
  if (i < kAdTile) {
    int id = -1;
    if (i < rows) {
      const int raw = ids[t0 + i];
      id = checked_id(raw, adapters);
      if (report && id != raw) record_status(status, MOE_ERR_INVALID);
    }
    u.ids[i] = id;
  }
  __syncthreads();
  if (i < kAdTile) {
    const int id = u.ids[i];
    int before = 0, lower = 0;  // sorted by id, rows of one id in their order
    for (int j = 0; j < kAdTile; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(&u.ids[j]);
      const int v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        lower += v[q] >= 0 && v[q] < id ? 1 : 0;
        before += v[q] == id && j + q < i ? 1 : 0;
      }
    }
    if (id >= 0) u.row[lower + before] = static_cast<int16_t>(i);
  }
  __syncthreads();
  // sorted position p starts a unit when its row's adapter differs from p - 1's
  if (i < 32) {
    int valid = 0;
    for (int j = i; j < kAdTile; j += 32) valid += u.ids[j] >= 0 ? 1 : 0;
    valid = __reduce_add_sync(0xffffffffu, valid);
    int n = 0;
    for (int p0 = 0; p0 < valid; p0 += 32) {
      const int p = p0 + i;
      const bool on = p < valid;
      const int id = on ? u.ids[u.row[p]] : -1;
      const int prev = on && p > 0 ? u.ids[u.row[p - 1]] : -1;
      const bool lead = on && (p == 0 || id != prev);
      const uint32_t m = __ballot_sync(0xffffffffu, lead);
      if (lead) {
        const int at = n + __popc(m & ((1u << i) - 1));
        u.start[at] = static_cast<int16_t>(p);
        u.id[at] = id;
      }
      n += __popc(m);
    }
    if (i == 0) {
      u.n = n;
      u.start[n] = static_cast<int16_t>(valid);
    }
  }
  __syncthreads();
}

// p[r][j] over one K range for up to 8 NT rows of one unit and 16 MT rows of A:
// the rows of A are the M side of m16n8k16 MMAs, tokens the N side.  A lane's
// 16-byte loads (columns 8 (lane % 4) .. + 7 of a 32-column step) feed two MMAs
// of which each takes the same columns of both operands, in an order of its
// own that the sum does not see.
template <int MT, int NT>
__device__ __forceinline__ void shrink_unit(const ShrinkArgs& s, const uint16_t* A, int r0,
                                            const int16_t* rows, int c, int t0, int k0, int k1,
                                            float (*red)[16 * MT][8 * NT], float* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
  const uint16_t* ap[MT][2];
  bool aon[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + 16 * m + 8 * h + g;
      aon[m][h] = r < s.R;
      ap[m][h] = A + static_cast<size_t>(aon[m][h] ? r : 0) * s.K + 8 * q;
    }
  const uint16_t* xp[NT];
  bool xon[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xon[n] = 8 * n + g < c;
    xp[n] = s.x + static_cast<size_t>(t0 + (xon[n] ? rows[8 * n + g] : 0)) * s.K + 8 * q;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
  for (int k = k0 + 32 * warp; k < k1; k += 32 * kShWarps) {
    uint4 av[MT][2], xv[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) av[m][h] = aon[m][h] ? ldg16(ap[m][h] + k) : zero;
#pragma unroll
    for (int n = 0; n < NT; ++n) xv[n] = xon[n] ? ldg16(xp[n] + k) : zero;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_bf16(acc[m][n], av[m][0].x, av[m][1].x, av[m][0].y, av[m][1].y, xv[n].x, xv[n].y);
        mma_bf16(acc[m][n], av[m][0].z, av[m][1].z, av[m][0].w, av[m][1].w, xv[n].z, xv[n].w);
      }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[warp][16 * m + g + 8 * (i >> 1)][8 * n + 2 * q + (i & 1)] = acc[m][n][i];
  __syncthreads();
  const int nr = min(16 * MT, s.R - r0);
  for (int i = threadIdx.x; i < nr * c; i += 32 * kShWarps) {
    const int n = i / nr, r = i - n * nr;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kShWarps; ++w) v += red[w][r][n];
    out[static_cast<size_t>(t0 + rows[n]) * s.R + r0 + r] = v;
  }
  __syncthreads();
}

}  // namespace

// CTA (m, z, u): tokens of tile m, K slice z, units u, u + gridDim.z, ...
template <int MT>
__global__ void __launch_bounds__(32 * kShWarps) adapter_shrink_kernel(const ShrinkArgs s) {
  grid_launch_dependents();
  extern __shared__ __align__(16) uint8_t sh_smem[];
  __shared__ __align__(16) Units u;
  const int t0 = blockIdx.x * kAdTile;
  group_rows(u, s.ids, t0, min(kAdTile, s.T - t0), s.adapters, s.status,
             blockIdx.y == 0 && blockIdx.z == 0);
  const int steps = s.K / 32;  // K % 32 == 0
  const int k0 = static_cast<int>(static_cast<long long>(steps) * blockIdx.y / s.slices) * 32;
  const int k1 = static_cast<int>(static_cast<long long>(steps) * (blockIdx.y + 1) / s.slices) * 32;
  float* out = s.part + static_cast<size_t>(blockIdx.y) * s.T * s.R;
  for (int i = blockIdx.z; i < u.n; i += gridDim.z) {
    const uint16_t* A = s.a + static_cast<size_t>(u.id[i]) * s.R * s.K;
    const int first = u.start[i], end = u.start[i + 1];
    for (int p = first; p < end;) {
      const int left = end - p;
      for (int r0 = 0; r0 < s.R; r0 += 16 * MT) {
        if (left <= 8)
          shrink_unit<MT, 1>(s, A, r0, u.row + p, left, t0, k0, k1,
                             reinterpret_cast<float(*)[16 * MT][8]>(sh_smem), out);
        else
          shrink_unit<MT, 4>(s, A, r0, u.row + p, min(left, 32), t0, k0, k1,
                             reinterpret_cast<float(*)[16 * MT][32]>(sh_smem), out);
      }
      p += left <= 8 ? left : min(left, 32);
    }
  }
}

namespace {

// The low-rank vector of token t, scaled, into v[0 .. R) (a whole warp).
__device__ __forceinline__ void load_low(const AdapterArgs& a, int t, int id, float* v) {
  const float sc = a.scale ? a.scale[id] : 1.f;
  for (int j = threadIdx.x & 31; j < a.R; j += 32) {
    float s = 0.f;
    for (int z = 0; z < a.slices; ++z)
      s += a.part[(static_cast<size_t>(z) * a.T + t) * a.R + j];
    v[j] = s * sc;
  }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

constexpr int kSpThreads = 256;  // warp 0: TMA, 1: MMA + TMEM, 2-5: TMEM -> smem; all: the sums
constexpr int kSpWBytes = 128 * 64 * 2;
constexpr int kSpMaxCluster = 8;

struct SplitShape {
  int tb;      // tokens to a block (the MMA's N), a multiple of 16
  int stages;
  int cluster;  // CTAs that share an output tile, each with its K range
  uint32_t cols;  // TMEM columns
  size_t smem;
};

}  // namespace

// Cluster (x = rank, y, z): rows 128 y of W, tokens tb z; rank j takes the
// K steps [j n / cluster, (j + 1) n / cluster) of n = ceil(K / 64).
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
  __shared__ float low[kSpThreads / 32][kMaxRank];
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
  if (warp == 1) {
    tmem_alloc(&tmem_slot, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;
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
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, cols);
  }
  grid_wait();  // the partial low-rank vectors are complete
  // token by token: rank r takes tokens r, r + ranks, ... in turn with its
  // warps; a lane sums four columns over the cluster, in the order of the ranks
  const int n = n0 + 4 * lane;
  for (int i = warp * ranks + rank; i < tokens; i += ranks * (kSpThreads / 32)) {
    const int t = t0 + i;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < ranks; ++r) {
      const float4 o = ld_cluster_f4(mapa_shared(red + i * 128 + 4 * lane, r));
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
    const int id = checked_id(a.ids[t], a.adapters);
    if (id >= 0) {  // the same for the whole warp
      __syncwarp();
      load_low(a, t, id, low[warp]);
      __syncwarp();
      if (n < a.N) {  // N % 8 == 0: all four columns or none
        const uint16_t* b = a.b + (static_cast<size_t>(id) * a.N + n) * a.R;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < a.R; j += 8) {
          const float4 l0 = *reinterpret_cast<const float4*>(&low[warp][j]);
          const float4 l1 = *reinterpret_cast<const float4*>(&low[warp][j + 4]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 w = ldg16(b + static_cast<size_t>(c) * a.R + j);
            s[c] = fmaf(__uint_as_float(w.x << 16), l0.x, s[c]);
            s[c] = fmaf(__uint_as_float(w.x & 0xffff0000u), l0.y, s[c]);
            s[c] = fmaf(__uint_as_float(w.y << 16), l0.z, s[c]);
            s[c] = fmaf(__uint_as_float(w.y & 0xffff0000u), l0.w, s[c]);
            s[c] = fmaf(__uint_as_float(w.z << 16), l1.x, s[c]);
            s[c] = fmaf(__uint_as_float(w.z & 0xffff0000u), l1.y, s[c]);
            s[c] = fmaf(__uint_as_float(w.w << 16), l1.z, s[c]);
            s[c] = fmaf(__uint_as_float(w.w & 0xffff0000u), l1.w, s[c]);
          }
        }
        v.x += s[0]; v.y += s[1]; v.z += s[2]; v.w += s[3];
      }
    }
    if (n < a.N) {
      uint2 o;
      o.x = f32_to_bf16_bits(v.x) | (static_cast<uint32_t>(f32_to_bf16_bits(v.y)) << 16);
      o.y = f32_to_bf16_bits(v.z) | (static_cast<uint32_t>(f32_to_bf16_bits(v.w)) << 16);
      *reinterpret_cast<uint2*>(a.y + static_cast<size_t>(t) * a.N + n) = o;
    }
  }
  cluster_sync_all();  // no CTA leaves while another reads its tile
}

namespace {

// [rows][cols] bf16, boxes of 64 columns and box_rows rows, 128-byte swizzle.
bool map_rows(CUtensorMap* m, const uint16_t* base, int rows, int cols, int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(cols) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

int shrink_slices(int T, int K) {
  const int tiles = (T + kAdTile - 1) / kAdTile;
  const int most = std::max(1, K / 256);  // a 32-column step for each of the eight warps
  return std::min(most, std::max(1, (2 * num_sms() + tiles - 1) / tiles));
}

int shrink_groups(int T) {
  const int tiles = (T + kAdTile - 1) / kAdTile;
  if (tiles > 8) return 4;
  return std::min(16, (std::min(T, kAdTile) + 3) / 4);
}

SplitShape split_shape(int T, int K, int N) {
  SplitShape s;
  const int blocks = (T + 255) / 256;
  s.tb = ((T + blocks - 1) / blocks + 15) / 16 * 16;
  const int tiles = (N + 127) / 128 * blocks;
  const int steps = (K + 63) / 64;
  // about one CTA to an SM; two fit with up to 64 tokens
  int c = std::max(1, std::min(kSpMaxCluster, (num_sms() + tiles / 2) / tiles));
  s.cluster = std::min(c, steps);
  const int stage = kSpWBytes + s.tb * 128;
  const int budget = s.tb <= 64 ? 104 * 1024 : 204 * 1024;
  s.stages = std::min(8, budget / stage);
  s.cols = 32;
  while (s.cols < static_cast<uint32_t>(s.tb)) s.cols *= 2;
  s.smem = std::max<size_t>(static_cast<size_t>(s.stages) * stage, static_cast<size_t>(s.tb) * 512) +
           1024;
  return s;
}

int launch_split(const AdapterArgs& a, int* status, cudaStream_t st) {
  const SplitShape sh = split_shape(a.T, a.K, a.N);
  CUtensorMap mw, mx;
  if (!map_rows(&mw, a.w, a.N, a.K, 128) || !map_rows(&mx, a.x, a.T, a.K, sh.tb)) return MOE_ERR_CUDA;
  MOE_TRY_CUDA(cudaFuncSetAttribute(adapter_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(sh.smem)));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sh.cluster, (a.N + 127) / 128, (a.T + sh.tb - 1) / sh.tb);
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = sh.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = sh.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, adapter_split_kernel, mw, mx, a, sh.tb, sh.stages, sh.cols,
                                  status, static_cast<long long>(kDefaultWaitNs)));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

int launch_shrink(const AdapterArgs& a, int* status, cudaStream_t st) {
  ShrinkArgs s{};
  s.x = a.x;
  s.a = a.a;
  s.ids = a.ids;
  s.T = a.T;
  s.K = a.K;
  s.R = a.R;
  s.adapters = a.adapters;
  s.slices = a.slices;
  s.part = const_cast<float*>(a.part);
  s.status = status;
  const dim3 grid((a.T + kAdTile - 1) / kAdTile, a.slices, shrink_groups(a.T));
  if (a.R <= 16) {
    const int smem = kShWarps * 16 * 32 * 4;
    adapter_shrink_kernel<1><<<grid, 32 * kShWarps, smem, st>>>(s);
  } else {
    const int smem = kShWarps * 32 * 32 * 4;
    adapter_shrink_kernel<2><<<grid, 32 * kShWarps, smem, st>>>(s);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_adapter_linear_workspace_size(int T, int K, int N, int R) {
  (void)N;
  if (T <= 0 || K <= 0 || R <= 0) return 256;
  return align_up(static_cast<size_t>(shrink_slices(T, K)) * T * R * sizeof(float), 256);
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
  a.slices = shrink_slices(T, K);
  a.part = static_cast<float*>(ws);
  a.y = y;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rc = launch_shrink(a, status, st);
  if (rc) return rc;
  return launch_split(a, status, st);
}
