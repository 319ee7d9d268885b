// The low-rank vectors of the adapter projection: low[t] = scale x[t] A^T, A the
// [R, K] of token t's adapter (see adapter.cu).
//
// The tokens of a tile of 128 are sorted by adapter in shared memory.  The K
// range of a tile is split over the CTAs of a cluster, whose fp32 sums meet in
// distributed shared memory and are added in the order of the ranks.
//
//  - adapter_shrink_warp_kernel, few tokens: bound by reading the A of each
//    adapter in use, and in practice by latency.  A warp takes up to 16 tokens
//    of one adapter; where a CTA has fewer such items than warps, several
//    warps share an item's columns, so that a single token's 2 R K bytes are
//    still spread over 64 warps.
//  - adapter_shrink_tile_kernel, many tokens: bound by reading x.  tcgen05 over
//    the whole tile: tokens are the M side, the rows of A of the adapters that
//    occur in the tile (as many as fit 256 columns at a time) the N side, both
//    through a TMA ring; each token then keeps its own adapter's columns.
#include <algorithm>

#include "adapter.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kAdTile = 128;
constexpr int kShWarps = 8;
constexpr int kShMaxCluster = 8;
constexpr int kItemRows = 16;

struct ShrinkArgs {
  const uint16_t* x;
  const uint16_t* a;
  const int32_t* ids;
  const float* scale;
  int T, K, R, adapters;
  float* low;  // [T, R]
  int* status;
};

// The rows of a tile, sorted by adapter, and the work in them: item j is up to
// `cut` rows row[at[j]] .. of one adapter id[j] (the low byte of row is the row).
struct __align__(16) Items {
  int32_t ids[kAdTile];
  int16_t row[kAdTile];
  int16_t at[kAdTile];
  int16_t count[kAdTile];
  int32_t id[kAdTile];
  int n;
};

// Sorts the tile's rows and cuts them into items (all threads call).  A row's
// place is counted against the other 127 rows, in their order.
__device__ void make_items(Items& u, int cut, const int32_t* ids, int t0, int rows,
                           int adapters, int* status, bool report) {
  const int i = threadIdx.x;
  if (i < kAdTile) {
    int id = -1;
    if (i < rows) {
      const int raw = ids[t0 + i];
      id = checked_id(raw, adapters);
      if (report && id != raw && raw != -1) record_status(status, MOE_ERR_INVALID);
    }
    u.ids[i] = id;
  }
  __syncthreads();
  if (i < kAdTile) {
    const int id = u.ids[i];
    int before = 0, lower = 0;  // sorted by id, rows of one id in their order
    for (int j = 0; j < rows; j += 4) {  // rows after the last have no adapter
      const int4 o = *reinterpret_cast<const int4*>(&u.ids[j]);
      const int v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        lower += v[q] >= 0 && v[q] < id ? 1 : 0;
        before += v[q] == id && j + q < i ? 1 : 0;
      }
    }
    // `before` is the row's place among its adapter's: every cut-th opens an item
    if (id >= 0) u.row[lower + before] = static_cast<int16_t>(before % cut == 0 ? i | 0x100 : i);
  }
  __syncthreads();
  if (i < 32) {
    int valid = 0;
    for (int j = i; j < kAdTile; j += 32) valid += u.ids[j] >= 0 ? 1 : 0;
    valid = __reduce_add_sync(0xffffffffu, valid);
    int n = 0;
    for (int p0 = 0; p0 < valid; p0 += 32) {
      const int p = p0 + i;
      const bool lead = p < valid && (u.row[p] & 0x100);
      const uint32_t m = __ballot_sync(0xffffffffu, lead);
      if (lead) {
        const int j = n + __popc(m & ((1u << i) - 1));
        u.at[j] = static_cast<int16_t>(p);
        u.id[j] = u.ids[u.row[p] & 0xff];
      }
      n += __popc(m);
    }
    __syncwarp();
    for (int j = i; j < n; j += 32)
      u.count[j] = static_cast<int16_t>((j + 1 < n ? u.at[j + 1] : valid) - u.at[j]);
    if (i == 0) u.n = n;
  }
  __syncthreads();
}

}  // namespace

// Cluster (rank = x) of CTAs over tile y: each takes a slice of K and the
// tile's items z, z + gridDim.z, ..., at most eight of them.  MT: 16-row tiles
// of the rank.
template <int MT>
__global__ void __launch_bounds__(32 * kShWarps) adapter_shrink_warp_kernel(const ShrinkArgs s) {
  grid_wait();
  grid_launch_dependents();  // whose own reads of x and w are then safe
  extern __shared__ __align__(16) float sh_low[];  // [warp][kItemRows][R]
  __shared__ Items u;
  const int t0 = blockIdx.y * kAdTile;
  const int rank = blockIdx.x, ranks = gridDim.x, groups = gridDim.z, z = blockIdx.z;
  make_items(u, kItemRows, s.ids, t0, min(kAdTile, s.T - t0), s.adapters, s.status,
             rank == 0 && z == 0);
  const int items = min((u.n - z + groups - 1) / groups, kShWarps);
  if (u.n <= z) return;  // the whole cluster: it has the same z
  // warps to an item: 8, 4, 2 or 1
  const int sub = items == 1 ? 8 : items == 2 ? 4 : items <= 4 ? 2 : 1;
  const int warp = threadIdx.x >> 5;
  const int steps = s.K / 32;  // K % 32 == 0
  const int k0 = steps * rank / ranks, k1 = steps * (rank + 1) / ranks;
  if (warp / sub < items) {
    const int j = z + warp / sub * groups, part = warp % sub;
    const uint16_t* A = s.a + static_cast<size_t>(u.id[j]) * s.R * s.K;
    const uint16_t* x = s.x + static_cast<size_t>(t0) * s.K;
    const int c = u.count[j];
    const int a0 = (k0 + (k1 - k0) * part / sub) * 32, a1 = (k0 + (k1 - k0) * (part + 1) / sub) * 32;
    float* out = sh_low + warp * kItemRows * s.R;
    if (c <= 8)
      shrink_item<MT, 1>(x, A, s.K, s.R, u.row + u.at[j], c, a0, a1, out);
    else
      shrink_item<MT, 2>(x, A, s.K, s.R, u.row + u.at[j], c, a0, a1, out);
  }
  cluster_sync_all();
  // the ranks take the items' rows in turn: 4 values to a thread
  const int quads = s.R / 4, per_item = kItemRows * quads;
  for (int i = rank * 32 * kShWarps + threadIdx.x; i < items * per_item;
       i += ranks * 32 * kShWarps) {
    const int l = i / per_item, p = i % per_item / quads, e = i % quads * 4;
    const int j = z + l * groups;
    if (p >= u.count[j]) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < ranks; ++r) {
      const uint32_t at = mapa_shared(sh_low + (l * sub * kItemRows + p) * s.R + e, r);
      for (int q = 0; q < sub; ++q) {
        const float4 o = ld_cluster_f4(at + q * kItemRows * s.R * 4);
        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
      }
    }
    const float sc = s.scale ? s.scale[u.id[j]] : 1.f;
    const int t = t0 + (u.row[u.at[j] + p] & 0xff);
    *reinterpret_cast<float4*>(s.low + static_cast<size_t>(t) * s.R + e) =
        make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
  }
  cluster_sync_all();  // no CTA leaves while another reads its sums
}

namespace {

constexpr int kStThreads = 192;  // warp 0: TMA, 1: MMA + TMEM, 2-5: epilogue
constexpr int kStXBytes = kAdTile * 64 * 2;
constexpr int kStMaxCols = 256;
constexpr int kStMaxStages = 8;
constexpr int kStSmem = 200 * 1024;

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

}  // namespace

// Cluster (rank = x) of CTAs over tile y; ma: [adapters R][K], boxes of R rows.
__global__ void __launch_bounds__(kStThreads, 1)
    adapter_shrink_tile_kernel(const __grid_constant__ CUtensorMap mx,
                               const __grid_constant__ CUtensorMap ma, const ShrinkArgs s,
                               long long wait_ns) {
  grid_wait();
  grid_launch_dependents();  // whose own reads of x and w are then safe
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[kStMaxStages], empty[kStMaxStages], accfull, accempty, done;
  __shared__ uint32_t tmem_slot;
  __shared__ int cta_abort;
  __shared__ Items u;
  __shared__ int16_t of_row[kAdTile];  // the row's adapter among the tile's (-1: none)
  const Waiter wt{&cta_abort, s.status, wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, ranks = gridDim.x;
  const int t0 = blockIdx.y * kAdTile;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&accfull, 1);
    mbar_init(&accempty, 4);
    mbar_init(&done, 1);
    cta_abort = 0;
    fence_mbarrier_init();
  }
  if (threadIdx.x < kAdTile) of_row[threadIdx.x] = -1;
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kStMaxCols);
    tmem_relinquish();
  }
  tc_fence_before();
  // the barriers in here cover the initialisation too
  make_items(u, kAdTile, s.ids, t0, min(kAdTile, s.T - t0), s.adapters, s.status, rank == 0);
  tc_fence_after();
  const uint32_t tbase = tmem_slot;
  const int n = u.n;
  for (int j = warp; j < n; j += kStThreads / 32)
    for (int p = lane; p < u.count[j]; p += 32) of_row[u.row[u.at[j] + p] & 0xff] = j;
  __syncthreads();

  // the ring goes by the columns that a pass needs
  float* sums = reinterpret_cast<float*>(smem);  // [kAdTile][R]
  uint8_t* ring = smem + kAdTile * s.R * 4;  // R % 8 == 0: whole KiB
  const int per = kStMaxCols / s.R;  // adapters to a pass
  const int passes = (n + per - 1) / per;
  const int most = (min(n, per) * s.R + 15) / 16 * 16;
  const int stage_bytes = kStXBytes + (most * 128 + 1023) / 1024 * 1024;
  const int stages = min(kStMaxStages,
                         static_cast<int>(smem_raw + kStSmem - ring) / stage_bytes);
  const int steps = (s.K + 63) / 64;
  const int s0 = steps * rank / ranks, s1 = steps * (rank + 1) / ranks;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensor_map(&mx);
      prefetch_tensor_map(&ma);
      uint32_t it = 0;
      bool ok = true;
      for (int pass = 0; pass < passes && ok; ++pass) {
        const int d0 = pass * per, d1 = min(n, d0 + per);
        const uint32_t bytes = kStXBytes + (d1 - d0) * s.R * 128;
        for (int k = s0; k < s1; ++k, ++it) {
          const int i = it % stages;
          if (!mbar_wait(&empty[i], ((it / stages) & 1u) ^ 1u, wt)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + i * stage_bytes;
          mbar_arrive_expect_tx(&full[i], bytes);
          tma_g2s_2d(st, &mx, &full[i], k * 64, t0);
          for (int d = d0; d < d1; ++d)
            tma_g2s_3d(st + kStXBytes + (d - d0) * s.R * 128, &ma, &full[i], k * 64, 0, u.id[d]);
        }
      }
      drain_ring(full, it, stages, s.status);
    }
  } else if (warp == 1) {
    uint32_t it = 0;
    bool ok = true;
    for (int pass = 0; pass < passes && ok; ++pass) {
      const int cols = (min(n - pass * per, per) * s.R + 15) / 16 * 16;
      const uint32_t idesc = idesc_bf16(kAdTile, cols);
      if (!__all_sync(0xffffffffu, mbar_wait(&accempty, (pass & 1u) ^ 1u, wt))) break;
      tc_fence_after();
      for (int k = s0; k < s1; ++k, ++it) {
        const int i = it % stages;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[i], (it / stages) & 1u, wt))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t da = smem_desc_sw128(ring + i * stage_bytes);
        const uint64_t db = smem_desc_sw128(ring + i * stage_bytes + kStXBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_warp(tbase, da + 2 * kk, db + 2 * kk, idesc, (k != s0) | (kk != 0));
        umma_commit_warp(&empty[i]);
      }
      if (ok) umma_commit_warp(&accfull);
    }
    umma_commit_warp(&done);
    mbar_drain(&done, 0, s.status);
  } else {
    const int q = warp & 3;
    const int row = 32 * q + lane;
    const int mine = of_row[row];
    for (int pass = 0; pass < passes; ++pass) {
      if (!__all_sync(0xffffffffu, mbar_wait(&accfull, pass & 1u, wt))) break;
      tc_fence_after();
      const int d0 = pass * per, d1 = min(n, d0 + per);
      for (int d = d0; d < d1; ++d) {
        if (!__any_sync(0xffffffffu, mine == d)) continue;
        for (int c = 0; c < s.R; c += 8) {
          uint32_t r[8];
          tmem_ld8(tbase + (static_cast<uint32_t>(32 * q) << 16) + (d - d0) * s.R + c, r);
          tmem_ld_wait();
          if (mine == d) {
            float4* o = reinterpret_cast<float4*>(sums + row * s.R + c);
            o[0] = make_float4(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]),
                               __uint_as_float(r[3]));
            o[1] = make_float4(__uint_as_float(r[4]), __uint_as_float(r[5]), __uint_as_float(r[6]),
                               __uint_as_float(r[7]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, kStMaxCols);
  }
  // the ranks take the rows in turn: 4 values to a thread, summed in rank order
  const int quads = s.R / 4;
  for (int i = rank * kStThreads + threadIdx.x; i < kAdTile * quads; i += ranks * kStThreads) {
    const int row = i / quads, e = i % quads * 4;
    const int d = of_row[row];
    if (d < 0) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < ranks; ++r) {
      const float4 o = ld_cluster_f4(mapa_shared(sums + row * s.R + e, r));
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
    const float sc = s.scale ? s.scale[u.id[d]] : 1.f;
    *reinterpret_cast<float4*>(s.low + static_cast<size_t>(t0 + row) * s.R + e) =
        make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
  }
  cluster_sync_all();  // no CTA leaves while another reads its sums
}

namespace {

template <int MT>
int launch_warp(const ShrinkArgs& s, cudaStream_t st) {
  const int tiles = (s.T + kAdTile - 1) / kAdTile, rows = std::min(s.T, kAdTile);
  const int ranks = std::max(1, std::min(kShMaxCluster, s.K / 64));
  // groups of items: about one CTA to an SM, which leaves room for the kernel
  // that streams W beside it; at most eight items each
  const int groups = std::min(rows, std::max((rows + kShWarps - 1) / kShWarps,
                                             num_sms() / (ranks * tiles)));
  auto kern = adapter_shrink_warp_kernel<MT>;
  const int smem = kShWarps * kItemRows * s.R * 4;
  if (smem > 48 * 1024)
    MOE_TRY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(ranks, tiles, groups);
  cfg.blockDim = dim3(32 * kShWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  set_adapter_attrs(&cfg, attr, ranks);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kern, s));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

int launch_tile(const ShrinkArgs& s, cudaStream_t st) {
  const int tiles = (s.T + kAdTile - 1) / kAdTile;
  const int ranks =
      std::max(1, std::min({kShMaxCluster, num_sms() / tiles, (s.K + 63) / 64}));
  CUtensorMap mx, ma;
  const uint64_t dims[3] = {static_cast<uint64_t>(s.K), static_cast<uint64_t>(s.R),
                            static_cast<uint64_t>(s.adapters)};
  const uint64_t strides[2] = {static_cast<uint64_t>(s.K) * 2,
                               static_cast<uint64_t>(s.K) * s.R * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(s.R), 1};
  if (!adapter_map_rows(&mx, s.x, s.T, s.K, kAdTile) ||
      !encode_tensor_map(&ma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, s.a, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B))
    return MOE_ERR_CUDA;
  MOE_TRY_CUDA(cudaFuncSetAttribute(adapter_shrink_tile_kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kStSmem));
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(ranks, tiles);
  cfg.blockDim = dim3(kStThreads);
  cfg.dynamicSmemBytes = kStSmem;
  cfg.stream = st;
  set_adapter_attrs(&cfg, attr, ranks);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, adapter_shrink_tile_kernel, mx, ma, s,
                                  static_cast<long long>(kDefaultWaitNs)));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

int launch_adapter_shrink(const AdapterArgs& a, int* status, cudaStream_t st) {
  ShrinkArgs s{};
  s.x = a.x;
  s.a = a.a;
  s.ids = a.ids;
  s.scale = a.scale;
  s.T = a.T;
  s.K = a.K;
  s.R = a.R;
  s.adapters = a.adapters;
  s.low = a.low;
  s.status = status;
  if (a.T > kSplitTokens) return launch_tile(s, st);
  if (a.R <= 16) return launch_warp<1>(s, st);
  if (a.R <= 32) return launch_warp<2>(s, st);
  if (a.R <= 64) return launch_warp<4>(s, st);
  return launch_warp<8>(s, st);
}

}  // namespace moe
