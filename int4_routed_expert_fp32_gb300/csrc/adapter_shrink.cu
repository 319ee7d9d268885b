// The low-rank vectors of the adapter projection: low[t] = scale x[t] A^T, A the
// [R, K] of token t's adapter (see adapter.cu).
//
// The tokens of a tile of 128 are sorted by adapter in shared memory.  tcgen05
// over the whole tile: tokens are the M side, the rows of A of the adapters that
// occur in the tile (as many as fit `cols` columns at a time) the N side, both
// through a TMA ring; each token then keeps its own adapter's columns.  The MMAs
// of rows that do not use an adapter are wasted, and cost nothing that matters:
// the kernel is bound by reading x and the A in use.  The K range of a tile is
// split over the CTAs of a cluster, whose fp32 sums meet in distributed shared
// memory and are added in the order of the ranks; with few tokens, which can
// have an adapter each, the adapters are dealt to further clusters.
//
// Measured: 2047 tokens of K = 7168, rank 16 (30.8 MB): 15 us, of which 5 pass
// before the first tile has arrived (arguments, the sort of the rows, a copy's
// latency), 6.5 over the copies (4.7 TB/s) and 3 in the clusters' sum.
#include <algorithm>

#include "adapter.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kAdTile = 128;
constexpr int kShMaxCluster = 8;

struct ShrinkArgs {
  const int32_t* ids;
  const float* scale;
  int T, K, R, adapters;
  int per, stages;  // adapters to a pass, slots of the ring
  int xrows;        // rows of x in a slot: a multiple of 8, those there are
  float* low;       // [T, R]
  int* status;
};

// The rows of a tile, sorted by adapter, and the adapters in it: item j is the
// count[j] rows row[at[j]] .. of adapter id[j] (the low byte of row is the row; 0x100
// marks an adapter's first).
struct __align__(16) Items {
  int32_t ids[kAdTile];
  int16_t row[kAdTile];
  int16_t at[kAdTile];
  int16_t count[kAdTile];
  int32_t id[kAdTile];
  int n;
};

// Sorts the tile's rows and lists their adapters (all threads call).  A row's
// place is counted against the other 127 rows, in their order.
__device__ void make_items(Items& u, const int32_t* ids, int t0, int rows, int adapters,
                           int* status, bool report) {
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
    // `before` is the row's place among its adapter's
    if (id >= 0) u.row[lower + before] = static_cast<int16_t>(before == 0 ? i | 0x100 : i);
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

constexpr int kStThreads = 192;  // warp 0: TMA, 1: MMA + TMEM, 2-5: epilogue
constexpr int kStMaxCols = 256;
constexpr int kStMaxStages = 8;

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

}  // namespace

// Cluster (rank = x) of CTAs over tile y and passes z, z + gridDim.z, ...; ma:
// [adapters][R][K], boxes of R rows of one adapter.  STALL (tests only): the copies
// stop before stage stall_at.
template <bool STALL>
__global__ void __launch_bounds__(kStThreads, 1)
    adapter_shrink_tile_kernel(const __grid_constant__ CUtensorMap mx,
                               const __grid_constant__ CUtensorMap ma, const ShrinkArgs s,
                               long long wait_ns, int stall_at) {
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&mx);
    prefetch_tensor_map(&ma);
  }
  grid_wait();
  grid_launch_dependents();  // whose own reads of x and w are then safe
  const int rank = blockIdx.x, ranks = gridDim.x;
  const int t0 = blockIdx.y * kAdTile;
  const int steps = (s.K + 63) / 64;
  const int s0 = steps * rank / ranks, s1 = steps * (rank + 1) / ranks;
  // x on its way to L2 while the rows are sorted
  if (threadIdx.x >= kStThreads - 32)
    for (int k = s0 + threadIdx.x - (kStThreads - 32); k < s1; k += 32)
      prefetch_tile_2d(&mx, k * 64, t0);
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
  make_items(u, s.ids, t0, min(kAdTile, s.T - t0), s.adapters, s.status,
             rank == 0 && blockIdx.z == 0);
  tc_fence_after();
  const uint32_t tbase = tmem_slot;
  const int n = u.n;
  for (int j = warp; j < n; j += kStThreads / 32)
    for (int p = lane; p < u.count[j]; p += 32) of_row[u.row[u.at[j] + p] & 0xff] = j;
  __syncthreads();

  // the tile's adapters in even shares
  const int per = max(1, min(s.per, (n + static_cast<int>(gridDim.z) - 1) / static_cast<int>(gridDim.z)));
  const int stages = s.stages;
  const int passes = (n + per - 1) / per;
  // a slot: A, then x.  The MMA's M side is 128 rows all the same: with fewer rows
  // of x it goes on into what follows (the sums, after the last slot), whose
  // products are no token's
  const int abytes = (per * s.R + 15) / 16 * 2048;
  const int xbytes = s.xrows * 128;
  const int stage_bytes = abytes + xbytes;
  uint8_t* ring = smem;
  float* sums = reinterpret_cast<float*>(ring + stages * stage_bytes);  // [xrows][R]

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int pass = blockIdx.z; pass < passes && ok; pass += gridDim.z) {
        const int d0 = pass * per, d1 = min(n, d0 + per);
        const uint32_t bytes = xbytes + (d1 - d0) * s.R * 128;
        for (int k = s0; k < s1; ++k, ++it) {
          const int i = it % stages;
          if ((STALL && static_cast<int>(it) == stall_at) ||
              !mbar_wait(&empty[i], ((it / stages) & 1u) ^ 1u, wt)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + i * stage_bytes;
          mbar_arrive_expect_tx(&full[i], bytes);
          tma_g2s_2d(st + abytes, &mx, &full[i], k * 64, t0);
          for (int d = d0; d < d1; ++d)
            tma_g2s_3d(st + (d - d0) * s.R * 128, &ma, &full[i], k * 64, 0, u.id[d]);
        }
      }
      drain_ring(full, it, stages, s.status);
    }
  } else if (warp == 1) {
    uint32_t it = 0;
    bool ok = true;
    for (int pass = blockIdx.z, turn = 0; pass < passes && ok; pass += gridDim.z, ++turn) {
      const int cols = (min(n - pass * per, per) * s.R + 15) / 16 * 16;
      const uint32_t idesc = idesc_bf16(kAdTile, cols);
      if (!__all_sync(0xffffffffu, mbar_wait(&accempty, (turn & 1u) ^ 1u, wt))) break;
      tc_fence_after();
      for (int k = s0; k < s1; ++k, ++it) {
        const int i = it % stages;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[i], (it / stages) & 1u, wt))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t da = smem_desc_sw128(ring + i * stage_bytes + abytes);
        const uint64_t db = smem_desc_sw128(ring + i * stage_bytes);
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
    for (int pass = blockIdx.z, turn = 0; pass < passes; pass += gridDim.z, ++turn) {
      if (!__all_sync(0xffffffffu, mbar_wait(&accfull, turn & 1u, wt))) break;
      tc_fence_after();
      const int d0 = pass * per, d1 = min(n, d0 + per);
      for (int d = d0; d < d1; ++d) {
        if (!__any_sync(0xffffffffu, mine == d)) continue;
        for (int c = 0; c < s.R; c += 8) {
          uint32_t r[8];
          __syncwarp();  // the lanes of other adapters went past the last stores
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
  // Tensor memory goes back before the wait for the other ranks, which may still
  // wait for theirs behind another kernel's CTA (see kSmBytes)
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, kStMaxCols);
  }
  cluster_sync_all();
  // the ranks take the rows in turn: 4 values to a thread, summed in rank order
  const int quads = s.R / 4;
  for (int i = rank * kStThreads + threadIdx.x; i < kAdTile * quads; i += ranks * kStThreads) {
    const int row = i / quads, e = i % quads * 4;
    const int d = of_row[row];
    if (d < 0 || d / per % gridDim.z != blockIdx.z) continue;  // none, or another cluster's
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

constexpr int kAlone = 198 * 1024;  // shared memory where no other kernel is to fit beside

// A slot of `per` adapters' A and xrows rows of x; what the CTA needs beside them.
constexpr int shrink_slot(int per, int R, int xrows) {
  return (per * R + 15) / 16 * 2048 + xrows * 128;
}

constexpr int shrink_fixed(int R, int xrows) {
  const int sums = xrows * R * 4, over = (kAdTile - xrows) * 128;
  return (sums > over ? sums : over) + 1024;
}

constexpr int shrink_stages(int bytes, int per, int R, int xrows) {
  const int n = (bytes - shrink_fixed(R, xrows)) / shrink_slot(per, R, xrows);
  return n < 2 ? 2 : n > kStMaxStages ? kStMaxStages : n;
}

// Above kSplitTokens the tile kernel starts beside this one, takes all of an SM's
// tensor memory and keeps it until this one has finished: a CTA of each must not
// fit an SM together, whatever the rank.
constexpr bool shrink_fills_sm() {
  for (int R = 8; R <= 128; R += 8) {
    const int per = kStMaxCols / R;
    const int smem = shrink_stages(kAlone, per, R, kAdTile) * shrink_slot(per, R, kAdTile) +
                     shrink_fixed(R, kAdTile);
    if (smem + kTileSmemLeast + 2 * kSmCtaBytes <= kSmBytes) return false;
  }
  return true;
}

static_assert(shrink_fills_sm(), "a tile CTA could keep the tensor memory that the shrink waits for");

}  // namespace

int launch_adapter_shrink(const AdapterArgs& a, int* status, cudaStream_t st,
                          const AdapterStall* stall) {
  const bool stop = stall && stall->kernel == 0;
  auto kern = stop ? adapter_shrink_tile_kernel<true> : adapter_shrink_tile_kernel<false>;
  ShrinkArgs s{};
  s.ids = a.ids;
  s.scale = a.scale;
  s.T = a.T;
  s.K = a.K;
  s.R = a.R;
  s.adapters = a.adapters;
  s.low = a.low;
  s.status = status;
  const int tiles = (s.T + kAdTile - 1) / kAdTile, rows = std::min(s.T, kAdTile);
  const int steps = (s.K + 63) / 64;
  // Many tokens: one cluster to a tile, all the columns a pass can have.  Few:
  // adapters dealt to clusters, some 150 CTAs in all if every token has its own.
  int groups = 1;
  s.per = kStMaxCols / s.R;
  if (s.T <= kSplitTokens) {
    const int want = std::min(rows, std::max(1, num_sms() / (kShMaxCluster * tiles)));
    s.per = std::min(s.per, (rows + want - 1) / want);
    groups = std::min(want, (rows + s.per - 1) / s.per);
  }
  // Little enough for the projection kernel to start beside it, where that leaves
  // two slots, if need be with half the adapters to a pass; else its CTAs come when
  // these have gone (32 tokens of rank 32: 17 us against 27; with fewer adapters
  // still, x is read too often: 64 tokens of rank 64, 63 us against 41).
  s.xrows = (rows + 7) / 8 * 8;
  const int fixed = shrink_fixed(s.R, s.xrows), room = s.T <= 64 ? 50 * 1024 : 84 * 1024;
  auto two_fit = [&](int per) { return fixed + 2 * shrink_slot(per, s.R, s.xrows) <= room; };
  const int beside = two_fit(s.per) ? s.per : (s.per + 1) / 2;
  int bytes = kAlone;
  if (s.T <= kSplitTokens && adapter_beside(s.T, s.R) && two_fit(beside)) {
    s.per = beside;
    bytes = room;
  }
  s.stages = shrink_stages(bytes, s.per, s.R, s.xrows);
  const int smem = s.stages * shrink_slot(s.per, s.R, s.xrows) + fixed;
  MOE_TRY_CUDA(adapter_smem(reinterpret_cast<const void*>(kern)));
  int ranks = 1;
  MOE_TRY_CUDA(adapter_cluster(reinterpret_cast<const void*>(kern), kStThreads, smem,
                               tiles * groups, std::min(kShMaxCluster, steps), &ranks));
  CUtensorMap mx, ma;
  const uint64_t dims[3] = {static_cast<uint64_t>(s.K), static_cast<uint64_t>(s.R),
                            static_cast<uint64_t>(s.adapters)};
  const uint64_t strides[2] = {static_cast<uint64_t>(s.K) * 2,
                               static_cast<uint64_t>(s.K) * s.R * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(s.R), 1};
  if (!adapter_map_rows(&mx, a.x, s.T, s.K, s.xrows) ||
      !encode_tensor_map(&ma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.a, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B))
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(ranks, tiles, groups);
  cfg.blockDim = dim3(kStThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  set_adapter_attrs(&cfg, attr, ranks);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kern, mx, ma, s,
                                  stop ? stall->wait_ns : static_cast<long long>(kDefaultWaitNs),
                                  stop ? stall->stage : 0));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
