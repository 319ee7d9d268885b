// The adapter projection for many tokens (see adapter.cu), on CTA pairs: y =
// x W^T plus the low-rank term, bound by the tensor cores.
//
// A cluster of two CTAs walks output tiles of 256 tokens x BN columns, each CTA
// holding 128 of the tokens and half of the columns' weights: an MMA
// (cta_group::2) of M = 256, N = BN, K = 16 reads 128 rows of A and BN / 2 of B
// from each SM's shared memory, which leaves room for the copies beside it; one
// CTA's 128 x 256 MMA would read and write more than the shared memory's rate.
// Two TMEM accumulators: a tile's epilogue runs under the next tile's MMAs.
//
// The low-rank term is more K columns of the same accumulation.  For every
// adapter that occurs in the tile's 256 rows, one stage (two for ranks over 32,
// four over 64) has as A operand the scaled vectors s p of the rows that use
// it and zeros in the others, and as B operand the adapter's rows of lora_b.  p
// is taken as hi + lo, both bf16: 16 bits of significand, so that its rounding
// stays 2^-8 of the output's.  Up to rank 32 hi and lo sit side by side in the
// 64 columns of one stage and meet the same B.
//
// A row of lora_b with an infinity or NaN would reach the other rows of the
// tile through their zeros.  The warps that write the A operand therefore look
// at the B rows as they arrive; such a row is set to zero, and the epilogue
// adds it by hand to the tokens of its own adapter.
//
// Per CTA: warp 0 (one thread) TMA; warp 1 of rank 0 issues the MMAs; warps
// 2-5 the epilogue of the CTA's 128 rows; warps 6-9 the tile's list of
// adapters and the A operands of its low-rank stages; warps 10 and up hand those
// to the MMA warp.  Every wait on an mbarrier is bounded.
//
// Handing over.  The MMA warp of rank 0 reads what threads of rank 1 wrote to
// their shared memory, so the chain from the writes to the MMA has a release and
// an acquire at cluster scope.  Each takes some 0.4 us; done by the A warps or by
// the MMA warp, one stage after the other, they make it 445 us in place of 357
// (T = 8192, 8 adapters of rank 64 in every tile).  They are left to warps that take
// the stages in turn.
//
// Measured with the shrink before it: T = 8192, K = 3584, N = 7168, 8 adapters of
// rank 64, requests of consecutive tokens: 270 us (1.60 PFLOP/s), and 290 to 297 in
// runs of 0.1 s and more, under the power cap (1.45 to 1.49, where cuBLAS sustains
// 1.74).  T = 2047, K = 7168, N = 3584, 16 of rank 16: 81.5 us (1.30 PFLOP/s), about
// 15 of them the shrink.
#include <math.h>

#include <algorithm>

#include "adapter.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kTlRows = 256;                 // tokens of a tile, 128 to a CTA
constexpr int kTlABytes = 128 * 64 * 2;      // the CTA's half of a stage's A
constexpr int kTlStages = 6;
constexpr int kFillWarp0 = 6;
constexpr int kPassWarp0 = 10;

// Four warps hand over; two at ranks over 32, where a stage's MMAs take longer and
// more threads would leave too few registers (T = 8192, 8 adapters of rank 64:
// 362 us with two, 382 with four; T = 512, 64 of rank 16: 109 and 105).
constexpr int pass_warps(bool wide) { return wide ? 2 : 4; }
constexpr int tile_threads(bool wide) { return 32 * (kPassWarp0 + pass_warps(wide)); }

template <int BN>
struct TileShape {
  static constexpr int kBRows = BN / 2;
  static constexpr int kBBytes = kBRows * 64 * 2;
  static constexpr int kStageBytes = kTlABytes + kBBytes;
  static constexpr int kSmem = kTlStages * kStageBytes + 1024;
  static_assert(kBBytes % 1024 == 0 && BN % 32 == 0 && 2 * BN <= 512, "tile");
  static_assert(fills_half_sm(kSmem), "CTAs of two pair kernels must not meet on an SM");
  static_assert(kSmem >= kTileSmemLeast, "what the shrink kernel counts with");
};

// 2-D tensor copy into this CTA's shared memory whose completion is counted on
// a barrier of either CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_pair_g2s_2d(void* dst, const CUtensorMap* map, uint32_t bar,
                                                int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// D (+)= A[smem] B[smem] over the CTA pair, kind::f16; a whole converged warp
// of rank 0, one lane elected in the instruction.
__device__ __forceinline__ void umma_pair_f16_warp(uint32_t d_tmem, uint64_t a_desc,
                                                   uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, p;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void fill_barrier() {  // the 128 threads of warps 6-9
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

__device__ __forceinline__ bool fill_all(bool v) {  // whether v holds for all of them
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Bits 15 and 31 tell whether the low or high bf16 of a word is an infinity or NaN:
// an exponent of all ones carries into them (the others stay below).
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return (w & 0x7f807f80u) + 0x00800080u;
}

// A tile's adapters, double buffered by tile parity: written by warps 6-9, read
// by every role of the CTA.
struct __align__(16) TileList {  // an array of two: each 16-byte aligned
  int32_t ids[kTlRows];      // of the tile's rows
  int32_t adapter[kTlRows];  // adapter d, in the order of first occurrence
  int16_t of_row[128];       // d of this CTA's rows (-1: none)
  uint32_t leads[kTlRows / 32];
  int n;
};

static_assert(sizeof(TileList) % 16 == 0, "ids is read in 16-byte vectors");

// bad[u & 7][d] == u + 1 (16 bits): in the pair's u-th tile rows of adapter d's
// lora_b were set to zero, in either CTA.  Never reset: the A warps of the peer
// can be several tiles ahead, but at most seven (six stages, one to a tile at
// least, and the tile whose epilogue is to read it); a stale match only makes
// the epilogue look at the rows for itself.
constexpr int kBadRing = 8;

// On the error path of rank 1: its copies of x and W count on rank 0's barriers,
// where those of a stage that rank 0 never armed cannot be waited for.  A copy takes
// a microsecond or two; its issuer stays this long after the last.
constexpr int64_t kSettleNs = 10000000;

__device__ __forceinline__ void settle_copies() {
  const uint64_t t0 = global_timer_ns();
  while (static_cast<int64_t>(global_timer_ns() - t0) < kSettleNs) __nanosleep(10000);
}

}  // namespace

// WIDE: R > 32, a hi and a lo stage for every 64 columns of the rank.  STALL (tests
// only): each CTA's copies stop before stage stall_at.
template <int BN, bool WIDE, bool STALL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(tile_threads(WIDE), 1)
    adapter_tile_kernel(const __grid_constant__ CUtensorMap mx,
                        const __grid_constant__ CUtensorMap mw,
                        const __grid_constant__ CUtensorMap mb, const AdapterArgs a, int* status,
                        long long wait_ns, int stall_at) {
  grid_launch_dependents();
  using S = TileShape<BN>;
  constexpr int kThreads = tile_threads(WIDE), kPassWarps = pass_warps(WIDE);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[kTlStages];   // rank 0: both CTAs' operands are there
  __shared__ __align__(8) uint64_t sfree[kTlStages];  // the stage's MMAs are done
  __shared__ __align__(8) uint64_t sgo[kTlStages];    // a low-rank stage's slot is free
  __shared__ __align__(8) uint64_t bland[kTlStages];  // and its B (this CTA's half) there
  __shared__ __align__(8) uint64_t awrote[kTlStages];  // and its A, and B looked over
  __shared__ __align__(8) uint64_t passed[kTlStages];  // rank 0: the same in rank 1
  __shared__ __align__(8) uint64_t accfull[2], accempty[2], listfull[2], listempty[2], mma_done;
  __shared__ uint32_t tmem_slot;
  __shared__ int cta_abort;
  __shared__ TileList lists[2];
  __shared__ uint16_t bad[kBadRing][kTlRows];
  const Waiter wt{&cta_abort, status, wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kTlStages; ++s) {
      mbar_init(&full[s], 2);  // rank 0's producer, and the warp that hands over
      mbar_init(&sfree[s], 1);
      mbar_init(&sgo[s], 1);
      mbar_init(&bland[s], 1);
      mbar_init(&awrote[s], 4);
      mbar_init(&passed[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 8);  // rank 0: the epilogue warps of both CTAs
      mbar_init(&listfull[b], 4);
      // producer, epilogue warps, warps 10 and up, rank 0's MMA warp
      mbar_init(&listempty[b], 5 + kPassWarps + (rank == 0 ? 1 : 0));
    }
    mbar_init(&mma_done, 1);
    cta_abort = 0;
    fence_mbarrier_init();
  }
  for (int i = threadIdx.x; i < kBadRing * kTlRows; i += kThreads) (&bad[0][0])[i] = 0;
  if (warp == 1) {
    tmem_alloc_pair(&tmem_slot, 512);
    tmem_relinquish_pair();
  }
  // both CTAs' barriers exist before either CTA arrives on the other's
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;

  const int tn = (a.N + BN - 1) / BN, tm = (a.T + kTlRows - 1) / kTlRows;
  const int tiles = tn * tm;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int ksteps = (a.K + 63) / 64;
  const int blocks = WIDE ? (a.R + 63) / 64 : 1;  // 64-column blocks of the rank
  const int parts = WIDE ? 2 : 1;                 // hi and lo stages of a block

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensor_map(&mx);
      prefetch_tensor_map(&mw);
      prefetch_tensor_map(&mb);
      const uint32_t full0 = mapa_shared(full, 0);
      uint32_t it = 0, uc = 0;
      uint32_t bused = 0, bpar = 0;  // slots that held a B, and the parity of the next use
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++uc) {
        const int n0 = (t % tn) * BN + static_cast<int>(rank) * S::kBRows;
        const int m0 = (t / tn) * kTlRows + static_cast<int>(rank) * 128;
        for (int k = 0; k < ksteps; ++k, ++it) {
          const int s = it % kTlStages;
          if ((STALL && static_cast<int>(it) == stall_at) ||
              !mbar_wait(&sfree[s], ((it / kTlStages) & 1u) ^ 1u, wt)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * S::kStageBytes;
          if (rank == 0) {
            mbar_arrive_expect_tx(&full[s], 2 * S::kStageBytes);
            mbar_arrive(&full[s]);
          }
          tma_pair_g2s_2d(st, &mx, full0 + 8u * s, k * 64, m0);
          tma_pair_g2s_2d(st + kTlABytes, &mw, full0 + 8u * s, k * 64, n0);
        }
        if (!ok) break;
        const int b = uc & 1;
        if (!mbar_wait(&listfull[b], (uc >> 1) & 1u, wt)) {
          ok = false;
          break;
        }
        const TileList& l = lists[b];
        const int stages = l.n * blocks * parts;
        for (int e = 0; e < stages; ++e, ++it) {
          const int s = it % kTlStages;
          if ((STALL && static_cast<int>(it) == stall_at) ||
              !mbar_wait(&sfree[s], ((it / kTlStages) & 1u) ^ 1u, wt)) {
            ok = false;
            break;
          }
          const int blk = e / (l.n * parts), d = e / parts % l.n;
          mbar_arrive(&sgo[s]);
          mbar_arrive_expect_tx(&bland[s], S::kBBytes);
          tma_g2s_3d(smem + s * S::kStageBytes + kTlABytes, &mb, &bland[s], 64 * blk, n0,
                     l.adapter[d]);
          bused |= 1u << s;
          bpar ^= 1u << s;
          if (rank == 0) mbar_arrive(&full[s]);
        }
        mbar_arrive(&listempty[b]);
      }
      // the issued copies land before the pair can leave: rank 0 sees both
      // CTAs' on its barriers, and the closing cluster barrier holds rank 1.  B's land
      // on the CTA's own; the A warps have seen them unless they gave up
      for (int s = 0; s < kTlStages; ++s)
        if ((bused >> s) & 1u) mbar_drain(&bland[s], ((bpar >> s) & 1u) ^ 1u, status);
      if (rank == 0)
        drain_ring(full, it, kTlStages, status);
      else if (!ok)
        settle_copies();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(kTlRows, BN);
      uint32_t it = 0, uc = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++uc) {
        const int b = uc & 1;
        const uint32_t ph = (uc >> 1) & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait(&accempty[b], ph ^ 1u, wt))) break;
        tc_fence_after();
        const uint32_t acc = tbase + b * BN;
        for (int k = 0; k < ksteps; ++k, ++it) {
          const int s = it % kTlStages;
          if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (it / kTlStages) & 1u, wt))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = smem_desc_sw128(smem + s * S::kStageBytes);
          const uint64_t db = smem_desc_sw128(smem + s * S::kStageBytes + kTlABytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_pair_f16_warp(acc, da + 2 * kk, db + 2 * kk, idesc, (k | kk) != 0);
          umma_pair_commit_warp(&sfree[s]);
        }
        if (!ok) break;
        if (!__all_sync(0xffffffffu, mbar_wait(&listfull[b], ph, wt))) break;
        const int n = lists[b].n;
        const int stages = n * blocks * parts;
        for (int e = 0; e < stages; ++e, ++it) {
          const int s = it % kTlStages;
          if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (it / kTlStages) & 1u, wt))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = smem_desc_sw128(smem + s * S::kStageBytes);
          const uint64_t db = smem_desc_sw128(smem + s * S::kStageBytes + kTlABytes);
          const int blk = e / (n * parts);
          const int k16 = (min(a.R - 64 * blk, 64) + 15) / 16;
          for (int kk = 0; kk < k16; ++kk) {
            umma_pair_f16_warp(acc, da + 2 * kk, db + 2 * kk, idesc, 1);
            // up to rank 32 lo is 32 columns (64 bytes) behind hi
            if (!WIDE) umma_pair_f16_warp(acc, da + 4 + 2 * kk, db + 2 * kk, idesc, 1);
          }
          umma_pair_commit_warp(&sfree[s]);
        }
        if (lane == 0) mbar_arrive(&listempty[b]);
        if (ok) umma_pair_commit_warp(&accfull[b]);
      }
      // every MMA completes before either CTA frees its TMEM or leaves
      umma_pair_commit_warp(&mma_done);
    }
  } else if (warp < kFillWarp0) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const uint32_t leader_accempty = mapa_shared(accempty, 0);
    uint32_t uc = 0;
    for (int t = pair; t < tiles; t += pairs, ++uc) {
      const int b = uc & 1;
      const int n0 = (t % tn) * BN;
      const int row = (t / tn) * kTlRows + static_cast<int>(rank) * 128 + 32 * q + lane;
      // warp-uniform outcome: tcgen05.ld needs the whole warp
      const uint32_t ph = (uc >> 1) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(&accfull[b], ph, wt, 256) &&
                                       mbar_wait(&listfull[b], ph, wt)))
        break;
      tc_fence_after();
      // adapters with a row of lora_b that is not finite: by hand, below (the other
      // CTA's flags were written before the accumulator's last MMA)
      asm volatile("fence.acq_rel.cluster;" ::: "memory");
      const TileList& l = lists[b];
      const int d = l.of_row[32 * q + lane];
      const bool by_hand =
          d >= 0 && *reinterpret_cast<const volatile uint16_t*>(&bad[uc % kBadRing][d]) ==
                        static_cast<uint16_t>(uc + 1);
#pragma unroll 1
      for (int c0 = 0; c0 < BN; c0 += 32) {
        uint32_t r[32];
        __syncwarp();  // rows beyond T and rows done by hand took their own ways
        tmem_ld32(tbase + (static_cast<uint32_t>(32 * q) << 16) + b * BN + c0, r);
        tmem_ld_wait();
        if (c0 + 32 == BN) {  // the accumulator goes back to the MMA warp
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(leader_accempty + 8u * b);
        }
        const int col = n0 + c0;
        if (row < a.T && col < a.N) {
          uint16_t* dst = a.y + static_cast<size_t>(row) * a.N + col;
          if (by_hand) {
            const int id = l.adapter[d];
            for (int i = 0; i < 32 && col + i < a.N; ++i) {
              const uint16_t* br = a.b + (static_cast<size_t>(id) * a.N + col + i) * a.R;
              float v = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == i) v = __uint_as_float(r[j]);
              bool odd = false;
              for (int j = 0; j < a.R; ++j) odd |= (br[j] & 0x7f80u) == 0x7f80u;
              if (odd) {
                for (int j = 0; j < a.R; ++j)
                  v = fmaf(a.low[static_cast<size_t>(row) * a.R + j], bf16_bits_to_f32(br[j]), v);
              }
              dst[i] = f32_to_bf16_bits(v);
            }
          } else {
            uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(r[8 * v + 2 * i]))) |
                       (static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(r[8 * v + 2 * i + 1])))
                        << 16);
              if (col + 8 * v < a.N) d4[v] = make_uint4(w[0], w[1], w[2], w[3]);  // N % 8 == 0
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&listempty[b]);
    }
  } else if (warp < kPassWarp0) {
    // --------------------------- the tile's adapters and the low-rank A operand
    const int i = threadIdx.x - 32 * kFillWarp0;  // row of this CTA
    uint32_t it = 0, uc = 0, gpar = 0, bpar = 0;  // parities of sgo[s] and bland[s], bit s
    bool ok = true;
    grid_wait();  // the low-rank vectors are complete
    for (int t = pair; t < tiles; t += pairs, ++uc) {
      const int b = uc & 1;
      const int m0 = (t / tn) * kTlRows;
      TileList& l = lists[b];
      // the four warps leave together or go on together: barriers follow
      if (!fill_all(ok && mbar_wait(&listempty[b], ((uc >> 1) & 1u) ^ 1u, wt))) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = i + 128 * h;
        int id = -1;
        if (m0 + r < a.T) {
          id = checked_id(a.ids[m0 + r], a.adapters);
        }
        l.ids[r] = id;
      }
      fill_barrier();
      // a row leads when no row before it has its adapter
      int first[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = i + 128 * h;
        const int id = l.ids[r];
        int f = r;
        if (id >= 0) {
          for (int j = 0; j < r; j += 4) {
            const int4 o = *reinterpret_cast<const int4*>(&l.ids[j]);
            const int hit = o.x == id ? 0 : o.y == id ? 1 : o.z == id ? 2 : o.w == id ? 3 : 4;
            if (hit < 4) {
              f = min(f, j + hit);
              break;
            }
          }
        }
        __syncwarp();
        const uint32_t m = __ballot_sync(0xffffffffu, id >= 0 && f == r);
        if ((i & 31) == 0) l.leads[r >> 5] = m;
        first[h] = id >= 0 ? f : -1;
      }
      fill_barrier();
      int my_d = -1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = i + 128 * h;
        if (first[h] < 0) continue;
        int d = __popc(l.leads[first[h] >> 5] & ((1u << (first[h] & 31)) - 1u));
        for (int w = 0; w < (first[h] >> 5); ++w) d += __popc(l.leads[w]);
        if (first[h] == r) l.adapter[d] = l.ids[r];
        if (h == static_cast<int>(rank)) my_d = d;
      }
      l.of_row[i] = static_cast<int16_t>(my_d);
      if (i == 0) {
        int n = 0;
        for (int w = 0; w < kTlRows / 32; ++w) n += __popc(l.leads[w]);
        l.n = n;
      }
      fill_barrier();
      if ((i & 31) == 0) mbar_arrive(&listfull[b]);
      const int n = l.n;
      const int row = m0 + static_cast<int>(rank) * 128 + i;
      it += ksteps;
      // Looks over the B of slot s, after which the stage's operands are there.
      auto finish = [&](int s, int d) {
        const bool got = mbar_wait(&bland[s], (bpar >> s) & 1u, wt);
        bpar ^= 1u << s;
        if (!__all_sync(0xffffffffu, got)) return false;
        uint8_t* B = smem + s * S::kStageBytes + kTlABytes;
        if (i < S::kBRows) {
          uint32_t odd = 0;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(B + i * 128 + ((c ^ (i & 7)) << 4));
            odd |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
          }
          if (odd & 0x80008000u) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(B + i * 128 + (c << 4)) = make_uint4(0, 0, 0, 0);
            for (uint32_t to = 0; to < 2; ++to)
              asm volatile("st.relaxed.cluster.shared::cluster.u16 [%0], %1;" ::"r"(
                               mapa_shared(&bad[uc % kBadRing][d], to)),
                           "h"(static_cast<uint16_t>(uc + 1))
                           : "memory");
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
          }
        }
        fence_async_smem();  // this row of A and of B, for the MMAs
        __syncwarp();
        if (lane == 0) mbar_arrive(&awrote[s]);
        return true;
      };
      int last = -1, last_d = 0;  // the stage whose A is written and B not yet seen
      for (int blk = 0; blk < blocks && ok; ++blk) {
        // this row's vector: hi and lo of columns 64 blk .. (or all, R <= 32)
        constexpr int kWords = WIDE ? 32 : 16;
        uint32_t hi[kWords], lo[kWords];
        if (n == 0) break;
#pragma unroll
        for (int j = 0; j < kWords; j += 2) {
          const int c = 64 * blk + 2 * j;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (my_d >= 0 && c < a.R)  // R % 8 == 0
            v = *reinterpret_cast<const float4*>(a.low + static_cast<size_t>(row) * a.R + c);
          uint32_t h0, l0, h1, l1;
          split_bf16(v.x, h0, l0);
          split_bf16(v.y, h1, l1);
          hi[j] = h0 | (h1 << 16);
          lo[j] = l0 | (l1 << 16);
          split_bf16(v.z, h0, l0);
          split_bf16(v.w, h1, l1);
          hi[j + 1] = h0 | (h1 << 16);
          lo[j + 1] = l0 | (l1 << 16);
        }
        for (int e = 0; e < n * parts && ok; ++e, ++it) {
          const int d = e / parts, part = e % parts;
          const int s = it % kTlStages;
          const bool got = mbar_wait(&sgo[s], (gpar >> s) & 1u, wt);
          gpar ^= 1u << s;
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          uint8_t* A = smem + s * S::kStageBytes;
          // 16-byte chunk c of row i sits at chunk c ^ (i & 7)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (d == my_d) {
              if constexpr (WIDE) {
                v = part == 0 ? make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3])
                              : make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
              } else {
                const int q = 4 * (c & 3);
                v = c < 4 ? make_uint4(hi[q], hi[q + 1], hi[q + 2], hi[q + 3])
                          : make_uint4(lo[q], lo[q + 1], lo[q + 2], lo[q + 3]);
              }
            }
            *reinterpret_cast<uint4*>(A + i * 128 + ((c ^ (i & 7)) << 4)) = v;
          }
          // the stage before, whose B has had this long to arrive
          if (last >= 0) ok = finish(last, last_d);
          last = s;
          last_d = d;
        }
      }
      if (ok && last >= 0) ok = finish(last, last_d);
    }
  } else if (lane == 0) {
    // ------------------- low-rank stages, every kPassWarps-th, to the MMA warp
    const uint32_t leader_passed = mapa_shared(passed, 0);
    uint32_t it = 0, uc = 0, par = 0, count = 0;  // par: parities of awrote[s] and passed[s]
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs, ++uc) {
      const int b = uc & 1;
      if (!mbar_wait(&listfull[b], (uc >> 1) & 1u, wt)) break;
      const int stages = lists[b].n * blocks * parts;
      mbar_arrive(&listempty[b]);
      it += ksteps;
      for (int e = 0; e < stages; ++e, ++it, ++count) {
        const int s = it % kTlStages;
        const uint32_t ph = (par >> s) & 1u;
        par ^= 1u << s;
        if (count % kPassWarps != static_cast<uint32_t>(warp - kPassWarp0)) continue;
        if (!mbar_wait(&awrote[s], ph, wt) || (rank == 0 && !mbar_wait(&passed[s], ph, wt))) {
          ok = false;
          break;
        }
        if (rank == 0) {
          mbar_acquire_cluster(&passed[s], ph);
          mbar_arrive(&full[s]);
        } else {
          mbar_arrive_remote_release(leader_passed + 8u * s);
        }
      }
    }
  }
  // every MMA is done before rank 0 arrives, every copy landed and every
  // epilogue read its accumulators before either CTA passes
  if (warp == 1 && rank == 0) mbar_drain(&mma_done, 0, status);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    mbar_drain(&mma_done, 0, status);  // rank 0's last commit has arrived here too
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

namespace {

template <int BN, bool WIDE, bool STALL = false>
int launch_tile(const AdapterArgs& a, int* status, cudaStream_t st,
                const AdapterStall* stall = nullptr) {
  CUtensorMap mx, mw, mb;
  const uint64_t dims[3] = {static_cast<uint64_t>(a.R), static_cast<uint64_t>(a.N),
                            static_cast<uint64_t>(a.adapters)};
  const uint64_t strides[2] = {static_cast<uint64_t>(a.R) * 2,
                               static_cast<uint64_t>(a.N) * a.R * 2};
  const uint32_t box[3] = {64, BN / 2, 1};
  if (!adapter_map_rows(&mx, a.x, a.T, a.K, 128) || !adapter_map_rows(&mw, a.w, a.N, a.K, BN / 2) ||
      !encode_tensor_map(&mb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.b, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B))
    return MOE_ERR_CUDA;
  auto kern = adapter_tile_kernel<BN, WIDE, STALL>;
  MOE_TRY_CUDA(adapter_smem(reinterpret_cast<const void*>(kern)));
  const long tiles = static_cast<long>((a.N + BN - 1) / BN) * ((a.T + kTlRows - 1) / kTlRows);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<long>(tiles, num_sms() / 2)));
  cfg.blockDim = dim3(tile_threads(WIDE));
  cfg.dynamicSmemBytes = TileShape<BN>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  set_adapter_attrs(&cfg, attr, 0);  // the cluster is the kernel's own
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kern, mx, mw, mb, a, status,
                                  STALL ? stall->wait_ns : static_cast<long long>(kDefaultWaitNs),
                                  STALL ? stall->stage : 0));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

int launch_adapter_tile(const AdapterArgs& a, int* status, cudaStream_t st,
                        const AdapterStall* stall) {
  if (stall && stall->kernel == 1)  // one width of the two
    return a.R > 32 ? launch_tile<192, true, true>(a, status, st, stall)
                    : launch_tile<192, false, true>(a, status, st, stall);
  // the width whose last wave of tiles leaves fewer columns idle
  const long pairs = num_sms() / 2, tm = (a.T + kTlRows - 1) / kTlRows;
  auto cost = [&](long bn) {
    const long tiles = tm * ((a.N + bn - 1) / bn);
    return (tiles + pairs - 1) / pairs * bn;
  };
  const bool wide = a.R > 32;
  if (cost(192) < cost(256))
    return wide ? launch_tile<192, true>(a, status, st) : launch_tile<192, false>(a, status, st);
  return wide ? launch_tile<256, true>(a, status, st) : launch_tile<256, false>(a, status, st);
}

}  // namespace moe
