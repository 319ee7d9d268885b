// A shared projection with the low-rank adapters of many requests:
//   y[t] = x[t] W^T + s_a (x[t] A_a^T) B_a^T,  a = ids[t]  (-1: no adapter),
// x bf16 [T, K], W bf16 [N, K], A bf16 [adapters, R, K], B bf16 [adapters, N,
// R], y bf16 [T, N]; fp32 accumulation, one rounding of the sum.  MoeBlock has
// it in place of the latent projections ("Kimi K3 latent up-projection" page,
// KimiSparseMoeBlock listing); no page has adapters.
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
// Lines between the kernels, us in a graph (K 7168, N 3584, R 16 but where said).
// Split against tile kernel: T 256 of one adapter 35.6 against 36.2 (K 3584, N
// 7168: 44.6 against 23.6), of 64 adapters 39.6 against 104; T 512 of one 55.5
// against 36.3, of 8 64.7 against 40, of 64 81 against 105.  What decides is the
// number of distinct adapters, which the host does not know.
//
//  - adapter_split_kernel, few tokens: bound by reading W.  128 rows of W are
//    the MMA's M side and up to 128 tokens its N side; the K range is split
//    over the CTAs of a cluster, which add their accumulators through
//    distributed shared memory in the order of their ranks, so that 100 and
//    more SMs stream W whatever N is.  The low-rank term is a dot product of
//    length R per output with each token's own rows of B, on mma.sync: 16 rows
//    of B are the M side, and p as hi + lo, both bf16, two of the N columns.
//    K = 7168, N = 3584 (51 MB of W), rank 16: one token 14.4 to 15.2 us, of
//    which W takes 6.6 at the HBM rate, the prologue 2 and the clusters' sum 3 to
//    4; 32 tokens with an adapter each (K = 3584, N = 7168) 18.3 with the shrink,
//    9.7 of them W and the adapters; 256 tokens of rank 32 (N = 2048) 38.7.
//  - adapter_tile_kernel (adapter_tile.cu), many tokens: bound by the tensor
//    cores; the low-rank term is R more columns of K for each adapter that
//    occurs in an output tile's rows.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "adapter.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kMaxRank = 128;
constexpr int kMaxExtent = 65535 * 128;  // tokens, and columns: blocks of 128 in a grid's y

constexpr int kSpTokens = 128;   // tokens to a block, at most
constexpr int kSpWBytes = 128 * 64 * 2;
constexpr int kSpMaxCluster = 8;

// Up to here the split kernel does the shrink itself: every output tile reads the
// adapters' A again (T R of them in place of 128 rows of W a tile), one token after
// the other.  One launch against two, us in a graph / issued one by one (K 7168, N
// 3584): T 1, R 16: 14.9 / 15.8 against 14.7 / 22.6; T 2, R 32: 15.1 / 15.9 and
// 14.8 / 24.0; T 4, R 16: 21.5 / 21.3 and 15.0 / 24.2; T 8, R 8: 29 / 29 and 15.2 /
// 23.9.  K = N = 2048: T 4, R 16 9.1 / 14.7 and 9.3 / 24.0; T 8, R 8 11.5 / 14.6 and
// 9.9 / 23.1.
constexpr int kFusedTokens = 4;
constexpr int kFusedLow = 64;  // T R

bool fused(int T, int R) { return T <= kFusedTokens && T * R <= kFusedLow; }

struct SplitShape {
  int tb;      // tokens to a block (the MMA's N), a multiple of 16
  int stages;
  int cluster;  // CTAs that share an output tile, each with its K range
  uint32_t cols;  // TMEM columns
  int wave;       // tokens whose B is in one of two buffers
  int buf0, buf1;  // their offsets in shared memory
  size_t smem;
};

// By one warp: out[r] = p b[r]^T for the rows r < rows of b [rows][R] in shared
// memory (0 up to 128), p given as hi[R] and lo[R].  A lane's 16-byte loads of b
// (columns 8 (lane % 4) .. + 7 of 32) feed two MMAs, as in shrink_token.
__device__ __forceinline__ void expand_token(const uint16_t* b, int rows, int R,
                                             const uint16_t* hi, float* out) {
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int m0 = 0; m0 < 8; m0 += 4) {
    float acc[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
    for (int k = 8 * q; k - 8 * q < R; k += 32) {
      const bool in = k < R;
      // N column 0: hi, 1: lo
      const uint4 p = in && g < 2 ? *reinterpret_cast<const uint4*>(hi + g * R + k) : zero;
      uint4 w[4][2];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * (m0 + m) + 8 * h;
          w[m][h] = in && r < rows ? *reinterpret_cast<const uint4*>(b + (r + g) * R + k) : zero;
        }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        mma_bf16(acc[m], w[m][0].x, w[m][1].x, w[m][0].y, w[m][1].y, p.x, p.y);
        mma_bf16(acc[m], w[m][0].z, w[m][1].z, w[m][0].w, w[m][1].w, p.z, p.w);
      }
    }
    float v[4][2];
    bool odd = false;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[m][h] = acc[m][2 * h] + acc[m][2 * h + 1];
        odd |= !(fabsf(v[m][h]) < INFINITY);
      }
    if (q == 0) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) out[16 * (m0 + m) + 8 * h + g] = v[m][h];
    }
    if (__any_sync(0xffffffffu, odd && q == 0)) {
      __syncwarp();  // the rows above are written
      // an infinity times hi and times lo can have two signs: one product
      for (int r = 16 * m0 + lane; r < min(16 * m0 + 64, rows); r += 32) {
        float u = 0.f;
        for (int j = 0; j < R; ++j)
          u = fmaf(bf16_bits_to_f32(hi[j]) + bf16_bits_to_f32(hi[R + j]),
                   bf16_bits_to_f32(b[r * R + j]), u);
        if (!(fabsf(u) < INFINITY)) out[r] = u;
      }
    }
  }
  __syncwarp();
}

}  // namespace

// Warp 0: TMA, 1: MMA + TMEM, 4 and up: TMEM -> shared memory; all: the sums.  8
// warps where an SM is to hold a CTA of the shrink beside them, 16 elsewhere.
// FUSED: the low-rank vectors too (T R <= kFusedLow, one block of tokens).  B of
// the tokens is fetched into shared memory while W streams: a read of global
// memory at the end costs 1 us and more a token, measured.
// Cluster (x = rank, y, z): rows 128 y of W, tokens tb z; rank j takes the
// K steps [j n / cluster, (j + 1) n / cluster) of n = ceil(K / 64).
// STALL (tests only): the copies stop before stage stall_at, or (-1) those of B never
// come.
template <bool FUSED, int THREADS, bool STALL>
__global__ void __launch_bounds__(THREADS, FUSED || THREADS == 512 ? 1 : 2)
    adapter_split_kernel(const __grid_constant__ CUtensorMap mw,
                         const __grid_constant__ CUtensorMap mx, const AdapterArgs a,
                         const SplitShape sh, int* status, long long wait_ns, int stall_at) {
  constexpr int kSpThreads = THREADS;
  constexpr int kLowWarps = THREADS / 32 - 2;  // warps 2 and up
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full[8], empty[8], done, bfull[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int cta_abort;
  // The block's tokens in the order of their adapters; each rank takes a stretch of
  // it, so that tokens that share an adapter share the copy of its B: slot j holds
  // adapter slot_id[j], and local token j (order[p0 + j]) uses slot slot_of[j]
  // (slot_first[s]: the first that uses slot s).
  __shared__ __align__(16) int32_t ids[kSpTokens];
  __shared__ int16_t order[kSpTokens], slot_of[kSpTokens], slot_first[kSpTokens];
  __shared__ int32_t slot_id[kSpTokens];
  __shared__ int slots;
  __shared__ float lowp[kLowWarps + 1][kFusedLow];  // FUSED: the warps' sums, and the CTA's
  __shared__ __align__(16) uint16_t lowv[2 * kFusedLow];  // FUSED: as lows below
  __shared__ __align__(16) float lowout[kSpThreads / 32][128];  // a token's low-rank term
  const Waiter wt{&cta_abort, status, wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&mw);
    prefetch_tensor_map(&mx);
  }
  const int tb = sh.tb, stages = sh.stages;
  const int stage_bytes = kSpWBytes + tb * 128;
  const int ranks = gridDim.x, rank = blockIdx.x;
  const int n0 = blockIdx.y * 128, t0 = blockIdx.z * tb;
  const int tokens = min(tb, a.T - t0);
  const int p0 = tokens * rank / ranks;
  const int mine = tokens * (rank + 1) / ranks - p0;  // tokens of this rank
  const int rows = min(128, a.N - n0);                // N % 8 == 0
  if (FUSED) grid_wait();
  grid_launch_dependents();
  if (threadIdx.x < kSpTokens)
    ids[threadIdx.x] =
        threadIdx.x < tokens ? checked_id(a.ids[t0 + threadIdx.x], a.adapters) : INT_MAX;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    mbar_init(&bfull[0], 1);
    mbar_init(&bfull[1], 1);
    cta_abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, sh.cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;
  const int steps = (a.K + 63) / 64;
  const int s0 = steps * rank / ranks, s1 = steps * (rank + 1) / ranks;
  // B of the slots of wave w (one thread): bulk copies of whole [rows][R] blocks
  const uint32_t block = static_cast<uint32_t>(rows) * a.R * 2;
  auto fetch_wave = [&](int w) {
    const int j0 = w * sh.wave, j1 = min(slots, j0 + sh.wave);
    if (j0 >= j1) return;
    uint64_t* bar = &bfull[w & 1];
    uint8_t* buf = smem + (w & 1 ? sh.buf1 : sh.buf0);
    mbar_arrive_expect_tx(bar, (j1 - j0) * block);
    if (STALL && stall_at < 0) return;
    for (int j = j0; j < j1; ++j)
      bulk_g2s(buf + (j - j0) * 256 * a.R,
               a.b + (static_cast<size_t>(slot_id[j]) * a.N + n0) * a.R, block, bar);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      for (int k = s0; k < s1; ++k, ++it) {
        const int s = it % stages;
        if ((STALL && static_cast<int>(it) == stall_at) ||
            !mbar_wait(&empty[s], ((it / stages) & 1u) ^ 1u, wt))
          break;
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
    // sort the tokens: one counts the others before it
    const int i = threadIdx.x - 64;
    if (i < tokens) {
      const int id = ids[i];
      int p = 0;
      for (int j = 0; j < tokens; j += 4) {  // beyond the last: INT_MAX
        const int4 o = *reinterpret_cast<const int4*>(&ids[j]);
        const int v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) p += v[q] < id || (v[q] == id && j + q < i) ? 1 : 0;
      }
      order[p] = static_cast<int16_t>(i);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS - 64) : "memory");
    if (warp == 2) {
      int n = 0;
      for (int j0 = 0; j0 < mine; j0 += 32) {
        const int j = j0 + lane;
        const int id = j < mine ? ids[order[p0 + j]] : -1;
        const bool lead = id >= 0 && (j == 0 || ids[order[p0 + j - 1]] != id);
        const uint32_t m = __ballot_sync(0xffffffffu, lead);
        const int at = n + __popc(m & (0xffffffffu >> (31 - lane))) - 1;
        if (lead) {
          slot_id[at] = id;
          slot_first[at] = static_cast<int16_t>(j);
        }
        if (j < mine) slot_of[j] = static_cast<int16_t>(id >= 0 ? at : -1);
        n += __popc(m);
      }
      if (lane == 0) slots = n;
      __syncwarp();
      if (lane == 0) fetch_wave(0);
      __syncwarp();
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
          shrink_token<1>(x, A, a.K, a.R, a0, a1, out);
        else
          shrink_token<4>(x, A, a.K, a.R, a0, a1, out);
      }
    }
  }
  // every copy has landed and every MMA is done: the ring becomes the fp32
  // tile [tokens][128 columns of y]
  __syncthreads();
  mbar_drain(&done, 0, status);  // complete: each reader observes it for itself
  if (threadIdx.x == 64) fetch_wave(1);  // its buffer may be part of the ring
  __syncwarp();
  tc_fence_after();
  float* red = reinterpret_cast<float*>(smem);
  // this rank's low-rank vectors as bf16 hi and lo parts: [token][2][R]
  uint16_t* lows = FUSED ? lowv : reinterpret_cast<uint16_t*>(red + tb * 128);
  if (warp >= 4) {
    const int q = warp & 3;  // lane quarter; 16 tokens in turn
    for (int c0 = 16 * ((warp >> 2) - 1); c0 < tb; c0 += 4 * (kSpThreads / 32 - 4)) {
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
  // tensor memory goes back before the wait for the other ranks (see kSmBytes)
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, sh.cols);
  }
  cluster_sync_all();
  if (FUSED) {
    if (threadIdx.x < tokens * a.R) {
      const int id = checked_id(a.ids[threadIdx.x / a.R], a.adapters);
      float v = 0.f;
      if (id >= 0) {
        for (int r = 0; r < ranks; ++r)
          v += ld_cluster_f1(mapa_shared(&lowp[kLowWarps][threadIdx.x], r));
        if (a.scale) v *= a.scale[id];
      }
      uint32_t hi, lo;
      split_bf16(v, hi, lo);
      uint16_t* l = lowv + threadIdx.x / a.R * 2 * a.R + threadIdx.x % a.R;
      l[0] = static_cast<uint16_t>(hi);
      l[a.R] = static_cast<uint16_t>(lo);
    }
    __syncthreads();
  } else {
    // the low-rank vectors are complete: those of this rank's tokens to shared
    // memory, in one round trip (read where they are used, each token would
    // wait for its own)
    grid_wait();
    const int quads = a.R / 4;
    for (int i = threadIdx.x; i < mine * quads; i += kSpThreads) {
      const int j = i / quads, e = i % quads * 4;
      if (slot_of[j] < 0) continue;
      const float4 v = *reinterpret_cast<const float4*>(
          a.low + static_cast<size_t>(t0 + order[p0 + j]) * a.R + e);
      uint32_t h[4], l[4];
      split_bf16(v.x, h[0], l[0]);
      split_bf16(v.y, h[1], l[1]);
      split_bf16(v.z, h[2], l[2]);
      split_bf16(v.w, h[3], l[3]);
      uint16_t* o = lows + j * 2 * a.R + e;
      *reinterpret_cast<uint2*>(o) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      *reinterpret_cast<uint2*>(o + a.R) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
    }
    __syncthreads();
  }
  // token by token, each by a warp: a lane sums four columns over the cluster, in
  // the order of the ranks.  Wave w: the tokens of its slots (the first also those
  // without an adapter)
  const int n = n0 + 4 * lane;
  const bool on = n < a.N;  // N % 8 == 0: all four columns or none
  const int fetches = (slots + sh.wave - 1) / sh.wave, waves = max(1, fetches);
  int issued = min(2, fetches);  // waves whose copies thread 64 has issued
  int j0 = 0;
  bool ok = true;
  for (int w = 0; w < waves; ++w) {
    const int j1 = (w + 1) * sh.wave < slots ? slot_first[(w + 1) * sh.wave] : mine;
    const uint8_t* buf = smem + (w & 1 ? sh.buf1 : sh.buf0);
    // A wave whose B does not come is left out with all after it, and no buffer is
    // filled again: its barrier's phase is still open (the parity of the phase after
    // next would read as complete, and another arrival is one too many).
    ok = ok && __all_sync(0xffffffffu,
                          slots == 0 || mbar_wait(&bfull[w & 1], (w >> 1) & 1u, wt));
    for (int j = ok ? j0 + warp : j1; j < j1; j += kSpThreads / 32) {
      const int i = order[p0 + j], slot = slot_of[j];
      float4 o[kSpMaxCluster];
#pragma unroll
      for (int r = 0; r < kSpMaxCluster; ++r)
        if (r < ranks) o[r] = ld_cluster_f4(mapa_shared(red + i * 128 + 4 * lane, r));
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (slot >= 0) {
        expand_token(reinterpret_cast<const uint16_t*>(buf + (slot - w * sh.wave) * 256 * a.R),
                     rows, a.R,
                     lows + (FUSED ? i : j) * 2 * a.R, lowout[warp]);
        s = *reinterpret_cast<const float4*>(&lowout[warp][4 * lane]);
        __syncwarp();  // read before the next token's are written
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kSpMaxCluster; ++r)
        if (r < ranks) {
          v.x += o[r].x; v.y += o[r].y; v.z += o[r].z; v.w += o[r].w;
        }
      if (on) {
        uint2 q;
        q.x = f32_to_bf16_bits(v.x + s.x) |
              (static_cast<uint32_t>(f32_to_bf16_bits(v.y + s.y)) << 16);
        q.y = f32_to_bf16_bits(v.z + s.z) |
              (static_cast<uint32_t>(f32_to_bf16_bits(v.w + s.w)) << 16);
        *reinterpret_cast<uint2*>(a.y + static_cast<size_t>(t0 + i) * a.N + n) = q;
      }
      __syncwarp();  // whole again for the next token's MMAs
    }
    j0 = j1;
    if (w + 2 < waves) {  // the wave's buffer takes the one after next
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      if (threadIdx.x == 64 && ok) {
        fetch_wave(w + 2);
        issued = w + 3;
      }
    }
  }
  // the copies land before the CTA can leave; on the normal path they have
  if (threadIdx.x == 64)
    for (int w = max(0, issued - 2); w < issued; ++w)
      mbar_drain(&bfull[w & 1], (w >> 1) & 1u, status);
  cluster_sync_all();  // no CTA leaves while another reads its tile
}

// Asked of the runtime once for each kernel, cluster size and amount of shared
// memory; what a device holds does not change.  A query that fails is an error
// and is not kept: the cluster's size decides the order of the sums.
cudaError_t adapter_cluster(const void* kernel, int threads, int smem, int clusters, int most,
                            int* size) {
  struct Known {
    const void* kernel;
    int device, threads, smem, size, held;
  };
  constexpr int kRoom = 1024;  // beyond, the answer is not kept
  static std::mutex mu;
  static Known known[kRoom];
  static int kept = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (*size = most; *size > 1; --*size) {
    int held = -1;
    for (int i = 0; i < kept && held < 0; ++i) {
      const Known& k = known[i];
      if (k.kernel == kernel && k.device == device && k.threads == threads && k.smem == smem &&
          k.size == *size)
        held = k.held;
    }
    if (held < 0) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(*size);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = *size;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&held, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (kept < kRoom) known[kept++] = Known{kernel, device, threads, smem, *size, held};
    }
    if (held >= clusters) return cudaSuccess;
  }
  return cudaSuccess;
}

namespace {

int split_tiles(int T, int N) {
  return (N + 127) / 128 * ((T + kSpTokens - 1) / kSpTokens);
}

SplitShape split_shape(int T, int R, int cluster) {
  SplitShape s;
  const bool beside = adapter_beside(T, R);
  const int blocks = (T + kSpTokens - 1) / kSpTokens;
  s.tb = ((T + blocks - 1) / blocks + 15) / 16 * 16;
  s.cluster = cluster;
  const int stage = kSpWBytes + s.tb * 128;
  // ~92 KiB in flight an SM, and of B what leaves room for a CTA of the shrink
  s.stages = std::min(8, (beside ? 104 : 132) * 1024 / stage);
  s.cols = 32;
  while (s.cols < static_cast<uint32_t>(s.tb)) s.cols *= 2;
  // the ring, and in its place the fp32 tile and the rank's low-rank vectors
  const int most = (s.tb + s.cluster - 1) / s.cluster;  // tokens of a rank
  const int tail = s.tb * 512 + most * R * 4;
  const int ring = std::max(s.stages * stage, (tail + 1023) / 1024 * 1024);
  // B: a buffer of its own; the second in what the tail leaves of the ring, if
  // it takes a token, else in the first one's upper half
  const int token = 256 * R;
  const int bytes = std::min(std::max(beside && T > 64 ? 32 * 1024 : 64 * 1024, 2 * token), most * token);
  const int fit = bytes / token, rest = (ring - tail) / token;
  s.buf0 = ring;
  if (fit >= most || rest >= 1) {
    s.wave = fit >= most ? most : std::min(fit, rest);
    s.buf1 = tail;
  } else {
    s.wave = fit / 2;  // at least two tokens fit
    s.buf1 = ring + s.wave * token;
  }
  s.smem = static_cast<size_t>(ring) + bytes + 1024;
  return s;
}

template <bool FUSED, int THREADS, bool STALL = false>
int launch_split(const AdapterArgs& a, int* status, cudaStream_t st,
                 const AdapterStall* stall = nullptr) {
  auto kern = adapter_split_kernel<FUSED, THREADS, STALL>;
  // at most one CTA to an SM (a second one on some would take twice the time),
  // and as many clusters as the device holds at once
  const int tiles = split_tiles(a.T, a.N);
  const int most = std::min({kSpMaxCluster, std::max(1, num_sms() / tiles), (a.K + 63) / 64});
  SplitShape sh = split_shape(a.T, a.R, most);
  MOE_TRY_CUDA(adapter_smem(reinterpret_cast<const void*>(kern)));
  int held = 1;
  MOE_TRY_CUDA(adapter_cluster(reinterpret_cast<const void*>(kern), THREADS,
                               static_cast<int>(sh.smem), tiles, most, &held));
  if (held < most) sh = split_shape(a.T, a.R, held);  // fewer ranks, more tokens to each
  CUtensorMap mw, mx;
  if (!adapter_map_rows(&mw, a.w, a.N, a.K, 128) || !adapter_map_rows(&mx, a.x, a.T, a.K, sh.tb))
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sh.cluster, (a.N + 127) / 128, (a.T + sh.tb - 1) / sh.tb);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = sh.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  set_adapter_attrs(&cfg, attr, sh.cluster);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kern, mw, mx, a, sh, status,
                                  STALL ? stall->wait_ns : static_cast<long long>(kDefaultWaitNs),
                                  !STALL ? 0 : stall->kernel == 2 ? -1 : stall->stage));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_adapter_linear_workspace_size(int T, int K, int N, int R) {
  (void)K;
  (void)N;
  if (T <= 0 || R <= 0 || fused(T, R)) return 0;
  return align_up(static_cast<size_t>(T) * R * sizeof(float), 256);
}

// moe_adapter_linear; stall: moe_adapter_linear_stall_selftest.
static int adapter_linear(const uint16_t* x, const uint16_t* w, const uint16_t* lora_a,
                          const uint16_t* lora_b, const int32_t* ids, const float* scale, int T,
                          int K, int N, int R, int adapters, uint16_t* y, void* ws,
                          size_t ws_bytes, const AdapterStall* stall, void* stream) {
  if (T < 0 || K <= 0 || N <= 0 || R <= 0 || adapters <= 0) return MOE_ERR_INVALID;
  if (K % 32 != 0 || N % 8 != 0 || R % 8 != 0 || R > kMaxRank) return MOE_ERR_UNSUPPORTED;
  if (T > kMaxExtent || N > kMaxExtent) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const size_t need = moe_adapter_linear_workspace_size(T, K, N, R);
  if (!x || !w || !lora_a || !lora_b || !ids || !y || (need && !ws)) return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16) ||
      !aligned(ids, 4) || !aligned(scale, 4) || !aligned(y, 16) || !aligned(ws, 256))
    return MOE_ERR_INVALID;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  // CTAs write y and the workspace while others still read the inputs
  const size_t y_bytes = static_cast<size_t>(T) * N * 2;
  const struct {
    const void* p;
    size_t bytes;
  } inputs[] = {{x, static_cast<size_t>(T) * K * 2},
                {w, static_cast<size_t>(N) * K * 2},
                {lora_a, static_cast<size_t>(adapters) * R * K * 2},
                {lora_b, static_cast<size_t>(adapters) * N * R * 2},
                {ids, static_cast<size_t>(T) * 4},
                {scale, scale ? static_cast<size_t>(adapters) * 4 : 0}};
  for (const auto& in : inputs)
    if (overlap(in.p, in.bytes, y, y_bytes) || overlap(in.p, in.bytes, ws, need))
      return MOE_ERR_INVALID;
  if (overlap(y, y_bytes, ws, need)) return MOE_ERR_INVALID;
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
  if (fused(T, R)) {
    if (stall && stall->kernel != 0) return launch_split<true, 256, true>(a, status, st, stall);
    return launch_split<true, 256>(a, status, st);
  }
  const int rc = launch_adapter_shrink(a, status, st, stall);
  if (rc) return rc;
  if (T > kSplitTokens) return launch_adapter_tile(a, status, st, stall);
  if (stall && stall->kernel != 0)
    return adapter_beside(T, R) ? launch_split<false, 256, true>(a, status, st, stall)
                                : launch_split<false, 512, true>(a, status, st, stall);
  return adapter_beside(T, R) ? launch_split<false, 256>(a, status, st)
                              : launch_split<false, 512>(a, status, st);
}

extern "C" int moe_adapter_linear(const uint16_t* x, const uint16_t* w, const uint16_t* lora_a,
                                  const uint16_t* lora_b, const int32_t* ids, const float* scale,
                                  int T, int K, int N, int R, int adapters, uint16_t* y, void* ws,
                                  size_t ws_bytes, void* stream) {
  moe::Range range_("moe_adapter_linear");
  return adapter_linear(x, w, lora_a, lora_b, ids, scale, T, K, N, R, adapters, y, ws, ws_bytes,
                        nullptr, stream);
}

extern "C" int moe_adapter_linear_stall_selftest(
    const uint16_t* x, const uint16_t* w, const uint16_t* lora_a, const uint16_t* lora_b,
    const int32_t* ids, const float* scale, int T, int K, int N, int R, int adapters, int kernel,
    int stall_stage, int64_t limit_ns, uint16_t* y, void* ws, size_t ws_bytes, void* stream) {
  moe::Range range_("moe_adapter_linear_stall_selftest");
  if (kernel < 0 || kernel > 2 || stall_stage < 0) return MOE_ERR_INVALID;
  if (limit_ns < 1000 || limit_ns > 5000000000LL) return MOE_ERR_INVALID;
  if ((kernel == 0 && fused(T, R)) || (kernel == 2 && T > kSplitTokens))
    return MOE_ERR_UNSUPPORTED;  // no such kernel in this call
  const AdapterStall stall{kernel, stall_stage, limit_ns};
  return adapter_linear(x, w, lora_a, lora_b, ids, scale, T, K, N, R, adapters, y, ws, ws_bytes,
                        &stall, stream);
}
