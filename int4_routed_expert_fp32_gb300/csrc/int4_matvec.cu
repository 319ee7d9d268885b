// y = x W^T for packed int4 weights with a bf16 scale per 32 columns and at most 16 rows x.
//
// The weights are read once and bound the time from some tens of MB on; below that it is
// latency: launch, one trip to HBM, one reduction.  A cluster of CTAs takes blocks of
// 32 rows of W and splits K; of a CTA's eight warps some split its columns, the others
// have other blocks.  A warp copies its own weights two or three steps of 2 KB ahead
// (cp.async), on from one block into the next.  What a warp copies it reads
// itself, so no warp waits for another before the sums are joined: over the warps in
// shared memory, over the cluster in that of its CTAs, both in a fixed order.
//
// A CTA turns its columns of the tokens into fp16 in shared memory first, in the order in
// which a packed word pairs its nibbles, each token's 128 columns scaled by a power of
// two of their own (exact, undone in fp32); the weights' first copies are under way
// meanwhile.  Where they do not fit, it goes through them in slices.
//
// Products: m16n8k16 MMAs on the nibbles as fp16, 1032 + q and 72 + q, exactly; the
// accumulator starts from minus the constants' part (one value for a token and group),
// and each group's sum is scaled and added in fp32.  One ldmatrix gives a lane the
// words of two groups; the two row tiles of a block share the tokens' fragments, whose
// reads of shared memory cost more than the weights' own for 16 tokens.
#include <cuda_fp16.h>

#include <atomic>

#include "adapter.cuh"
#include "common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTiles = 2;                        // row tiles of a block
constexpr int kRows = 16 * kTiles;
constexpr int kStepWords = kRows * 64;           // bytes of packed weights
constexpr int kScalePitch = 12;                  // 4 scales of a row in 4-byte pieces
constexpr int kStepBytes = kStepWords + kRows * kScalePitch;
constexpr int kMaxTokens = 16;
constexpr int kMostBlocks = 16;                  // of a cluster: their sums are in shared memory
constexpr int kMostColumns = 1 << 20, kMostRows = 1 << 30;
constexpr int kMostCluster = 8;
constexpr int kSumPitch = kRows + 4;             // lanes' tokens and rows in different banks
constexpr int kPerSm = 113 * 1024;               // shared memory with which two CTAs fit an SM
constexpr int kLoads = 4;                        // 16-byte loads of x under way in a thread

// Steps of 128 columns that a warp copies ahead.  16 tokens need the room for themselves.
__host__ __device__ constexpr int depth(int T) { return T <= 8 ? 3 : 2; }

struct MatvecArgs {
  const uint16_t* x;
  const uint8_t* w;
  const uint8_t* scale;
  uint16_t* y;
  int64_t x_ld;
  int T, N, K;
  int slice;     // columns of a slice, a multiple of 128
  int slices;    // of K: CTA r of a cluster has slices r, r + ranks, ...
  int ranks;     // CTAs of a cluster
  int split;     // warps that share a slice's columns
  int blocks;    // blocks of a cluster
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "l"(policy)
               : "memory");
}

__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Nibbles of a word as fp16 pairs (columns 0 4, 1 5, 2 6, 3 7): 1032 + q in the even
// pairs, 72 + q in the odd ones.  The second constant of each operation is in a
// register that the compiler does not see through, as an instruction takes only one
// immediate.
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&q)[4]) {
  const uint32_t w8 = w >> 8;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0x6a;" : "=r"(q[0]) : "r"(w), "r"(lo));  // (w & a) ^ b
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0x6a;" : "=r"(q[1]) : "r"(w), "r"(hi));
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0x6a;" : "=r"(q[2]) : "r"(w8), "r"(lo));
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0x6a;" : "=r"(q[3]) : "r"(w8), "r"(hi));
}

// The steps of 128 columns of one warp, on a block and slice.
struct Item {
  int row0;   // first row of the block
  int col0;   // first column
  int steps;
};

// Bytes of a token's row in shared memory: rows 64 bytes apart in the banks.
__host__ __device__ __forceinline__ int row_pitch(int slice) { return slice * 2 + 64; }

struct Layout {
  int start, unit, steps, red, sums, total;
  __host__ __device__ __forceinline__ explicit Layout(const MatvecArgs& a) {
    const int padded = (a.T + 7) / 8 * 8;
    start = a.T * row_pitch(a.slice);  // [slice / 32][padded / 2]: values of two tokens, twice
    unit = start + a.slice / kGroup * padded * 8;  // [slice / 128][padded]: undoes their scaling
    steps = unit + a.slice / 128 * padded * 4;     // the warps' steps
    red = steps + kWarps * depth(a.T) * kStepBytes;  // [warp][T][kSumPitch]
    sums = red + (a.split > 1 ? kWarps * a.T * kSumPitch * 4 : 0);  // [blocks][T][kSumPitch]
    total = sums + a.blocks * a.T * kSumPitch * 4;
  }
};

template <int NB, bool kScales8>
__global__ void __launch_bounds__(kThreads, 2) int4_matvec_kernel(const MatvecArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const Layout lay(a);
  constexpr int kPad = NB * 8, kDepth = depth(kPad);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int ks = warp & (a.split - 1), rb = warp / a.split, abreast = kWarps / a.split;
  const int groups = a.K / kGroup;
  const int rank = a.ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int block0 = blockIdx.x / a.ranks * a.blocks;
  const int blocks = min(a.blocks, (a.N + kRows - 1) / kRows - block0);
  const int slices = (a.slices - rank + a.ranks - 1) / a.ranks;  // this CTA's
  const int turns = (blocks + abreast - 1) / abreast;            // of a slice
  const uint64_t once = [] {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
  }();
  uint32_t magic_lo, magic_hi;
  asm volatile("mov.b32 %0, 0x64086408;" : "=r"(magic_lo));
  asm volatile("mov.b32 %0, 0x54805480;" : "=r"(magic_hi));

  auto item_of = [&](int turn) {  // turns count on over the slices
    Item it;
    const int sl = turn / turns, b = (turn - sl * turns) * abreast + rb;
    const int col0 = (rank + sl * a.ranks) * a.slice;
    const int steps = (min(a.slice, a.K - col0) + 127) / 128;
    const int each = (steps + a.split - 1) / a.split;
    it.steps = b < blocks ? max(0, min(each, steps - ks * each)) : 0;
    it.row0 = (block0 + b) * kRows;
    it.col0 = col0 + ks * each * 128;
    return it;
  };
  // The copies run ahead of the products through the same steps.  Where they are:
  int to_turn = -1, to_steps = 0, to_rows = 0, to_groups = 0, to_slot = 0;
  const uint8_t* to_w = nullptr;
  int64_t to_scale = 0;  // byte offset
  const int64_t rows8 = (int64_t)a.K * 4;  // bytes of 8 rows
  uint8_t* mine = smem + lay.steps + warp * kDepth * kStepBytes;
  // The next step: 16-byte pieces of rows swizzled by row / 2, and the scales.  Rows
  // behind the last and columns behind the last are left as they are.
  auto load = [&] {
    while (to_steps == 0) {
      if (++to_turn >= turns * slices) {
        to_steps = -1;
        break;
      }
      const Item it = item_of(to_turn);
      to_steps = it.steps;
      to_rows = a.N - it.row0;
      to_groups = groups - it.col0 / kGroup;
      to_w = a.w + (int64_t)(it.row0 + g) * (a.K / 2) + it.col0 / 2 + t * 16;
      to_scale = ((int64_t)(it.row0 + lane) * groups + it.col0 / kGroup) * 2;
    }
    if (to_steps > 0) {
      uint8_t* st = mine + to_slot * kStepBytes;
      const uint32_t to = smem_u32(st);
      const uint8_t* w = to_w;
#pragma unroll
      for (int h = 0; h < 2 * kTiles; ++h) {
        const int r = g + 8 * h;
        if (t < to_groups && r < to_rows) copy16(to + r * 64 + ((t ^ (r >> 1 & 3)) << 4), w, once);
        w += rows8;
      }
      if (lane < to_rows) {
        if (kScales8) {
          copy8(to + kStepWords + lane * 8, a.scale + to_scale);
        } else {
          // at most 8 bytes, which begin on 4 bytes or 2 behind them
          const int64_t word = to_scale & ~3LL, end = to_scale + 2 * min(to_groups, 4);
          uint8_t* dst = st + kStepWords + lane * kScalePitch;
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            if (word + 4 * p >= end) continue;
            if (word + 4 * p + 4 <= (int64_t)a.N * groups * 2)
              cp_async_4(dst + 4 * p, a.scale + word + 4 * p);
            else  // the last scale of an odd number
              *reinterpret_cast<uint16_t*>(dst + 4 * p) =
                  *reinterpret_cast<const uint16_t*>(a.scale + word + 4 * p);
          }
        }
      }
      to_w += 64;
      to_scale += 8;
      to_groups -= 4;
      --to_steps;
      to_slot = to_slot + 1 == kDepth ? 0 : to_slot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  grid_wait();  // x, or the weights, may come from the kernel before
  grid_launch_dependents();
  // the first copies of weights; x is made ready meanwhile
#pragma unroll 1
  for (int j = 0; j < kDepth; ++j) load();

  float* start = reinterpret_cast<float*>(smem + lay.start);
  float* unit = reinterpret_cast<float*>(smem + lay.unit);
  float* red = reinterpret_cast<float*>(smem + lay.red);
  float* sums = reinterpret_cast<float*>(smem + lay.sums);
  const int pitch = row_pitch(a.slice);
  int slot = 0;
#pragma unroll 1
  for (int turn = 0; turn < turns * slices; ++turn) {
    if (turn % turns == 0) {
      // x of this slice as fp16 in pair order; 16 lanes have the 128 columns of a scale
      const int col0 = (rank + turn / turns * a.ranks) * a.slice, cols = min(a.slice, a.K - col0);
      const int pieces = (cols + 127) / 128 * 16, all = a.T * pieces;
      if (turn > 0) __syncthreads();  // the slice before has been read
#pragma unroll 1
      for (int base = tid; base - lane < all; base += kLoads * kThreads) {
        uint4 v[kLoads];
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          const int i = base + l * kThreads, k = i / pieces, c = i - k * pieces;
          v[l] = make_uint4(0u, 0u, 0u, 0u);
          if (i < all && 8 * c < cols)
            v[l] = __ldcg(reinterpret_cast<const uint4*>(a.x + k * a.x_ld + col0 + 8 * c));
        }
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          const int i = base + l * kThreads, k = i / pieces, c = i - k * pieces;
          if (i - lane >= all) break;  // of the whole warp
          const uint32_t w[4] = {v[l].x, v[l].y, v[l].z, v[l].w};
          uint32_t m = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            m = max(m, w[j] << 16 & 0x7fff0000u);
            m = max(m, w[j] & 0x7fff0000u);
          }
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
          // a power of two that brings the largest value to [2^14, 2^15), at most 2^126; 1
          // where it is 0 or not finite
          const int field = static_cast<int>(m >> 23);
          const int up = m == 0u || field == 255 ? 127 : min(127 + 14 + 127 - field, 253);
          const float by = __uint_as_float(static_cast<uint32_t>(up) << 23);
          __half2 p[4];
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // columns j and j + 4
            const uint32_t lo = (w[j >> 1] >> (16 * (j & 1))) << 16;
            const uint32_t hi = (w[2 + (j >> 1)] >> (16 * (j & 1))) << 16;
            p[j] = __floats2half2_rn(__uint_as_float(lo) * by, __uint_as_float(hi) * by);
            s = fmaf(j & 1 ? -72.f : -1032.f, __low2float(p[j]) + __high2float(p[j]), s);
          }
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          if (i < all) {
            *reinterpret_cast<uint4*>(smem + k * pitch + 16 * c) = *reinterpret_cast<const uint4*>(p);
            if (!(c & 3)) {
              float* to = start + ((c >> 2) * (kPad / 2) + (k >> 1)) * 4 + (k & 1);
              to[0] = s;
              to[2] = s;
            }
            if (!(c & 15))
              unit[(c >> 4) * kPad + k] = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
          }
        }
      }
      __syncthreads();
    }
    const Item cur = item_of(turn);
    const int first = (cur.col0 / 128 - (rank + turn / turns * a.ranks) * (a.slice / 128));  // step
    const uint8_t* xs[NB];  // the lane's fragments of the step, of tokens 8n + g
#pragma unroll
    for (int n = 0; n < NB; ++n)  // a token that is not there is the last one: no column of
      xs[n] = smem + min(8 * n + g, a.T - 1) * pitch + first * 256 + t * 16;  // the product
    const float* cs = start + first * (8 * kPad) + t * 4;                     // reaches another
    const float* us = unit + first * kPad + 2 * t;
    int left = groups - cur.col0 / kGroup;
    float acc[kTiles][NB][4];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
#pragma unroll 1
    for (int j = 0; j < cur.steps; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      __syncwarp();
      const uint8_t* st = mine + slot * kStepBytes;
      // two words with the four scales of each of the lane's rows
      uint32_t sc[2 * kTiles][2];
#pragma unroll
      for (int h = 0; h < 2 * kTiles; ++h) {
        if (kScales8) {
          const uint2 v = *reinterpret_cast<const uint2*>(st + kStepWords + (g + 8 * h) * 8);
          sc[h][0] = v.x;
          sc[h][1] = v.y;
        } else {
          const uint32_t* v =
              reinterpret_cast<const uint32_t*>(st + kStepWords + (g + 8 * h) * kScalePitch);
          const int odd = ((cur.row0 + g + 8 * h & groups) + groups - left & 1) * 16;
          sc[h][0] = __funnelshift_r(v[0], v[1], odd);
          sc[h][1] = __funnelshift_r(v[1], v[2], odd);
          // groups behind the last: x is zero there, whatever the words are, which must not
          // meet a scale that is not finite
          if (left < 4) {
            if (left < 2) sc[h][0] &= 0xffffu;
            sc[h][1] = left < 3 ? 0u : sc[h][1] & 0xffffu;
          }
        }
      }
      float part[kTiles][NB][4];  // set by the first group
#pragma unroll
      for (int pair = 0; pair < 2; ++pair) {
        uint32_t wr[kTiles][4];
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const int r = 16 * m + (lane & 15);
          const uint32_t from =
              smem_u32(st) + r * 64 + (((2 * pair + (lane >> 4)) ^ (r >> 1 & 3)) << 4);
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                       : "=r"(wr[m][0]), "=r"(wr[m][1]), "=r"(wr[m][2]), "=r"(wr[m][3])
                       : "r"(from)
                       : "memory");
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int gr = 2 * pair + h;
          uint4 v[NB];
          float4 c[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            v[n] = *reinterpret_cast<const uint4*>(xs[n] + gr * 64);
            c[n] = *reinterpret_cast<const float4*>(cs + gr * (2 * kPad) + 16 * n);
          }
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            uint32_t lo[4], hi[4];
            nibbles(wr[m][2 * h], magic_lo, magic_hi, lo);
            nibbles(wr[m][2 * h + 1], magic_lo, magic_hi, hi);
            const uint32_t w0 = sc[2 * m][pair], w8 = sc[2 * m + 1][pair];
            const float f0 = __uint_as_float(h ? w0 & 0xffff0000u : w0 << 16);
            const float f8 = __uint_as_float(h ? w8 & 0xffff0000u : w8 << 16);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              float d[4], e[4];
              mma_f16(d, lo[0], hi[0], lo[1], hi[1], v[n].x, v[n].y, c[n].x, c[n].y, c[n].z, c[n].w);
              mma_f16(e, lo[2], hi[2], lo[3], hi[3], v[n].z, v[n].w, d[0], d[1], d[2], d[3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float f = i < 2 ? f0 : f8;
                part[m][n][i] = gr == 0 ? f * e[i] : fmaf(f, e[i], part[m][n][i]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float2 u = *reinterpret_cast<const float2*>(us + 8 * n);
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[m][n][i] = fmaf(i & 1 ? u.y : u.x, part[m][n][i], acc[m][n][i]);
        xs[n] += 256;
      }
      cs += 8 * kPad;
      us += kPad;
      left -= 4;
      slot = slot + 1 == kDepth ? 0 : slot + 1;
      __syncwarp();
      load();
    }
    // a block's sums: of its one warp, or of its warps in order; those of the slices in order
    const int sl = turn / turns, b0 = (turn - sl * turns) * abreast;
    float* to = a.split > 1 ? red + warp * a.T * kSumPitch : sums + (b0 + rb) * a.T * kSumPitch;
    if (a.split > 1 || b0 + rb < blocks) {
      const bool add = a.split == 1 && sl > 0;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = 8 * n + 2 * t + i;
          if (k >= a.T) continue;
#pragma unroll
          for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float* p = to + k * kSumPitch + 16 * m + 8 * h + g;
              const float v = acc[m][n][2 * h + i];
              *p = add ? *p + v : v;
            }
        }
    }
    if (a.split > 1) {
      __syncthreads();
      // a warp an output row's 32 values
#pragma unroll 1
      for (int q = warp; q < abreast * a.T; q += kWarps) {
        const int b = q / a.T, k = q - b * a.T;
        if (b0 + b >= blocks) continue;
        const float* from = red + (b * a.split * a.T + k) * kSumPitch + lane;
        float part[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) part[w] = w < a.split ? from[w * a.T * kSumPitch] : 0.f;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part[w];
        float* sum = sums + ((b0 + b) * a.T + k) * kSumPitch + lane;
        *sum = sl > 0 ? *sum + v : v;
      }
      __syncthreads();
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // each CTA of the cluster has its share of the outputs, a warp 32 rows of one token
  if (a.ranks > 1)
    cluster_sync_all();
  else
    __syncthreads();
#pragma unroll 1
  for (int q = rank * kWarps + warp; q < blocks * a.T; q += a.ranks * kWarps) {
    float v = 0.f;
    if (a.ranks > 1) {
      const uint32_t at = smem_u32(sums + q * kSumPitch + lane);
      float part[kMostCluster];
#pragma unroll
      for (int c = 0; c < kMostCluster; ++c) {
        uint32_t from;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(min(c, a.ranks - 1)));
        part[c] = ld_cluster_f1(from);
      }
#pragma unroll
      for (int c = 0; c < kMostCluster; ++c) v += c < a.ranks ? part[c] : 0.f;
    } else {
      v = sums[q * kSumPitch + lane];
    }
    const int b = q / a.T, row = (block0 + b) * kRows + lane;
    if (row < a.N) a.y[(int64_t)(q - b * a.T) * a.N + row] = f32_to_bf16_bits(v);
  }
  if (a.ranks > 1) cluster_sync_all();  // until every CTA has read this one's sums
}

// n[i]: clusters of 2^i CTAs that the device holds at a time with two CTAs to an SM, asked
// once for a device; a question that fails is an error and is not kept.
template <int NB, bool kScales8>
cudaError_t clusters_at_once(int (&n)[4]) {
  constexpr int kDevices = 32;
  static std::atomic<int> known[kDevices][4];
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
    n[i] = device < kDevices ? known[device][i].load(std::memory_order_relaxed) : 0;
    if (n[i] > 0) continue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kMostCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kPerSm;
    cudaLaunchAttribute attr[2];
    set_adapter_attrs(&cfg, attr, 1 << i);
    e = cudaOccupancyMaxActiveClusters(&n[i], int4_matvec_kernel<NB, kScales8>, &cfg);
    if (e == cudaSuccess && device < kDevices)
      known[device][i].store(n[i], std::memory_order_relaxed);
  }
  return e;
}

// How the work is cut.  For each number of CTAs that share the columns (ranks) and of
// warps that share a CTA's (split), the time in steps of about 0.1 us: the steps that a
// warp goes through, one more a turn for the sums, two for every 16 bytes of x that a
// thread makes ready, and what a cluster costs to start and to join.  The fewest win.
// Measured, ranks and split: one row of 7168 x 7168, 1 and 8: 12.8 us, 4 and 2: 14.0; 3
// rows of 3585 x 2080, 1 and 8: 6.2, 4 and 4: 7.7; 16 rows of 16384 x 7168, 8 and 1: 32,
// 4 and 1: 38, 2 and 1: 46; 2 rows of 1160 x 13216, 4 and 8: 10.3, 2 and 8: 11.5.
template <int NB, bool kScales8>
int launch(MatvecArgs a, cudaStream_t st) {
  auto kern = int4_matvec_kernel<NB, kScales8>;
  MOE_TRY_CUDA(adapter_smem(reinterpret_cast<const void*>(kern)));
  const int joined[4] = {0, 5, 8, 12};
  int held[4];
  MOE_TRY_CUDA((clusters_at_once<NB, kScales8>(held)));
  const int steps = (a.K + 127) / 128, n_blocks = (a.N + kRows - 1) / kRows;
  MatvecArgs best = a;
  int64_t least = INT64_MAX;
  for (int i = 0; i < 4; ++i)
    for (int split = 1; split <= kWarps; split *= 2) {
      MatvecArgs b = a;
      b.ranks = 1 << i;
      b.split = split;
      const int abreast = kWarps / split, clusters = held[i];
      if (clusters < 1 || b.ranks > steps) continue;
      b.blocks = max(abreast, (n_blocks + clusters - 1) / clusters);
      const int waves = (b.blocks + kMostBlocks - 1) / kMostBlocks;
      b.blocks = max(abreast, (n_blocks + clusters * waves - 1) / (clusters * waves));
      // slices as few as fit, the same number in every CTA
      int per = 0;
      do {
        ++per;
        b.slice = (steps + per * b.ranks - 1) / (per * b.ranks) * 128;
        b.slices = (a.K + b.slice - 1) / b.slice;
      } while (Layout(b).total > kPerSm && b.slice > 128);
      if (b.slices < b.ranks) continue;
      const int turns = (b.blocks + abreast - 1) / abreast;
      const int each = (b.slice / 128 + split - 1) / split;
      const int64_t cost = static_cast<int64_t>(waves) *
          (static_cast<int64_t>(per) * (turns * (each + 1) + b.slice / 4 * a.T / kThreads) + joined[i]);
      if (cost >= least) continue;
      least = cost;
      best = b;
    }
  if (least == INT64_MAX) return MOE_ERR_CUDA;
  const Layout lay(best);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((n_blocks + best.blocks - 1) / best.blocks * best.ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = lay.total;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  set_adapter_attrs(&cfg, attr, best.ranks > 1 ? best.ranks : 0);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kern, best));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_int4_matvec(const uint16_t* x, int64_t x_ld, const int32_t* w_packed,
                               const uint16_t* w_scale, int T, int N, int K, uint16_t* y,
                               void* stream) {
  moe::Range range_("moe_int4_matvec");
  if (T < 0 || N <= 0 || K <= 0 || x_ld < K) return MOE_ERR_INVALID;
  if (T > kMaxTokens || K % kGroup != 0 || K > kMostColumns || N > kMostRows || x_ld % 8 != 0)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_packed || !w_scale || !y) return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(w_scale, 4) || !aligned(y, 2))
    return MOE_ERR_INVALID;
  // CTAs write y while others still read the inputs
  const size_t y_bytes = static_cast<size_t>(T) * N * 2, n = static_cast<size_t>(N) * K;
  if (overlap(x, (static_cast<size_t>(T - 1) * x_ld + K) * 2, y, y_bytes) ||
      overlap(w_packed, n / 2, y, y_bytes) || overlap(w_scale, n / 16, y, y_bytes))
    return MOE_ERR_INVALID;
  MatvecArgs a{};
  a.x = x;
  a.w = reinterpret_cast<const uint8_t*>(w_packed);
  a.scale = reinterpret_cast<const uint8_t*>(w_scale);
  a.y = y;
  a.x_ld = x_ld;
  a.T = T;
  a.N = N;
  a.K = K;
  // whether the scales of every 128 columns begin on 8 bytes
  const bool scales8 = K % 128 == 0 && aligned(w_scale, 8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T <= 8) return scales8 ? launch<1, true>(a, st) : launch<1, false>(a, st);
  return scales8 ? launch<2, true>(a, st) : launch<2, false>(a, st);
}
