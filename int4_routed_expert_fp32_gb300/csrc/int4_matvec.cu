// y = x W^T for packed int4 weights with a bf16 scale per 32 columns and at most 16 rows x.
//
// The weights are read once and bound the time from some MB on; below that it is
// latency: launch, one trip to HBM, one reduction.  So a CTA takes 16-row blocks of W,
// its eight warps split K (or, where K is short, the rows), and each warp copies its own
// weights three steps ahead (cp.async, 8 KB of them on their way), on from one
// block into the next.  What a warp copies it reads itself, so no warp waits for
// another before the sums are joined.
//
// The tokens are turned into fp16 in shared memory first, each scaled by a power of two
// (exact), in the order in which a packed word pairs its nibbles; the weights'
// first copies are under way meanwhile.  Where all of K does not fit, the CTA goes
// through K in slices and keeps its sums in shared memory.
//
// Products: m16n8k16 MMAs on the nibbles as fp16, 1032 + q and 72 + q, exactly; the
// accumulator starts from minus the constants' part (one value for a token and group),
// and each group's sum is scaled and added in fp32.  One ldmatrix gives a lane the
// words of two groups.
#include <cuda_fp16.h>

#include "adapter.cuh"
#include "common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kDepth = 3;              // steps of 128 columns a warp copies ahead
constexpr int kStepWords = 16 * 64;    // 16 rows of 4 groups
constexpr int kScalePitch = 12;        // 4 scales of a row, 4-byte pieces that hold them
constexpr int kStepBytes = kStepWords + 16 * kScalePitch + 64;  // a multiple of 128
constexpr int kMaxTokens = 16;
constexpr int kRoomForTokens = 60 * 1024;  // shared memory of a slice of x: two CTAs fit an SM

struct MatvecArgs {
  const uint16_t* x;
  const uint8_t* w;
  const uint8_t* scale;
  uint16_t* y;
  int64_t x_ld;
  int T, N, K;
  int slice;   // columns of a slice, a multiple of 128
  int split;   // warps that share a slice's columns
  int blocks;  // 16-row blocks of a CTA
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "l"(policy)
               : "memory");
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

// Where one warp's work on a block and slice lies.
struct Item {
  int row0;   // first row of the block (N or more: none)
  int step0;  // first step of 128 columns, in the slice
  int steps;
  int col0;   // first column of the slice
};

// Bytes of a token's row in shared memory: rows 64 bytes apart in the banks.
__host__ __device__ __forceinline__ int row_pitch(int slice) { return slice * 2 + 64; }

struct Layout {
  int start, steps, red, sums, total;
  __host__ __device__ __forceinline__ explicit Layout(const MatvecArgs& a) {
    const int padded = (a.T + 7) / 8 * 8;
    start = a.T * row_pitch(a.slice);                 // [slice / 32][padded] start values
    steps = start + a.slice / kGroup * padded * 4;    // the warps' steps
    red = steps + kWarps * kDepth * kStepBytes;       // [2][warp][16][padded]
    sums = red + 2 * kWarps * 16 * padded * 4;        // [blocks][16][padded]
    total = sums + (a.slice < a.K ? a.blocks * 16 * padded * 4 : 0);
  }
};

template <int NB>
__global__ void __launch_bounds__(kThreads, 2) int4_matvec_kernel(const MatvecArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t top[kMaxTokens];  // largest magnitude of a token in the slice
  const Layout lay(a);
  constexpr int kPad = NB * 8;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int ks = warp & (a.split - 1), rb = warp / a.split, abreast = kWarps / a.split;
  const int groups = a.K / kGroup;
  const int block0 = blockIdx.x * a.blocks;
  const int blocks = min(a.blocks, (a.N + 15) / 16 - block0);
  const int slices = (a.K + a.slice - 1) / a.slice;
  const int turns = (blocks + abreast - 1) / abreast;  // of a slice
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
    it.col0 = sl * a.slice;
    const int steps = (min(a.slice, a.K - it.col0) + 127) / 128;
    const int each = (steps + a.split - 1) / a.split;
    it.step0 = ks * each;
    it.steps = sl < slices && b < blocks ? max(0, min(each, steps - it.step0)) : 0;
    it.row0 = (block0 + b) * 16;
    return it;
  };
  uint8_t* mine = smem + lay.steps + warp * kDepth * kStepBytes;
  // Step j of an item: 16-byte pieces of rows swizzled by row / 2, and the scales.
  auto load = [&](int slot, const Item& it, int j) {
    const uint32_t to = smem_u32(mine) + slot * kStepBytes;
    const int col = it.col0 + (it.step0 + j) * 128;
    const int first = col / kGroup;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h, row = min(it.row0 + r, a.N - 1);
      if (first + t < groups)
        copy16(to + r * 64 + ((t ^ (r >> 1 & 3)) << 4),
               a.w + (int64_t)row * (a.K / 2) + col / 2 + t * 16, once);
    }
    // 8 bytes of scales of a row, which begin on 4 bytes or 2 behind them
#pragma unroll 1
    for (int p = lane; p < 48; p += 32) {
      const int r = p & 15, piece = p >> 4, row = min(it.row0 + r, a.N - 1);
      const int64_t at = ((int64_t)row * groups + first) * 2, word = (at & ~3LL) + 4 * piece;
      const int64_t end = min(at + 8, ((int64_t)row + 1) * groups * 2);  // of the row's scales
      uint8_t* dst = mine + slot * kStepBytes + kStepWords + r * kScalePitch + 4 * piece;
      if (word >= end) continue;
      if (word + 4 <= (int64_t)a.N * groups * 2)
        cp_async_4(dst, a.scale + word);
      else  // the last scale of an odd number
        *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(a.scale + word);
    }
  };

  grid_wait();  // x, or the weights, may come from the kernel before
  grid_launch_dependents();
  // the first copies of weights; x is made ready meanwhile
  Item cur = item_of(0);
  int slot = 0;
#pragma unroll 1
  for (int j = 0; j < kDepth; ++j) {
    if (j < cur.steps) load(j, cur, j);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  float* start = reinterpret_cast<float*>(smem + lay.start);
  const int pitch = row_pitch(a.slice);
#pragma unroll 1
  for (int turn = 0; turn < turns * slices; ++turn) {
    if (turn % turns == 0) {
      // x of this slice as fp16 in pair order
      const int cols = min(a.slice, a.K - cur.col0);
      __syncthreads();
      if (tid < kMaxTokens) top[tid] = 0u;
      __syncthreads();
      const int pieces = cols / 8;
#pragma unroll 1
      for (int k = 0; k < a.T; ++k) {
        uint32_t m = 0u;
#pragma unroll 1
        for (int c = tid; c < pieces; c += kThreads) {
          const uint4 v = __ldcg(reinterpret_cast<const uint4*>(a.x + k * a.x_ld + cur.col0 + 8 * c));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            m = max(m, w[i] << 16 & 0x7fff0000u);
            m = max(m, w[i] & 0x7fff0000u);
          }
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0 && m) atomicMax(&top[k], m);
      }
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < a.T; ++k) {
        // a power of two that brings the largest value to [2^14, 2^15), at most 2^126; 1 where
        // it is 0 or not finite
        const int field = static_cast<int>(top[k] >> 23);
        const int up = top[k] == 0u || field == 255 ? 127 : min(127 + 14 + 127 - field, 253);
        const float by = __uint_as_float(static_cast<uint32_t>(up) << 23);
#pragma unroll 1
        for (int c = tid; c < (pieces + 31) / 32 * 32; c += kThreads) {  // whole warps
          float s = 0.f;
          if (c < pieces) {
            const uint4 v =
                __ldcg(reinterpret_cast<const uint4*>(a.x + k * a.x_ld + cur.col0 + 8 * c));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            __half2 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // columns i and i + 4
              const uint32_t lo = (w[i >> 1] >> (16 * (i & 1))) << 16;
              const uint32_t hi = (w[2 + (i >> 1)] >> (16 * (i & 1))) << 16;
              p[i] = __floats2half2_rn(__uint_as_float(lo) * by, __uint_as_float(hi) * by);
              s = fmaf(i & 1 ? -72.f : -1032.f, __low2float(p[i]) + __high2float(p[i]), s);
            }
            *reinterpret_cast<uint4*>(smem + k * pitch + 16 * c) = *reinterpret_cast<const uint4*>(p);
          }
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          if (c < pieces && !(c & 3)) start[c / 4 * kPad + k] = s;
        }
      }
      __syncthreads();
    }
    const Item next = item_of(turn + 1);
    float acc[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    const int steps = max(kDepth, cur.steps);
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      __syncwarp();
      if (j < cur.steps) {
        const uint8_t* st = mine + slot * kStepBytes;
        const int step = cur.step0 + j, first = cur.col0 / kGroup + 4 * step;
        // the lane's row of an ldmatrix tile, and scales of rows g and g + 8
        const int r = (lane & 8) + (lane & 7);
        const int64_t at0 = (int64_t)min(cur.row0 + g, a.N - 1) * groups + first;
        const int64_t at8 = (int64_t)min(cur.row0 + g + 8, a.N - 1) * groups + first;
        const uint8_t* s0 = st + kStepWords + g * kScalePitch + (at0 & 1) * 2;
        const uint8_t* s8 = st + kStepWords + (g + 8) * kScalePitch + (at8 & 1) * 2;
#pragma unroll
        for (int pair = 0; pair < 2; ++pair) {
          if (first + 2 * pair >= groups) break;
          uint32_t wr[4];
          const uint32_t from = smem_u32(st) + r * 64 + (((2 * pair + (lane >> 4)) ^ (r >> 1 & 3)) << 4);
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                       : "=r"(wr[0]), "=r"(wr[1]), "=r"(wr[2]), "=r"(wr[3])
                       : "r"(from)
                       : "memory");
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int gr = 2 * pair + h;
            if (first + gr >= groups) break;
            uint32_t lo[4], hi[4];
            nibbles(wr[2 * h], magic_lo, magic_hi, lo);
            nibbles(wr[2 * h + 1], magic_lo, magic_hi, hi);
            const float f0 =
                __uint_as_float(*reinterpret_cast<const uint16_t*>(s0 + 2 * gr) << 16);
            const float f8 =
                __uint_as_float(*reinterpret_cast<const uint16_t*>(s8 + 2 * gr) << 16);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              // rows of tokens that are not there repeat the last one: no column of the
              // product reaches another
              const uint4 v = *reinterpret_cast<const uint4*>(
                  smem + min(8 * n + g, a.T - 1) * pitch + (4 * step + gr) * 64 + t * 16);
              const float2 c =
                  *reinterpret_cast<const float2*>(start + (4 * step + gr) * kPad + 8 * n + 2 * t);
              float d[4] = {c.x, c.y, c.x, c.y};
              mma_f16(d, lo[0], hi[0], lo[1], hi[1], v.x, v.y);
              mma_f16(d, lo[2], hi[2], lo[3], hi[3], v.z, v.w);
              acc[n][0] = fmaf(f0, d[0], acc[n][0]);
              acc[n][1] = fmaf(f0, d[1], acc[n][1]);
              acc[n][2] = fmaf(f8, d[2], acc[n][2]);
              acc[n][3] = fmaf(f8, d[3], acc[n][3]);
            }
          }
        }
      }
      __syncwarp();
      const int ahead = j + kDepth;
      if (ahead < cur.steps)
        load(slot, cur, ahead);
      else if (ahead >= steps && ahead - steps < next.steps)
        load(slot, next, ahead - steps);
      asm volatile("cp.async.commit_group;" ::: "memory");
      slot = slot + 1 == kDepth ? 0 : slot + 1;
    }
    float* red = reinterpret_cast<float*>(smem + lay.red) + (turn & 1) * kWarps * 16 * kPad;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float* p = red + (warp * 16 + g) * kPad + 8 * n + 2 * t;
      *reinterpret_cast<float2*>(p) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(p + 8 * kPad) = make_float2(acc[n][2], acc[n][3]);
    }
    __syncthreads();
    // one thread an output: warps of a block in order, then the slices in order
    const int sl = turn / turns, b0 = (turn - sl * turns) * abreast;
    float* sums = reinterpret_cast<float*>(smem + lay.sums);
#pragma unroll 1
    for (int i = tid; i < abreast * 16 * a.T; i += kThreads) {
      const int r = i & 15, k = (i >> 4) % a.T, b = (i >> 4) / a.T;
      if (b0 + b >= blocks) continue;
      float v = 0.f;
#pragma unroll 1
      for (int w = 0; w < a.split; ++w) v += red[((b * a.split + w) * 16 + r) * kPad + k];
      const int field = static_cast<int>(top[k] >> 23);
      const int up = top[k] == 0u || field == 255 ? 127 : min(127 + 14 + 127 - field, 253);
      v *= __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
      if (slices > 1) {
        float* sum = sums + ((b0 + b) * 16 + r) * kPad + k;
        if (sl > 0) v += *sum;
        *sum = v;
      }
      const int row = (block0 + b0 + b) * 16 + r;
      if (sl == slices - 1 && row < a.N) a.y[(int64_t)k * a.N + row] = f32_to_bf16_bits(v);
    }
    cur = next;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int NB>
int launch(MatvecArgs a, cudaStream_t st) {
  auto kern = int4_matvec_kernel<NB>;
  MOE_TRY_CUDA(adapter_smem(reinterpret_cast<const void*>(kern)));
  // as many columns as fit; at least 128
  const int padded = NB * 8;
  const int most = kRoomForTokens / (a.T * 2 + padded / 8) / 128 * 128;
  const int all = (a.K + 127) / 128 * 128;
  const int slices = (all + most - 1) / most;
  a.slice = ((all / 128 + slices - 1) / slices) * 128;
  // four steps a warp at least, else the warps have different rows
  const int steps = a.slice / 128;
  a.split = steps >= 32 ? 8 : steps >= 16 ? 4 : steps >= 8 ? 2 : 1;
  const int n_blocks = (a.N + 15) / 16;
  a.blocks = 1;
  int ctas = 1;
  const int want = Layout(a).total;
  MOE_TRY_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kern, kThreads, want));
  if (ctas < 1) return MOE_ERR_UNSUPPORTED;
  const int grid = ctas * num_sms();
  // whole rounds of the warps' blocks; with one slice a CTA's x costs little, and more CTAs
  // than fit at a time are no loss
  const int abreast = kWarps / a.split;
  a.blocks = (n_blocks + grid - 1) / grid;
  a.blocks = (a.blocks + abreast - 1) / abreast * abreast;
  if (a.blocks < abreast) a.blocks = abreast;
  if (a.blocks * abreast > 0 && n_blocks < abreast * num_sms()) a.blocks = abreast;
  const Layout lay(a);
  if (lay.total > 226 * 1024) return MOE_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((n_blocks + a.blocks - 1) / a.blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = lay.total;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  set_adapter_attrs(&cfg, attr, 0);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
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
  if (T > kMaxTokens || K % kGroup != 0 || x_ld % 8 != 0) return MOE_ERR_UNSUPPORTED;
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return T <= 8 ? launch<1>(a, st) : launch<2>(a, st);
}
