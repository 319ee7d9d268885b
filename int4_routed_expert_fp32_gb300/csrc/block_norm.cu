// The norms on both sides of a block's output, its gate and its residual, in
// one pass over the rows:
//   v  = y                    or  y / sqrt(mean y^2 + eps) * post_gain
//   v *= gate                 or  1 / (1 + exp(-gate))       (optional)
//   r  = x + scale * v        (x optional)
//   x_out = r rounded to x's type; h = r / sqrt(mean r^2 + eps) * pre_gain,
// h from the unrounded r ("Kimi K2.5 donor reference" page, RMSNorm mean
// square, normalisation and gain equations; the residual sums of its decoder
// layer).  All arithmetic and both sums of squares in fp32, one rounding per
// output.
//
// Bound: bytes.  Each element of y, x, gate, x_out and h crosses memory once:
// a row is held in registers (8 columns to a vector, VPT vectors to a thread)
// between the two reductions.  8 warps and more per row cost two block
// barriers each; rows of up to 1024 columns take one warp and none.
#include <math.h>

#include <algorithm>

#include "common.cuh"

namespace moe {

namespace {

enum Gate { kNoGate = 0, kGateFull = 1, kGateChannel = 2, kGateToken = 3 };

struct NormArgs {
  const uint16_t* y;
  const void* x;
  const uint16_t* post_gain;
  const uint16_t* gate;
  const uint16_t* pre_gain;
  void* x_out;
  uint16_t* h;
  int64_t y_ld, x_ld, gate_ld, x_out_ld, h_ld;
  int T, N, gate_mode, gate_sigmoid;
  float scale, eps;
};

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(f32_to_bf16_bits(f[2 * i])) |
           (static_cast<uint32_t>(f32_to_bf16_bits(f[2 * i + 1])) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// By the fast exponential and division: a relative error below 1e-6 for gates up to
// 8 in magnitude, where a bf16 output is rounded by up to 2^-8.  With expf and a
// rounded division 8192 x 7168 takes 111 us in place of 90 (fp32 stream 142 and 128).
__device__ __forceinline__ float gate_value(float g, int sigmoid) {
  return sigmoid ? __fdividef(1.f, 1.f + __expf(-g)) : g;
}

// Sum over the threads of a row: a warp (WARPS == 1), or the whole CTA, whose
// warps each add the partial sums in the same order.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (WARP) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

__device__ __forceinline__ float inv_rms(float ss, int N, float eps) {
  return 1.0f / sqrtf(ss / static_cast<float>(N) + eps);
}

// N % 8 == 0, every row 16-byte aligned.  WARP: a warp to a row, else a CTA.  Four
// CTAs of 256 threads to an SM: at 64 registers 8192 x 7168 with a gate runs in
// 92 us (6.4 TB/s), at 73 (three) in 102, at 48 (five, spilling) in 116.
template <bool XF32, bool WARP, int VPT, int THREADS = 256>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 4 : 1) block_norm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int step = WARP ? 32 : blockDim.x;
  const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                         : blockIdx.x;
  if (WARP && t >= a.T) return;
  const int nv = a.N >> 3;
  const uint4* yr = reinterpret_cast<const uint4*>(a.y + t * a.y_ld);
  const bool full = a.gate_mode == kGateFull;
  const uint4* gr = reinterpret_cast<const uint4*>(full ? a.gate + t * a.gate_ld : a.gate);
  // every load of the row in flight before the first use
  uint4 yv[VPT], xv[VPT * (XF32 ? 2 : 1)], gv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * step;
    if (v < nv) {
      yv[i] = yr[v];
      if (a.x) {
        if constexpr (XF32) {
          const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const float*>(a.x) + t * a.x_ld);
          xv[2 * i] = xr[2 * v];
          xv[2 * i + 1] = xr[2 * v + 1];
        } else {
          xv[i] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + t * a.x_ld)[v];
        }
      }
      if (full || a.gate_mode == kGateChannel) gv[i] = gr[v];
    }
  }
  float s = a.scale;
  if (a.gate_mode == kGateToken)
    s *= gate_value(bf16_bits_to_f32(a.gate[t * a.gate_ld]), a.gate_sigmoid);
  if (a.post_gain) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (tid + i * step < nv) {
        float f[8];
        unpack8(yv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
      }
    s *= inv_rms(row_sum<WARP>(ss, red[0]), a.N, a.eps);
  }
  float r[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * step;
    if (v < nv) {
      unpack8(yv[i], r[i]);
      if (a.post_gain) {
        float g[8];
        unpack8(reinterpret_cast<const uint4*>(a.post_gain)[v], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= g[j];
      }
      if (full || a.gate_mode == kGateChannel) {
        float g[8];
        unpack8(gv[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= gate_value(g[j], a.gate_sigmoid);
      }
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
      if (a.x) {
        if constexpr (XF32) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&xv[2 * i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
        } else {
          unpack8(xv[i], x);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i][j] = fmaf(r[i][j], s, x[j]);
        ss = fmaf(r[i][j], r[i][j], ss);
      }
      if (a.x_out) {
        if constexpr (XF32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.x_out) + t * a.x_out_ld) + 2 * v;
          o[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
          o[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
        } else {
          reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x_out) + t * a.x_out_ld)[v] = pack8(r[i]);
        }
      }
    }
  }
  if (!a.h) return;
  const float inv = inv_rms(row_sum<WARP>(ss, red[1]), a.N, a.eps);
  uint4* hr = reinterpret_cast<uint4*>(a.h + t * a.h_ld);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * step;
    if (v < nv) {
      float g[8];
      unpack8(reinterpret_cast<const uint4*>(a.pre_gain)[v], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= r[i][j] * inv;
      hr[v] = pack8(g);
    }
  }
}

// Eight consecutive bf16 of a row in shared memory, from element 8 v + s on (s < 8,
// the same for all threads): two 16-byte reads and a shift.
__device__ __forceinline__ uint4 shifted8(const uint4* p, int v, int s) {
  const uint4 a = p[v], b = p[v + 1];
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (s & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (s & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (s & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Widths that are no multiple of 8, dense rows (every row stride N, 16-byte
// aligned bases): row t begins t N mod 8 elements past a 16-byte boundary, in
// every tensor alike.  A thread takes vectors of 8 from the row's first boundary
// on, and threads 0 .. 14 also one of the up to 7 + 7 elements around them.  The
// gains and a channel's gate, whose columns do not move with the row, are held in
// shared memory and read with a shift; a CTA walks rows, so that they are loaded
// once.  8192 x 7001 with a gate: 155 us, 265 column by column (86 at the copy's
// rate): the shifts and single elements cost instructions, and at 64 registers the
// variants with two vectors a thread spill 36 to 108 bytes.
template <bool XF32, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? (VPT == 4 ? 2 : 4) : 1)
    block_norm_odd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint16_t gains[];  // post, pre, channel gate, each padded
  __shared__ float red[2][2][32];
  const int pitch = (a.N + 7) / 8 * 8 + 8;
  uint16_t* const post = gains;
  uint16_t* const pre = gains + pitch;
  uint16_t* const chan = gains + 2 * pitch;
  const bool full = a.gate_mode == kGateFull, channel = a.gate_mode == kGateChannel;
  for (int c = threadIdx.x; c < pitch; c += blockDim.x) {
    const bool in = c < a.N;
    if (a.post_gain) post[c] = in ? a.post_gain[c] : 0;
    if (a.h) pre[c] = in ? a.pre_gain[c] : 0;
    if (channel) chan[c] = in ? a.gate[c] : 0;
  }
  __syncthreads();
  const int tid = threadIdx.x, step = blockDim.x;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const int64_t base = t * a.N;
    const int head = min(static_cast<int>(-base & 7), a.N);  // elements before the boundary
    const int nv = (a.N - head) >> 3, tail = a.N - head - 8 * nv;
    const uint16_t* yr = a.y + base + head;
    const uint16_t* gr = full ? a.gate + base + head : nullptr;
    uint4 yv[VPT], xv[VPT * (XF32 ? 2 : 1)], gv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      if (v < nv) {
        yv[i] = reinterpret_cast<const uint4*>(yr)[v];
        if (a.x) {
          if constexpr (XF32) {
            const uint4* xr =
                reinterpret_cast<const uint4*>(static_cast<const float*>(a.x) + base + head);
            xv[2 * i] = xr[2 * v];
            xv[2 * i + 1] = xr[2 * v + 1];
          } else {
            xv[i] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + base + head)[v];
          }
        }
        if (full) gv[i] = reinterpret_cast<const uint4*>(gr)[v];
      }
    }
    // this thread's element around the vectors
    const int col = tid < head ? tid : tid >= 8 && tid - 8 < tail ? head + 8 * nv + tid - 8 : -1;
    float ye = 0.f, xe = 0.f, ge = 1.f;
    if (col >= 0) {
      ye = bf16_bits_to_f32(a.y[base + col]);
      if (a.x)
        xe = XF32 ? static_cast<const float*>(a.x)[base + col]
                  : bf16_bits_to_f32(static_cast<const uint16_t*>(a.x)[base + col]);
      if (full) ge = gate_value(bf16_bits_to_f32(a.gate[base + col]), a.gate_sigmoid);
      if (channel) ge = gate_value(bf16_bits_to_f32(chan[col]), a.gate_sigmoid);
      if (a.post_gain) ge *= bf16_bits_to_f32(post[col]);
    }
    float s = a.scale;
    if (a.gate_mode == kGateToken)
      s *= gate_value(bf16_bits_to_f32(a.gate[t * a.gate_ld]), a.gate_sigmoid);
    if (a.post_gain) {
      float ss = ye * ye;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (tid + i * step < nv) {
          float f[8];
          unpack8(yv[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
        }
      s *= inv_rms(row_sum<false>(ss, red[turn][0]), a.N, a.eps);
    }
    const float re = fmaf(ye * ge, s, xe);
    float ss = col >= 0 ? re * re : 0.f;
    float r[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      if (v < nv) {
        unpack8(yv[i], r[i]);
        float g[8];
        if (a.post_gain) {
          unpack8(shifted8(reinterpret_cast<const uint4*>(post), v, head), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] *= g[j];
        }
        if (full || channel) {
          unpack8(full ? gv[i] : shifted8(reinterpret_cast<const uint4*>(chan), v, head), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] *= gate_value(g[j], a.gate_sigmoid);
        }
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
        if (a.x) {
          if constexpr (XF32) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&xv[2 * i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
          } else {
            unpack8(xv[i], x);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[i][j] = fmaf(r[i][j], s, x[j]);
          ss = fmaf(r[i][j], r[i][j], ss);
        }
        if (a.x_out) {
          if constexpr (XF32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.x_out) + base + head) + 2 * v;
            o[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
            o[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
          } else {
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x_out) + base + head)[v] = pack8(r[i]);
          }
        }
      }
    }
    if (col >= 0 && a.x_out) {
      if (XF32)
        static_cast<float*>(a.x_out)[base + col] = re;
      else
        static_cast<uint16_t*>(a.x_out)[base + col] = f32_to_bf16_bits(re);
    }
    if (!a.h) {
      if (a.post_gain) __syncthreads();  // red is written again two rows on
      continue;
    }
    const float inv = inv_rms(row_sum<false>(ss, red[turn][1]), a.N, a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      if (v < nv) {
        float g[8];
        unpack8(shifted8(reinterpret_cast<const uint4*>(pre), v, head), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= r[i][j] * inv;
        reinterpret_cast<uint4*>(a.h + base + head)[v] = pack8(g);
      }
    }
    if (col >= 0) a.h[base + col] = f32_to_bf16_bits(re * inv * bf16_bits_to_f32(pre[col]));
  }
}

// Any width, stride and alignment: a CTA to a row, column by column, the row
// r in shared memory between its two uses.
template <bool XF32>
__global__ void __launch_bounds__(512) block_norm_any_kernel(const NormArgs a) {
  extern __shared__ float rrow[];
  __shared__ float red[2][32];
  const int64_t t = blockIdx.x;
  const uint16_t* yr = a.y + t * a.y_ld;
  float s = a.scale;
  if (a.gate_mode == kGateToken)
    s *= gate_value(bf16_bits_to_f32(a.gate[t * a.gate_ld]), a.gate_sigmoid);
  const uint16_t* gr = a.gate_mode == kGateFull ? a.gate + t * a.gate_ld
                       : a.gate_mode == kGateChannel ? a.gate : nullptr;
  if (a.post_gain) {
    float ss = 0.f;
    for (int c = threadIdx.x; c < a.N; c += blockDim.x) {
      const float f = bf16_bits_to_f32(yr[c]);
      ss = fmaf(f, f, ss);
    }
    s *= inv_rms(row_sum<false>(ss, red[0]), a.N, a.eps);
  }
  float ss = 0.f;
  for (int c = threadIdx.x; c < a.N; c += blockDim.x) {
    float f = bf16_bits_to_f32(yr[c]);
    if (a.post_gain) f *= bf16_bits_to_f32(a.post_gain[c]);
    if (gr) f *= gate_value(bf16_bits_to_f32(gr[c]), a.gate_sigmoid);
    float x = 0.f;
    if (a.x)
      x = XF32 ? static_cast<const float*>(a.x)[t * a.x_ld + c]
               : bf16_bits_to_f32(static_cast<const uint16_t*>(a.x)[t * a.x_ld + c]);
    f = fmaf(f, s, x);
    ss = fmaf(f, f, ss);
    rrow[c] = f;  // read back by the same thread only
    if (a.x_out) {
      if (XF32)
        static_cast<float*>(a.x_out)[t * a.x_out_ld + c] = f;
      else
        static_cast<uint16_t*>(a.x_out)[t * a.x_out_ld + c] = f32_to_bf16_bits(f);
    }
  }
  if (!a.h) return;
  const float inv = inv_rms(row_sum<false>(ss, red[1]), a.N, a.eps);
  for (int c = threadIdx.x; c < a.N; c += blockDim.x)
    a.h[t * a.h_ld + c] = f32_to_bf16_bits(rrow[c] * inv * bf16_bits_to_f32(a.pre_gain[c]));
}

constexpr int kMaxNormWidth = 32768;

template <bool XF32, int VPT, int THREADS>
int launch_odd(const NormArgs& a, int threads, cudaStream_t s) {
  auto kern = block_norm_odd_kernel<XF32, VPT, THREADS>;
  const int smem = 3 * ((a.N + 7) / 8 * 8 + 8) * 2;
  if (smem > 48 * 1024)
    MOE_TRY_CUDA(allow_most_smem(reinterpret_cast<const void*>(kern)));
  int fit = 1;
  MOE_TRY_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, threads, smem));
  kern<<<std::min(a.T, std::max(1, fit) * num_sms()), threads, smem, s>>>(a);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <bool XF32>
int launch_norm(const NormArgs& a, bool vec, bool dense, cudaStream_t s) {
  if (!vec && dense && a.N >= 64 && a.N <= 16384) {
    const int nv = a.N / 8;
    if (nv <= 256) return launch_odd<XF32, 1, 256>(a, (nv + 31) / 32 * 32, s);
    if (nv <= 512) return launch_odd<XF32, 2, 256>(a, ((nv + 1) / 2 + 31) / 32 * 32, s);
    if (nv <= 1024) return launch_odd<XF32, 4, 256>(a, ((nv + 3) / 4 + 31) / 32 * 32, s);
    return launch_odd<XF32, 2, 1024>(a, ((nv + 1) / 2 + 31) / 32 * 32, s);
  }
  if (!vec) {
    const size_t smem = static_cast<size_t>(a.N) * sizeof(float);
    auto kern = block_norm_any_kernel<XF32>;
    if (smem > 48 * 1024)
      MOE_TRY_CUDA(allow_most_smem(reinterpret_cast<const void*>(kern)));
    const int threads = std::min(512, (a.N + 31) / 32 * 32);
    kern<<<a.T, threads, smem, s>>>(a);
    MOE_LAUNCH_CHECK();
    return MOE_OK;
  }
  const int nv = a.N / 8;
  if (nv <= 128) {
    const int warps = 8;
    const unsigned grid = (a.T + warps - 1) / warps;
    if (nv <= 32)
      block_norm_kernel<XF32, true, 1><<<grid, 32 * warps, 0, s>>>(a);
    else if (nv <= 64)
      block_norm_kernel<XF32, true, 2><<<grid, 32 * warps, 0, s>>>(a);
    else
      block_norm_kernel<XF32, true, 4><<<grid, 32 * warps, 0, s>>>(a);
  } else {
    // Few rows: as many threads as vectors (latency).  Many: about 224 threads
    // with more loads each in flight, which leaves more rows to an SM (8192 x
    // 7168 with a gate: 4 vectors 91 us, 2 114, 1 117).  A vector of an fp32
    // stream is half as many again, and four of them spill: two at most (8192 x
    // 7168 with a gate: 4 vectors 142 us, 2 128, 1 205; 2049 x 3584: 4 20.5, 2
    // 15.4, 1 18.2; 8192 x 2048: 1 34.5; 305 x 7168: 4 7.8, 2 7.4).
    const int wide = XF32 ? 2 : 4;
    const int want = a.T <= 2 * num_sms() ? 1 : nv >= 768 ? wide : nv >= 384 ? 2 : 1;
    const int vpt = std::max(want, nv > 2048 ? 4 : nv > 1024 ? 2 : 1);
    const int threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
    if (vpt == 1 && threads <= 256)
      block_norm_kernel<XF32, false, 1><<<a.T, threads, 0, s>>>(a);
    else if (vpt == 1)
      block_norm_kernel<XF32, false, 1, 1024><<<a.T, threads, 0, s>>>(a);
    else if (vpt == 2 && threads <= 256)
      block_norm_kernel<XF32, false, 2><<<a.T, threads, 0, s>>>(a);
    else if (vpt == 2)
      block_norm_kernel<XF32, false, 2, 1024><<<a.T, threads, 0, s>>>(a);
    else if (XF32 || threads > 256)
      block_norm_kernel<XF32, false, 4, 1024><<<a.T, threads, 0, s>>>(a);
    else if constexpr (!XF32)
      block_norm_kernel<false, false, 4><<<a.T, threads, 0, s>>>(a);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_block_norm(const moe_block_norm_args* p, void* stream) {
  moe::Range range_("moe_block_norm");
  if (!p) return MOE_ERR_INVALID;
  if (p->T < 0 || p->N <= 0 || !(p->eps >= 0.f)) return MOE_ERR_INVALID;
  if (!(p->scale == p->scale) || isinf(p->scale) || isinf(p->eps)) return MOE_ERR_INVALID;
  if (p->gate_mode < MOE_GATE_NONE || p->gate_mode > MOE_GATE_TOKEN) return MOE_ERR_INVALID;
  if (p->N > kMaxNormWidth) return MOE_ERR_UNSUPPORTED;
  if (p->T == 0) return MOE_OK;
  const bool gate = p->gate_mode != MOE_GATE_NONE;
  if (!p->y || (!p->x_out && !p->h) || (gate && !p->gate)) return MOE_ERR_INVALID;
  if ((p->h != nullptr) != (p->pre_gain != nullptr)) return MOE_ERR_INVALID;
  const int64_t gate_cols = p->gate_mode == MOE_GATE_FULL ? p->N : 1;
  const bool gate_rows = p->gate_mode == MOE_GATE_FULL || p->gate_mode == MOE_GATE_TOKEN;
  if (p->y_ld < p->N || (p->x && p->x_ld < p->N) || (p->x_out && p->x_out_ld < p->N) ||
      (p->h && p->h_ld < p->N) || (gate_rows && p->gate_ld < gate_cols))
    return MOE_ERR_INVALID;
  const size_t item = p->x_f32 ? 4 : 2;
  if (!aligned(p->y, 2) || !aligned(p->x, item) || !aligned(p->x_out, item) || !aligned(p->h, 2) ||
      !aligned(p->post_gain, 2) || !aligned(p->pre_gain, 2) || !aligned(p->gate, 2))
    return MOE_ERR_INVALID;
  NormArgs a{};
  a.y = p->y;
  a.x = p->x;
  a.post_gain = p->post_gain;
  a.gate = gate ? p->gate : nullptr;
  a.pre_gain = p->pre_gain;
  a.x_out = p->x_out;
  a.h = p->h;
  a.y_ld = p->y_ld;
  a.x_ld = p->x_ld;
  a.gate_ld = p->gate_ld;
  a.x_out_ld = p->x_out_ld;
  a.h_ld = p->h_ld;
  a.T = p->T;
  a.N = p->N;
  a.gate_mode = p->gate_mode;
  a.gate_sigmoid = p->gate_sigmoid;
  a.scale = p->scale;
  a.eps = p->eps;
  // 16-byte vectors: widths and row strides of whole vectors, aligned bases
  auto rows16 = [](const void* q, int64_t ld, size_t b) {
    return !q || (aligned(q, 16) && ld * static_cast<int64_t>(b) % 16 == 0);
  };
  const bool vec = p->N % 8 == 0 && rows16(p->y, p->y_ld, 2) && rows16(p->x, p->x_ld, item) &&
                   rows16(p->x_out, p->x_out_ld, item) && rows16(p->h, p->h_ld, 2) &&
                   aligned(p->post_gain, 16) && aligned(p->pre_gain, 16) &&
                   (p->gate_mode != MOE_GATE_FULL || rows16(p->gate, p->gate_ld, 2)) &&
                   (p->gate_mode != MOE_GATE_CHANNEL || aligned(p->gate, 16));
  // rows that follow one another in every tensor, from 16-byte boundaries
  auto dense16 = [&](const void* q, int64_t ld) { return !q || (aligned(q, 16) && ld == p->N); };
  const bool dense = dense16(p->y, p->y_ld) && dense16(p->x, p->x_ld) &&
                     dense16(p->x_out, p->x_out_ld) && dense16(p->h, p->h_ld) &&
                     (p->gate_mode != MOE_GATE_FULL || dense16(p->gate, p->gate_ld));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p->x_f32 ? launch_norm<true>(a, vec, dense, s) : launch_norm<false>(a, vec, dense, s);
}
