// Routing from logits: scores, balance bias, groups, top-k, weights.
//
//   s_e = 1 / (1 + exp(-z_e))              or  exp(z_e - max z) / sum exp(z - max z)
//   c_e = s_e + b_e                        (no bias: the order of the z_e)
//   group score = max c  or  sum of the two largest c of the group
//   the topk_groups best groups stay; of their experts the k largest c, in
//   descending order (equal: lower id first); w = s / (sum s + 1e-20) * scale.
//
// One warp to a token, its E logits in registers.  A group is a run of L
// lanes and a lane a run of c consecutive experts of it, so that the two
// largest of every group come from one segmented shuffle tree and the order
// of the lanes is the order of the ids.
//
// Selection.  The k-th largest of the 32 lane maxima is a lower bound of the
// k-th largest key: only experts at or above it can be selected.  They are
// compacted (about k + 2 of 384 for logits of a router), one to a lane, and
// ranked against one another through shared memory, in place of k warp-wide
// argmax rounds over all registers.  Where more than 32 are left (few lanes hold
// the kept groups, k near 32) the range of keys is halved first.
//
// Rounding.  A key c = s + b in fp32 carries an error of some 1e-7, and two
// experts are as near as that in about one token of a hundred.  The decisions
// are those of 64-bit scores all the same: candidates within the slack of the
// bound are kept, and where two that matter lie within the error of one
// another the keys of the (few) candidates are evaluated again: sigmoid keys
// as pairs of fp32 values (fine_key), what those leave open in 64 bits.
// Without a bias the order of the scores is the order of the logits and no
// rounding decides anything.  Unavailable experts (z or c -inf or NaN) rank
// below all others, with weight 0; experts outside the kept groups are never
// chosen.
//
// Bound: instructions and the length of a token's chain of warp-wide steps, not
// bytes.  T = 8192, E = 384, 8 groups of which 4 stay, k = 8: 11.4 us for 12.7 MB
// (1.9 us at the HBM rate; 11 to 12 on one GPU or another); loads and keys alone are
// 4.9 of them, the groups 3.3.
// A warp holds a token because the registers then hold all keys: 32 warps fit an
// SM, and two rounds of them make the call.  At four CTAs of 8 warps to an SM (64
// registers) this variant stores 24 bytes a thread and loads 8 back; five spill more
// (12.7 us against 12.3 when measured), three are too few (13.1).  Softmax with a bias
// stores 96 and loads 304 there: 8192 x 384 in 8 groups 22 us.  A row with fewer
// than k experts left has all the others as candidates: 94 us where every row has 6.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "combine.cuh"
#include "common.cuh"
#include "route_select.cuh"

namespace moe {

namespace {

struct SelectArgs {
  const void* z;
  size_t ld, sp;
  int S;
  const float* bias;
  int T, E, k, G, tg, gs;  // gs: experts to a group
  int L, c;                // lanes to a group, experts to a lane
  int inv_L;               // ceil(2^16 / L): lane / L by a product, exact for lane < 32
  int best_only, renorm;   // group score: the best key only
  int vec, vec_bias;       // 4 logits, and biases, a load
  int full;                // every lane has c experts, and registers for no more
  float scale;
  int32_t* idx;
  float* w;
};

constexpr int kListBytes = 10;           // shared memory per expert: a 64-bit key and a 16-bit id
constexpr uint32_t kAbsent = 0;          // not a candidate: outside the kept groups
constexpr uint32_t kUnavail = 0x007fffffu;  // order_key(-inf)

// Unsigned order of floats (no NaN): a < b <=> order_key(a) < order_key(b),
// but for -0 < +0, which the callers remove.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t o) {
  return __uint_as_float(o ^ (static_cast<uint32_t>(~(static_cast<int32_t>(o) >> 31)) | 0x80000000u));
}

// e^x and 1 / y of the fast keys, whose values below fp32's normal range are 0.
__device__ __forceinline__ float fast_exp(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.44269504f));
  return e;
}

__device__ __forceinline__ float fast_rcp(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

__device__ __forceinline__ float clean(float z) {  // NaN -> -inf, -0 -> +0
  return fmaxf(z, -INFINITY) + 0.0f;
}

template <typename ZT>
__device__ __forceinline__ float logit(const SelectArgs& a, const ZT* row, int e) {
  if constexpr (sizeof(ZT) == 2) {
    return clean(bf16_bits_to_f32(row[e]));
  } else {
    float z = row[e];
    for (int p = 1; p < a.S; ++p) z += row[p * a.sp + e];
    return clean(z);
  }
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 64-bit score of one logit; m and sum: the softmax maximum and denominator.
template <bool SOFTMAX>
__device__ __forceinline__ double score64(float z, float m, double sum) {
  if (z == -INFINITY) return 0.0;
  if constexpr (SOFTMAX) {
    const double d = z == m ? 0.0 : static_cast<double>(z) - static_cast<double>(m);
    return exp(d) / sum;
  } else {
    return 1.0 / (1.0 + exp(-static_cast<double>(z)));
  }
}

__device__ __forceinline__ double key64(double s, float z, float b) {
  const double c = s + static_cast<double>(b);
  return (z == -INFINITY || c != c) ? static_cast<double>(-INFINITY) : c;
}

// exp(a - b), a <= b: of the rounded difference, corrected by what the
// rounding lost (up to 2^-24 |a - b| of the value).  Equal infinities: 1.
__device__ __forceinline__ float exp_diff(float a, float b) {
  if (a == b) return 1.f;
  const float d = a - b, back = d - a;
  if (d == -INFINITY) return 0.f;
  const float lost = (a - (d - back)) - (b + back);
  const float e = expf(d);
  return fmaf(e, lost, e);
}

// a + b = hi + lo, hi rounded to nearest (Knuth's exact sum of two floats).
__device__ __forceinline__ float two_sum(float a, float b, float& lo) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  lo = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return s;
}

// The key 1 / (1 + e^-z) + b as hi + lo within 1e-9: e^-|z| = 2^n e^r with the
// linear and quadratic terms of e^r as pairs and those above (at most 0.008) in
// fp32.  hi is the rounded sum, so that (hi, lo) compare in this order.
__device__ __forceinline__ float fine_key(float z, float b, float& low) {
  const float x = fmaxf(-fabsf(z), -80.f);
  const float n = rintf(x * 1.44269504f);
  // ln 2 = 11357 / 2^14 + c: the first product and difference are exact
  float r0, e0, t0, d0;
  const float r = two_sum(fmaf(-n, 0.69317626953125f, x), n * 2.90889713e-05f, r0);
  const float q = r * r, q0 = fmaf(r, r, -q);
  float tail = fmaf(r, 1.f / 40320.f, 1.f / 5040.f);
  tail = fmaf(r, tail, 1.f / 720.f);
  tail = fmaf(r, tail, 1.f / 120.f);
  tail = fmaf(r, tail, 1.f / 24.f);
  tail = r * q * fmaf(r, tail, 1.f / 6.f);
  const float t = two_sum(two_sum(1.f, r, e0), 0.5f * q, t0);
  t0 = (e0 + t0) + fmaf(r0, 1.f + r, 0.5f * q0) + tail;
  const float scale = exp2f(n);
  const float e = scale * two_sum(t, t0, e0);
  e0 *= scale;
  // 1 / (1 + e), or e / (1 + e) for z < 0
  const float d = two_sum(1.f, e, d0);
  d0 += e0;
  const float inv = fast_rcp(d);
  const float num = z < 0.f ? e : 1.f, num0 = z < 0.f ? e0 : 0.f;
  const float s = num * inv;
  const float s0 = inv * (fmaf(-s, d, num) + fmaf(-s, d0, num0));
  const float c = two_sum(s, b, low);
  if (!(fabsf(c) < INFINITY)) {
    low = 0.f;
    return c;
  }
  return two_sum(c, low + s0, low);
}

// Softmax denominator in 64 bits (warp-wide, rare).
template <typename ZT>
__device__ __noinline__ double softmax_sum64(const SelectArgs& a, const ZT* row, float m) {
  double sum = 0.0;
  for (int e = threadIdx.x & 31; e < a.E; e += 32) {
    const float z = logit(a, row, e);
    if (z == -INFINITY) continue;
    sum += z == m ? 1.0 : exp(static_cast<double>(z) - static_cast<double>(m));
  }
  return warp_sum64(sum);
}

// The same from fp32 exponentials, within a relative 5e-7 (2 steps each, and 2^-24
// |z - m| e^-|z - m| of the rounded differences).
template <typename ZT>
__device__ __noinline__ double softmax_sum_near(const SelectArgs& a, const ZT* row, float m) {
  double sum = 0.0;
  for (int e = threadIdx.x & 31; e < a.E; e += 32) {
    const float z = logit(a, row, e);
    if (z > -INFINITY) sum += z == m ? 1.f : expf(z - m);
  }
  return warp_sum64(sum);
}

// How far a difference of two biased softmax scores p + b can be off when both
// p share a denominator within 5e-7: an error of the difference of the p only.
__device__ __forceinline__ double shared_error(double p, double q) {
  return 2e-6 * fabs(p - q) + 1e-14;
}

// The segment leader's two largest of its L lanes' (hi >= lo) pairs.
template <typename F>
__device__ __forceinline__ void top2_segment(F& hi, F& lo, int r, int L) {
#pragma unroll 1
  for (int o = 1; o < L; o <<= 1) {
    const F oh = __shfl_down_sync(0xffffffffu, hi, o);
    const F ol = __shfl_down_sync(0xffffffffu, lo, o);
    if ((r & (2 * o - 1)) == 0 && r + o < L) {
      lo = hi > oh ? (lo > oh ? lo : oh) : (hi > ol ? hi : ol);
      hi = hi > oh ? hi : oh;
    }
  }
}

// Rank of group g among the G scores held by the segment leaders.
template <typename F>
__device__ __forceinline__ int group_rank(F score, int g, int G, int L) {
  const F mine = __shfl_sync(0xffffffffu, score, min(g, G - 1) * L);
  int rank = 0;
  for (int j = 0; j < G; ++j) {
    const F o = __shfl_sync(0xffffffffu, score, j * L);
    rank += (o > mine || (o == mine && j < g)) ? 1 : 0;
  }
  return rank;
}

// Whether this lane's group g is kept, from 64-bit scores of the n <= 32 listed
// experts, which hold the two best of every group (rare: the boundary between
// kept and dropped groups lies within the fp32 error).
template <typename ZT, bool SOFTMAX, bool BIAS>
__device__ __noinline__ bool group_kept64(const SelectArgs& a, const ZT* row, float m, int g,
                                          const uint16_t* cid, int n) {
  const int lane = threadIdx.x & 31;
  const double none = -INFINITY;
  float z = -INFINITY, b = 0.f;
  double e = 0.0;
  int of = -1;
  if (lane < n) {
    z = logit(a, row, cid[lane]);
    if constexpr (BIAS) b = a.bias[cid[lane]];
    of = cid[lane] / a.gs;
    e = score64<SOFTMAX>(z, m, 1.0);
  }
  __syncwarp();
  bool kept = false;
  for (int exact = SOFTMAX && BIAS ? 0 : 1; exact < 2; ++exact) {
    double sum = 1.0;
    if constexpr (SOFTMAX && BIAS)
      sum = exact ? softmax_sum64(a, row, m) : softmax_sum_near(a, row, m);
    const double p = e / sum;
    double key = z == -INFINITY ? none : p;
    if constexpr (BIAS) key = key64(p, z, b);
    if (lane >= n) key = none;
    double hi = none, lo = none, ph = 0.0, pl = 0.0;
    for (int j = 0; j < n; ++j) {
      const double v = __shfl_sync(0xffffffffu, key, j), pv = __shfl_sync(0xffffffffu, p, j);
      if (__shfl_sync(0xffffffffu, of, j) != g) continue;
      if (v > hi) {
        lo = hi;
        pl = ph;
        hi = v;
        ph = pv;
      } else if (v > lo) {
        lo = v;
        pl = pv;
      }
    }
    __syncwarp();
    double score = hi, part = ph;
    if (!a.best_only && hi > none && lo > none) {
      score = hi + lo;
      part = ph + pl;
    }
    kept = group_rank(score, g, a.G, a.L) < a.tg;
    if (exact) break;
    // decided, unless a kept and a dropped group are within what the sum leaves open
    bool open = false;
    for (int j = 0; j < a.G; ++j) {
      const double o = __shfl_sync(0xffffffffu, score, j * a.L);
      const double q = __shfl_sync(0xffffffffu, part, j * a.L);
      const bool other = __shfl_sync(0xffffffffu, kept, j * a.L);
      open |= g < a.G && other != kept && fabs(o - score) <= shared_error(q, part);
    }
    if (!__any_sync(0xffffffffu, open)) break;
  }
  return kept;
}

// The same from all experts (more than 32 listed: many keys within the error
// of one another).
template <typename ZT, bool SOFTMAX, bool BIAS>
__device__ __noinline__ bool group_kept64_all(const SelectArgs& a, const ZT* row, float m, int g,
                                              int r, int base, int cnt) {
  const double none = -INFINITY;
  double hi = none, lo = none;
  double sum = 1.0;
  if constexpr (SOFTMAX && BIAS) sum = softmax_sum64(a, row, m);
  for (int i = 0; i < cnt; ++i) {
    const float z = logit(a, row, base + i);
    if (z == -INFINITY) continue;
    double v = score64<SOFTMAX>(z, m, sum);
    if constexpr (BIAS) v = key64(v, z, a.bias[base + i]);
    if (v > hi) {
      lo = hi;
      hi = v;
    } else if (v > lo) {
      lo = v;
    }
  }
  __syncwarp();
  top2_segment(hi, lo, r, a.L);
  double score = hi;
  if (!a.best_only && hi > none && lo > none) score = hi + lo;
  return group_rank(score, g, a.G, a.L) < a.tg;
}

// Ranks of the n <= 32 candidates (one to a lane, in id order) by their 64-bit
// keys (rare: two that matter lie within the fp32 error of one another).
template <typename ZT, bool SOFTMAX>
__device__ __noinline__ int rank64(const SelectArgs& a, const ZT* row, float m, int id, int n,
                                   double* ckey) {
  const int lane = threadIdx.x & 31;
  float z = -INFINITY, b = 0.f;
  double e = 0.0;  // sigmoid score, or softmax numerator
  if (lane < n) {
    z = logit(a, row, id);
    b = a.bias[id];
    e = score64<SOFTMAX>(z, m, 1.0);
  }
  __syncwarp();
  int rank = 0;
  for (int exact = SOFTMAX ? 0 : 1; exact < 2; ++exact) {
    double sum = 1.0;
    if constexpr (SOFTMAX) sum = exact ? softmax_sum64(a, row, m) : softmax_sum_near(a, row, m);
    const double key = lane < n ? key64(e / sum, z, b) : -INFINITY;
    rank = 0;
    for (int j = 0; j < n; ++j) {
      const double other = __shfl_sync(0xffffffffu, key, j);
      rank += (other > key || (other == key && j < lane)) ? 1 : 0;
    }
    if (exact) break;
    // decided, unless neighbours in the order are within what the sum leaves open
    __syncwarp();
    if (lane < n) ckey[rank] = key;
    __syncwarp();
    const double gap = lane < n && rank > 0 ? ckey[rank - 1] - key : INFINITY;
    __syncwarp();
    if (lane < n) ckey[rank] = e / sum;
    __syncwarp();
    const bool open = lane < n && rank > 0 && rank <= a.k &&
                      gap <= shared_error(ckey[rank - 1], e / sum);
    if (!__any_sync(0xffffffffu, open)) break;
  }
  return lane < n ? rank : 32;
}

// The k best of n > 32 candidates (few lanes hold the kept groups, k near 32, or
// equal keys): 64-bit keys in shared memory, k rounds of the largest.  Lane q
// returns the id of rank q (-1: q >= k).
template <typename ZT, bool SOFTMAX, bool BIAS>
__device__ __noinline__ int select_many(const SelectArgs& a, const ZT* row, float m, double* ckey,
                                        uint16_t* cid, int n) {
  const int lane = threadIdx.x & 31;
  double sum = 1.0;
  if constexpr (SOFTMAX && BIAS) sum = softmax_sum64(a, row, m);
  for (int j = lane; j < n; j += 32) {
    const int e = cid[j];
    const float z = logit(a, row, e);
    double v = z;
    if constexpr (BIAS) v = key64(score64<SOFTMAX>(z, m, sum), z, a.bias[e]);
    ckey[j] = v;
  }
  __syncwarp();
  int id = -1;
  for (int q = 0; q < a.k; ++q) {
    double best = -INFINITY;
    int at = n;  // position = id order
    for (int j = lane; j < n; j += 32) {
      if (cid[j] & 0x8000u) continue;
      if (at == n || ckey[j] > best) {
        best = ckey[j];
        at = j;
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, d);
      const int oa = __shfl_xor_sync(0xffffffffu, at, d);
      if (oa < n && (at == n || ob > best || (ob == best && oa < at))) {
        best = ob;
        at = oa;
      }
    }
    if (lane == q) id = cid[at];
    __syncwarp();
    if (lane == q) cid[at] |= 0x8000u;
    __syncwarp();
  }
  return id;
}

// The weight (before the scale) of the lane's selected logit zz (-inf: none)
// where scores below fp32's range are among them:
// s = u exp(ref) / sum with u = exp(z' - ref), z' = z (softmax) or min(z, 0)
// over 1 + exp(-|z|) (sigmoid).  Renormalised, ref is the largest z' selected
// and exp(ref) cancels but for the stabiliser, so that their ratios are kept.
template <bool SOFTMAX>
__device__ __noinline__ float weight_far(const SelectArgs& a, float zz, float m, float sum) {
  const float zp = SOFTMAX ? zz : fminf(zz, 0.f);
  const float top = SOFTMAX ? m : 0.f;  // s = exp(z' - top) / sum
  const float ref = a.renorm ? fmaxf(warp_max(zp), -FLT_MAX) : top;
  float w = zz == -INFINITY ? 0.f : exp_diff(zp, ref);
  if constexpr (SOFTMAX) {
    if (!a.renorm) w /= sum;
  } else {
    w /= 1.0f + expf(-fabsf(zz));
  }
  if (a.renorm) {
    const float den = warp_sum(w);
    const float far = top - ref;
    if (far > 40.f) {  // the stabiliser weighs in
      const double stab = 1e-20 * sum * exp(static_cast<double>(top) - static_cast<double>(ref));
      w = static_cast<float>(w / (den + stab));
    } else {
      w = __fdiv_rn(w, den + 1e-20f * (far > 0.f ? sum * expf(far) : sum));
    }
  }
  return w;
}

}  // namespace

// Error bounds of the fast keys.  Sigmoid: the relative error of ex2.approx
// and of its rounded argument enters damped by s (1 - s) |z| <= 0.23, so s is
// within 3e-7 of its value, and the sum with b within half a step of |c|.
// Softmax: p |z - m| <= 0.37 likewise, but the denominator of up to 2048
// terms adds a relative 1e-6.
constexpr float kSlackSigmoid = 4e-7f, kSlackSoftmax = 2e-6f, kSlackStep = 1.3e-7f;
// What two keys of fine_key leave open (and what 64 bits do, for large biases).
constexpr float kFineNear = 4e-9f;
// Relative error of a sum of two unbiased scores, |z - m| up to 90.
constexpr float kSlackPair = 1.4e-5f;

template <typename ZT, int NPL, bool SOFTMAX, bool BIAS>
__global__ void __launch_bounds__(256, NPL <= 12 ? 4 : 3) route_select_kernel(const __grid_constant__ SelectArgs a) {
  extern __shared__ __align__(16) uint8_t rs_smem[];
  __shared__ __align__(16) uint32_t ranked[8][32];
  __shared__ float fine[BIAS && !SOFTMAX ? 8 : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  const ZT* row = static_cast<const ZT*>(a.z) + static_cast<size_t>(t) * a.ld;
  double* ckey = reinterpret_cast<double*>(rs_smem) + static_cast<size_t>(warp) * a.E;
  uint16_t* cid = reinterpret_cast<uint16_t*>(rs_smem + (blockDim.x >> 5) * a.E * sizeof(double)) +
                  static_cast<size_t>(warp) * a.E;

  const int g = (lane * a.inv_L) >> 16, r = lane - g * a.L;  // lane / L
  const int base = g * a.gs + r * a.c;
  const int cnt = g < a.G ? max(0, min(a.c, a.gs - r * a.c)) : 0;

  // NPL > 0: the lane's logits and keys are in registers; NPL == 0 (more
  // experts to a lane than are worth unrolling): in shared memory
  constexpr bool REG = NPL > 0;
  float zreg[REG ? NPL : 1];
  uint32_t oreg[REG ? NPL : 1];
  float* zmem = reinterpret_cast<float*>(rs_smem + ((blockDim.x >> 5) * a.E * kListBytes + 3) / 4 * 4) +
                static_cast<size_t>(warp) * 2 * a.E + base;
  uint32_t* omem = reinterpret_cast<uint32_t*>(zmem + a.E);
  auto Z = [&](int i) -> float& {
    if constexpr (REG) return zreg[i]; else return zmem[i];
  };
  auto O = [&](int i) -> uint32_t& {
    if constexpr (REG) return oreg[i]; else return omem[i];
  };
  const int NI = REG ? NPL : cnt;

  // ---- logits
  if (a.vec) {
#pragma unroll
    for (int i = 0; i < NI; i += 4) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (!REG || i < cnt) {
        if constexpr (sizeof(ZT) == 2) {
          const uint2 q = *reinterpret_cast<const uint2*>(row + base + i);
          v = make_float4(bf16_bits_to_f32(q.x & 0xffffu), bf16_bits_to_f32(q.x >> 16),
                          bf16_bits_to_f32(q.y & 0xffffu), bf16_bits_to_f32(q.y >> 16));
        } else {
          v = *reinterpret_cast<const float4*>(row + base + i);
          for (int p = 1; p < a.S; ++p) {
            const float4 q = *reinterpret_cast<const float4*>(row + p * a.sp + base + i);
            v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
          }
        }
      }
      Z(i) = clean(v.x); Z(i + 1) = clean(v.y); Z(i + 2) = clean(v.z); Z(i + 3) = clean(v.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) Z(i) = i < cnt ? logit(a, row, base + i) : -INFINITY;
  }

  // ---- softmax maximum and denominator
  float m = 0.f, sum = 1.f;
  if constexpr (SOFTMAX) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i) m = fmaxf(m, Z(i));
    m = warp_max(m);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      sum += Z(i) == -INFINITY ? 0.f : (Z(i) == m ? 1.f : fast_exp(Z(i) - m));
    sum = warp_sum(sum);
    if (sum == 0.f) sum = 1.f;  // no expert available: every score is 0
  }
  const float inv_sum = SOFTMAX ? 1.f / sum : 1.f;
  auto fast_score = [&](float v) {
    if constexpr (SOFTMAX)
      return v == -INFINITY ? 0.f : (v == m ? 1.f : fast_exp(v - m)) * inv_sum;
    else
      return fast_rcp(1.f + fast_exp(-v));
  };
  // of an expert's logit and bias (a sum of a score and a bias is never -0)
  auto fast_key = [&](float z, float b) {
    if constexpr (BIAS) {
      const float c = fmaxf(fast_score(z) + b, -INFINITY);
      return order_key(z == -INFINITY ? -INFINITY : c);
    }
    return order_key(z);
  };

  // ---- keys
  if constexpr (BIAS) {
    auto key = [&](int i, float b) { O(i) = fast_key(Z(i), b); };
    if (a.vec_bias) {
#pragma unroll
      for (int i = 0; i < NI; i += 4) {
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!REG || i < cnt) b = *reinterpret_cast<const float4*>(a.bias + base + i);
        key(i, b.x);
        key(i + 1, b.y);
        key(i + 2, b.z);
        key(i + 3, b.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) key(i, i < cnt ? a.bias[base + i] : 0.f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) O(i) = fast_key(Z(i), 0.f);
  }
  if (!a.full) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (i >= cnt) O(i) = kAbsent;
  }

  // ---- groups
  uint32_t mx = kAbsent;
  if (a.tg < a.G) {
    uint32_t uh = kAbsent, ul = kAbsent;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      ul = max(ul, min(uh, O(i)));
      uh = max(uh, O(i));
    }
    float hi = uh == kAbsent ? -INFINITY : key_value(uh);
    float lo = ul == kAbsent ? -INFINITY : key_value(ul);
    top2_segment(hi, lo, r, a.L);
    float score = hi, slack = 0.f;
    if (!a.best_only && hi > -INFINITY) {
      if constexpr (BIAS) {
        if (lo > -INFINITY) score = hi + lo;
      } else {  // the order of the logits gave the two; their scores are summed
        score = fast_score(hi) + (lo > -INFINITY ? fast_score(lo) : 0.f);
        slack = 2.f * kSlackPair * score + 1e-37f;  // and what is below fp32's range
      }
    }
    if constexpr (BIAS)
      slack = 4.f * (SOFTMAX ? kSlackSoftmax : kSlackSigmoid) +
              4.f * kSlackStep * (fabsf(hi) + (lo > -INFINITY ? fabsf(lo) : 0.f));
    // the best topk_groups groups: the highest score left, lowest group first
    const bool lead = g < a.G && r == 0;
    uint32_t left = lead ? order_key(score + 0.0f) : 0u, low = 0;
    bool kept = false;
    for (int j = 0; j < a.tg; ++j) {
      low = __reduce_max_sync(0xffffffffu, left);
      if (lane == __ffs(__ballot_sync(0xffffffffu, left == low)) - 1) {
        kept = true;
        left = 0;
      }
    }
    const uint32_t high = __reduce_max_sync(0xffffffffu, left);  // of the dropped ones
    kept = __shfl_sync(0xffffffffu, kept, min(g, a.G - 1) * a.L);
    float sl = 0.f;
    if constexpr (BIAS) {  // largest slack of any group
      sl = key_value(__reduce_max_sync(0xffffffffu, order_key(lead && slack < INFINITY ? slack : 0.f)));
    } else {
      if (!a.best_only)
        sl = key_value(__reduce_max_sync(0xffffffffu, order_key(lead ? slack : 0.f)));
    }
    // NaN (inf - inf) compares false: equal infinities are ties of their own
    if (sl > 0.f && key_value(low) - key_value(high) <= sl) {
      // the experts that can be among their group's two best
      float bound = __shfl_sync(0xffffffffu, lo, min(g, a.G - 1) * a.L);
      if constexpr (BIAS) {
        if (bound > -INFINITY && bound < INFINITY)
          bound -= 2.f * (SOFTMAX ? kSlackSoftmax : kSlackSigmoid) + 2.f * kSlackStep * fabsf(bound);
      }
      const uint32_t low_key = max(order_key(clean(bound)), kUnavail + 1);
      int take = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) take += O(i) >= low_key ? 1 : 0;
      int at = take;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += v;
      }
      const int listed = __shfl_sync(0xffffffffu, at, 31);
      if (listed <= 32) {
        at -= take;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (O(i) >= low_key) cid[at++] = static_cast<uint16_t>(base + i);
        __syncwarp();
        kept = group_kept64<ZT, SOFTMAX, BIAS>(a, row, m, g, cid, listed);
        __syncwarp();
      } else {
        kept = group_kept64_all<ZT, SOFTMAX, BIAS>(a, row, m, g, r, base, cnt);
      }
    }
    if (!kept) {
#pragma unroll
      for (int i = 0; i < NI; ++i) O(i) = kAbsent;
    }
    mx = kept ? uh : kAbsent;
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) mx = max(mx, O(i));
  }

  // ---- candidates: at or above the k-th largest lane maximum
  uint32_t thr = 0;
  if (a.k <= 12) {
    // the k-th largest distinct maximum (equal ones leave together): a bound
    // as good, and k reductions cost less than a sort
    uint32_t left = mx;
    for (int j = 0; j < a.k; ++j) {
      thr = __reduce_max_sync(0xffffffffu, left);
      if (left == thr) left = 0;
    }
  } else {
    uint32_t srt = mx;  // bitonic, descending over the lanes
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
      for (int d = size >> 1; d > 0; d >>= 1) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, srt, d);
        const bool keep_max = ((lane & size) == 0) == ((lane & d) == 0);
        srt = keep_max ? max(srt, other) : min(srt, other);
      }
    }
    thr = __shfl_sync(0xffffffffu, srt, a.k - 1);
  }
  thr = max(thr, kUnavail);
  constexpr float near = 2.f * (SOFTMAX ? kSlackSoftmax : kSlackSigmoid);
  auto with_slack = [&](uint32_t k) {
    if constexpr (BIAS) {
      const float v = key_value(k);
      if (v > -INFINITY && v < INFINITY)
        return order_key(clean(v - (near + 2.f * kSlackStep * fabsf(v))));
    }
    return k;
  };
  auto at_or_above = [&](uint32_t k) {  // in registers: one bit each
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (O(i) >= k) c += REG ? 1u << i : 1u;
    return c;
  };
  auto count = [](uint32_t c) { return REG ? __popc(c) : static_cast<int>(c); };
  uint32_t mine = at_or_above(with_slack(thr));
  int n = __reduce_add_sync(0xffffffffu, count(mine));
  if (n > 32) {
    // the bound is weak where few lanes hold the kept groups or k is near 32:
    // halve the range of keys until k to 32 experts are left
    uint32_t above = __reduce_max_sync(0xffffffffu, mx);  // fewer than k lie above it
    while (thr < above) {
      const uint32_t mid = thr + (above - thr + 1) / 2;
      if (__reduce_add_sync(0xffffffffu, count(at_or_above(mid))) < a.k) {
        above = mid - 1;
        continue;
      }
      thr = mid;
      mine = at_or_above(with_slack(thr));
      n = __reduce_add_sync(0xffffffffu, count(mine));
      if (n <= 32) break;
    }
  }
  int pos = count(mine);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, pos, d);
    if (lane >= d) pos += v;
  }
  pos -= count(mine);
  if constexpr (REG) {
    for (; mine; mine &= mine - 1) cid[pos++] = static_cast<uint16_t>(base + __ffs(mine) - 1);
  } else {
    thr = with_slack(thr);
    for (int i = 0; i < NI; ++i)
      if (O(i) >= thr) cid[pos++] = static_cast<uint16_t>(base + i);
  }
  __syncwarp();

  int my_id = -1, rank = 32;
  float my_z = -INFINITY, my_b = 0.f;
  if (n <= 32) {
    // one candidate to a lane, in id order; ranked against the others
    uint32_t key = 0;
    if (lane < n) {
      my_id = cid[lane];
      my_z = logit(a, row, my_id);
      if constexpr (BIAS) my_b = a.bias[my_id];
      key = fast_key(my_z, my_b);
    }
    uint32_t* keys = ranked[warp];
    keys[lane] = key;
    __syncwarp();
    rank = 0;
    for (int j = 0; j < n; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&keys[j]);  // 0 after the last
      const uint32_t other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        rank += other[q] > key || (other[q] == key && j + q < lane) ? 1 : 0;
    }
    if (lane >= n) rank = 32;
    bool close = false;
    if constexpr (BIAS) {
      // the keys in descending order; neighbours within their error are not
      // decided yet (infinite keys are: next to equal ones the ids decide)
      __syncwarp();
      if (lane < n) keys[rank] = key;
      __syncwarp();
      if (lane < n && lane > 0) {
        const float hi = key_value(keys[lane - 1]), lo = key_value(keys[lane]);
        close = hi < INFINITY && lo > -INFINITY && lane <= a.k &&
                hi - lo <= near + kSlackStep * (fabsf(hi) + fabsf(lo));
      }
    }
    if constexpr (BIAS && !SOFTMAX) {
      if (__any_sync(0xffffffffu, close)) {  // in some tokens of a thousand
        __syncwarp();
        float low = 0.f;
        const float c = lane < n ? fine_key(my_z, my_b, low) : 0.f;
        key = lane < n ? order_key(my_z == -INFINITY ? -INFINITY : clean(c)) : 0;
        if (key == kUnavail) low = 0.f;  // unavailable ones are equal, whatever their bias
        float* lows = fine[warp];
        keys[lane] = key;
        lows[lane] = low;
        __syncwarp();
        rank = 0;
        for (int j = 0; j < n; ++j) {
          const uint32_t other = keys[j];
          const float ol = lows[j];
          rank += other > key || (other == key && (ol > low || (ol == low && j < lane))) ? 1 : 0;
        }
        __syncwarp();
        if (lane < n) {
          keys[rank] = key;
          lows[rank] = low;
        } else {
          rank = 32;
        }
        __syncwarp();
        close = false;
        if (lane < n && lane > 0) {
          const float hi = key_value(keys[lane - 1]), lo = key_value(keys[lane]);
          close = hi < INFINITY && lo > -INFINITY && lane <= a.k &&
                  (hi - lo) + (lows[lane - 1] - lows[lane]) <= kFineNear + 1e-14f * fabsf(lo);
        }
      }
    }
    if constexpr (BIAS) {
      if (__any_sync(0xffffffffu, close))
        rank = rank64<ZT, SOFTMAX>(a, row, m, my_id, n, ckey);
    }
  } else {
    my_id = select_many<ZT, SOFTMAX, BIAS>(a, row, m, ckey, cid, n);
    if (my_id >= 0) {
      rank = lane;
      my_z = logit(a, row, my_id);
      if constexpr (BIAS) my_b = a.bias[my_id];
    }
  }

  // ---- weights of the selected, unbiased.  The divisions are the fast ones, off by
  // up to two steps of fp32 each: the weights' error is 7e-8 (rms), and 5e-8 with
  // rounded divisions, which take 3 to 5 % longer
  float zz = -INFINITY;
  if (rank < a.k) {
    zz = my_z;
    if constexpr (BIAS)  // a bias of -inf or NaN takes an expert out as well
      if (my_b != my_b || my_b == -INFINITY) zz = -INFINITY;
  }
  // scores far below 1 take their own way: they may be below fp32's range
  float w;
  if (__any_sync(0xffffffffu, zz > -INFINITY && (SOFTMAX ? m - zz > 80.f : zz < -80.f))) {
    w = weight_far<SOFTMAX>(a, zz, m, sum);
  } else {
    if constexpr (SOFTMAX)
      w = zz == -INFINITY ? 0.f : exp_diff(zz, m);
    else
      w = zz == -INFINITY ? 0.f : __fdividef(1.0f, 1.0f + expf(-zz));
    const float den = a.renorm ? warp_sum(w) + 1e-20f * sum : sum;
    w = __fdividef(w, den);
  }
  if (rank < a.k) {
    const size_t at = static_cast<size_t>(t) * a.k + rank;
    a.idx[at] = my_id;
    a.w[at] = w * a.scale;
  }
}

int check_route_config(const moe_route_config* cfg) {
  if (!cfg) return MOE_ERR_INVALID;
  const moe_route_config& c = *cfg;
  if (c.E <= 0 || c.k <= 0 || c.groups <= 0 || c.topk_groups <= 0) return MOE_ERR_INVALID;
  if (c.score != MOE_SCORE_SIGMOID && c.score != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID;
  if (c.group_score != MOE_GROUP_TOP2 && c.group_score != MOE_GROUP_MAX) return MOE_ERR_INVALID;
  if (c.topk_groups > c.groups) return MOE_ERR_INVALID;
  if (!(c.scale == c.scale) || isinf(c.scale)) return MOE_ERR_INVALID;
  if (c.E > kMaxExperts || c.groups > 32 || c.E % c.groups != 0 || c.k > kMaxTopK)
    return MOE_ERR_UNSUPPORTED;
  if (c.k > c.topk_groups * (c.E / c.groups)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

namespace {

template <typename ZT, int NPL>
int launch_npl(const moe_route_config& cfg, const SelectArgs& a, int warps, size_t smem,
               cudaStream_t s) {
  const bool soft = cfg.score == MOE_SCORE_SOFTMAX, bias = a.bias != nullptr;
  auto kern = soft ? (bias ? route_select_kernel<ZT, NPL, true, true>
                           : route_select_kernel<ZT, NPL, true, false>)
                   : (bias ? route_select_kernel<ZT, NPL, false, true>
                           : route_select_kernel<ZT, NPL, false, false>);
  kern<<<(a.T + warps - 1) / warps, 32 * warps, smem, s>>>(a);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <typename ZT>
int launch_type(const moe_route_config& cfg, const SelectArgs& a, int warps, size_t smem,
                cudaStream_t s) {
  if (a.c <= 4) return launch_npl<ZT, 4>(cfg, a, warps, smem, s);
  if (a.c <= 8) return launch_npl<ZT, 8>(cfg, a, warps, smem, s);
  if (a.c <= 12) return launch_npl<ZT, 12>(cfg, a, warps, smem, s);
  if (a.c <= 16) return launch_npl<ZT, 16>(cfg, a, warps, smem, s);
  return launch_npl<ZT, 0>(cfg, a, warps, smem, s);
}

}  // namespace

int launch_route_select(const moe_route_config& cfg, const void* in, bool bf16, size_t ld, int S,
                        size_t sp, const float* bias, int T, int32_t* topk_idx, float* topk_w,
                        cudaStream_t s) {
  SelectArgs a{};
  a.z = in;
  a.ld = ld;
  a.sp = sp;
  a.S = S;
  a.bias = bias;
  a.T = T;
  a.E = cfg.E;
  a.k = cfg.k;
  a.G = cfg.groups;
  a.tg = cfg.topk_groups;
  // all groups kept: one group of everything
  if (a.tg == a.G) a.G = a.tg = 1;
  a.gs = a.E / a.G;
  a.L = 32 / a.G;
  a.inv_L = (65536 + a.L - 1) / a.L;
  a.c = (a.gs + a.L - 1) / a.L;
  const size_t item = bf16 ? 2 : 4;
  if (a.gs % 4 == 0 && ld % 4 == 0 && sp % 4 == 0 && aligned(in, 4 * item)) {
    a.vec = 1;
    a.c = (a.c + 3) / 4 * 4;
  }
  a.vec_bias = a.vec && aligned(bias, 16);
  a.full = a.G * a.L == 32 && a.L * a.c == a.gs && (a.c > 16 || a.c % 4 == 0);
  a.best_only = cfg.group_score == MOE_GROUP_MAX;
  a.renorm = cfg.renorm;
  a.scale = cfg.scale;
  a.idx = topk_idx;
  a.w = topk_w;
  // eight tokens to a CTA once every SM has some; few tokens are spread over
  // the SMs; a large E leaves room for fewer candidate lists
  const int sms = num_sms();
  int warps = T >= 16 * sms ? 8 : (T >= 4 * sms ? 2 : 1);
  const size_t per = static_cast<size_t>(a.E) * (kListBytes + (a.c > 16 ? 8 : 0));
  static_assert(kMaxExperts * (kListBytes + 8) + 4 <= 40 * 1024, "one token's fits as it is");
  while (warps > 1 && warps * per > 40 * 1024) warps >>= 1;
  // a candidate list rounded up so that what follows it is 4-byte aligned
  const size_t smem = warps * per + 4;
  return bf16 ? launch_type<uint16_t>(cfg, a, warps, smem, s)
              : launch_type<float>(cfg, a, warps, smem, s);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_route_logits(const moe_route_config* cfg, const void* logits, int logits_bf16,
                                int64_t ld, const float* bias, int T, int32_t* topk_idx,
                                float* topk_w, void* stream) {
  moe::Range range_("moe_route_logits");
  const int rc = check_route_config(cfg);
  if (rc) return rc;
  if (T < 0 || ld < cfg->E) return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_INVALID;
  if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(topk_w, 4))
    return MOE_ERR_INVALID;
  return launch_route_select(*cfg, logits, logits_bf16 != 0, static_cast<size_t>(ld), 1, 0, bias, T,
                             topk_idx, topk_w, static_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_route_grouped_workspace_size(const moe_route_config* cfg, int T, int H) {
  if (!cfg) return 0;
  return moe_route_workspace_size(T, H, cfg->E);
}

extern "C" int moe_route_grouped(const moe_route_config* cfg, const uint16_t* x,
                                 const float* w_router, const uint16_t* w_terms, const float* bias,
                                 int T, int H, int32_t* topk_idx, float* topk_w, void* ws,
                                 size_t ws_bytes, void* stream) {
  moe::Range range_("moe_route_grouped");
  int rc = check_route_config(cfg);
  if (rc) return rc;
  if (T < 0 || H <= 0) return MOE_ERR_INVALID;
  if (H % 64 != 0) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !topk_idx || !topk_w || !ws) return MOE_ERR_INVALID;
  if (!aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(ws, 256))
    return MOE_ERR_INVALID;
  if (ws_bytes < moe_route_workspace_size(T, H, cfg->E)) return MOE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouterLogits z;
  rc = launch_router_logits(x, w_router, w_terms, T, H, cfg->E, ws, &z, s);
  if (rc) return rc;
  return launch_route_select(*cfg, z.part, false, z.st, z.S, z.sp, bias, T, topk_idx, topk_w, s);
}
