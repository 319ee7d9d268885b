// The routed experts of a few tokens (T <= 32) in two launches.
//
// What the work is: every weight of every chosen expert is read once and used
// for a handful of tokens, so the HBM rate bounds it and everything else has
// to hide behind the weights' stream.
//
//   few_front_kernel   the router's logits (one pass over its fp32 weight), x as
//                      fp16 in the order of the packed nibbles, counters to zero
//   few_kernel         two persistent CTAs per SM (one, with bf16 weights and from some
//                      15 tokens on: few_stages).  Every CTA selects the experts
//                      (the same arithmetic everywhere, cheaper than another
//                      launch), then takes units of work in ticket order: 16
//                      gate rows and the 16 up rows of the same columns, times the
//                      tokens (at most 2) of one chunk of one expert, or 32 rows of
//                      the down projections of a group of chunks, one after another.
//
// Tickets are taken in the order of the units, a CTA works on its own in ascending
// order, and a unit waits only for units with lower tickets (a down projection for
// its expert's h).  Those are held by CTAs that run, so the kernel ends whatever
// else holds SMs: no CTA waits for one that has not started.
//
// Roles of a CTA: warp 0 copies weights into a ring (TMA), warp 1 their scales and the
// tokens' rows (once the units they wait for are done), the last eight multiply, and
// two between them take the finished segments in turn.  Twelve warps and two CTAs leave
// 80 registers to a thread.  The ring runs on across units and phases, so the weights of
// a down projection arrive while its h is still being computed.  A slot holds 36 KB: half
// as much, in twice as many slots, costs more at every slot than it hides (32 tokens, 384
// experts of 7168 x 2048: 991 us against 862).
//
// The products use m16n8k16 MMAs: 16 weight rows, 8 columns.  At 8 tokens a
// weight byte is worth 32 operations, a hundredth of what would make the tensor
// cores matter; the cost is the conversion of the nibbles, the same for
// any MMA, and tcgen05 would add the trip of the converted weights through
// shared or tensor memory.  An SM takes 1100 cycles for a slot's products (an MMA of
// this form 8 cycles of a quarter of it, the logic operations that turn nibbles into fp16
// 2 each), HBM 1570: near enough to one another that they do not overlap fully.
//
// Measured (graphs of calls; behind it the bytes at the measured copy rate): the layer of
// one token, 8 of 384 experts, 7168 x 2048: 53 us, 31; of 32 tokens: 812 us, 689; 6
// tokens of 3584 x 1024, experts alone: 50 us, 20; 16 tokens of 256 x 128: 26 us, the
// latency of its steps.
#include "few.cuh"

#include <cuda_fp16.h>

#include "adapter.cuh"

namespace moe {

namespace {

constexpr int C = kFewColumns;
constexpr int kMul = 8;                      // warps that multiply, each a share of K
constexpr int kCopy = 2;                     // warps that copy: weights, the rest
constexpr int kFinish = 2;                   // warps that take finished segments
constexpr int kFirstMul = kCopy + kFinish;   // warps before the multiplying ones
constexpr int kThreads = 32 * (kFirstMul + kMul);
constexpr int kCtas = 2;                     // of an SM: one waits while the other multiplies
constexpr int kFrontThreads = 256;
constexpr int kFrontExperts = 2;             // router rows of a CTA
constexpr int kFrontTokens = 4;              // tokens at a time
static_assert(kFrontTokens * kFrontExperts == 8, "sums over the warp");
// float4 of a router row held by a thread: 7168 columns a pass over the tokens.  Wider rows
// take another (32 tokens, 384 small experts: H 7168 219 us, 7232 223).
constexpr int kFrontLoads = 7;

// Ring slot: weights (32 rows of C / 2 bytes: for each row block of 16, pieces of 128
// bytes of its rows, swizzled), scales (32 rows, swizzled), rows of tokens: fp16
// blocks with their start values, or bf16 rows in swizzled pieces like the weights.
constexpr int kWeightBytes = 32 * C / 2;
constexpr int kScaleBytes = 32 * C / 16;
constexpr int kStarts = 2 * C;  // where a row's start values lie
constexpr int kPitch4 = kFewBlock;
__host__ __device__ constexpr int slot_bytes(int rows_bytes) {
  return kWeightBytes + kScaleBytes + (rows_bytes + 1023) / 1024 * 1024;
}
// Room for the rows of tokens: of a chunk, or in 128-byte pieces of bf16.
__host__ __device__ __forceinline__ int rows_bytes(const FewArgs& a) {
  const int four = (a.T < kFewChunk ? a.T : kFewChunk) * kPitch4;
  const int two = a.L > 0 || a.S > 0 ? (a.T < kFewRows ? a.T : kFewRows) * (C / 2) : 0;
  const int parts = a.L > 0 || a.S > 0 ? 2 * (a.T < kFewRows / 2 ? a.T : kFewRows / 2) * (C / 2) : 0;
  const int wide = two > parts ? two : parts;
  return four > wide ? four : wide;
}

constexpr int kMaxSlots = 8;
constexpr int kAhead = 2;  // tickets a CTA holds
// The matrix of a unit's first row block, 4 bits a kind.
constexpr uint32_t kFirstMatrix =
    kFewLatDownW << 4 * kFewLatDown | kFewSharedGateW << 4 * kFewSharedUp |
    kFewGateW << 4 * kFewGateUp | kFewDownW << 4 * kFewDown |
    kFewSharedDownW << 4 * kFewSharedDown | kFewLatUpW << 4 * kFewLatUp;

// Partial sums of a finished segment for each finishing warp; at first what only the
// making of the lists needs.
__host__ __device__ __forceinline__ int sum_tokens(const FewArgs& a) {
  const int most = a.L > 0 || a.S > 0 ? kFewRows : kFewChunk;
  return a.T < most ? a.T : most;
}
__host__ __device__ __forceinline__ int sums_bytes(const FewArgs& a) {
  const int sums = kFinish * kMul * 2 * sum_tokens(a) * 16 * 4, lists = 6 * (a.E + a.T * a.k);
  return ((sums > lists ? sums : lists) + 15) / 16 * 16;
}

// One header per slot and per finishing warp.  A segment is what one chunk adds to
// a unit.
struct __align__(16) Header {
  int kind;   // FewKind, | kScaled, | kLastSlot, | kLastSegment
  int size;   // tokens, | columns of K << 16
  int which;  // expert chunk, or chunk of tokens
  int n0;     // first column of the output
  __device__ __forceinline__ int rows() const { return size & 0xffff; }
  __device__ __forceinline__ int cols() const { return size >> 16; }
};
constexpr int kLastSlot = 256;     // of its segment
constexpr int kLastSegment = 512;  // of its unit
// Added to the kind of a segment whose activations have units of their own (so that it is
// not is_int4: only multiply() meets it); then the slot's place in its segment stands above
// the other bits.  Set by the warp that copies the rows.
constexpr int kScaled = 128, kSlotShift = 11;
static_assert(kFewEnd < kScaled, "kinds");
static_assert(kFewWidth / kFewColumns <= 1 << (31 - kSlotShift), "the slot's place");

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The eight nibbles of a word as fp16 pairs (columns 0 4, 1 5, 2 6, 3 7), exactly but
// for a constant: in the low mantissa bits of 1024.0 a nibble makes 1032 + q, in
// bits 4-7 of 64.0 it makes 72 + q.  One shift and four three-input operations: as
// those take one immediate, the second constant of each has to come from a
// register that the compiler does not see through (else it makes two of them, 9.4
// instructions a word against 5.8).
struct Magic {
  uint32_t lo, hi;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x64086408;" : "=r"(lo));
    asm volatile("mov.b32 %0, 0x54805480;" : "=r"(hi));
  }
};

__device__ __forceinline__ void nibbles(uint32_t w, const Magic& m, uint32_t (&q)[4]) {
  const uint32_t w8 = w >> 8;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0x6a;" : "=r"(q[0]) : "r"(w), "r"(m.lo));  // (w & a) ^ b
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0x6a;" : "=r"(q[1]) : "r"(w), "r"(m.hi));
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0x6a;" : "=r"(q[2]) : "r"(w8), "r"(m.lo));
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0x6a;" : "=r"(q[3]) : "r"(w8), "r"(m.hi));
}

// So a product with the activations v starts from -(1032 sum of the even columns + 72
// sum of the odd ones): what one value of column c adds to it.
__device__ __forceinline__ float start_of(float v, int c) { return c & 1 ? -72.f * v : -1032.f * v; }

// Weights pass through L2 once and first make room again: else 200 MB of them a call would
// push everything else out, the kernels' own code too, which then comes from HBM line
// by line (10 us at the start of a call).
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void copy_once_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c1,
                                             int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void copy_once_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                             int c1, int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

__device__ __forceinline__ int load_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void add_release(int32_t* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ int add_acq_rel(int32_t* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Columns of K (int4) or of the bf16 rows that one slot holds, and the length of K.
__device__ __forceinline__ bool is_int4(int kind) { return (kind | 1) == kFewDown; }
static_assert(kFewGateUp == 2 && kFewDown == 3, "is_int4");
static_assert(C / 128 <= 2 * kMul && kMul == 8, "at most two steps a warp and slot");
__device__ __forceinline__ int length_of(const FewArgs& a, int kind) {
  switch (kind) {
    case kFewLatDown:
    case kFewSharedUp: return a.H;
    case kFewGateUp: return a.D;
    case kFewDown: return a.I;
    case kFewSharedDown: return a.S;
    default: return a.L;
  }
}

// Order of fp32 values as integers, above 0 for every value.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}

// ------------------------------------------------------------------ prologue

// CTAs below `routers` take kFrontExperts rows of the router, the next T a token
// each; the last CTA of all clears the counters.
__global__ void __launch_bounds__(kFrontThreads) few_front_kernel(const FewArgs a, int routers) {
  grid_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (static_cast<int>(blockIdx.x) == static_cast<int>(gridDim.x) - 1)
    for (int i = tid; i < a.n_counters; i += kFrontThreads) a.counters[i] = 0;

  if (static_cast<int>(blockIdx.x) < routers) {
    // A thread holds its columns of the router's rows and meets every token with
    // them: the weight is read once, from all SMs at once, and x comes from L2.
    __shared__ float part[kFewTokens][kFrontExperts][kFrontThreads / 32];
    const int e0 = blockIdx.x * kFrontExperts;
    constexpr int kStep = 4 * kFrontThreads * kFrontLoads;
    for (int h0 = 0; h0 < a.H; h0 += kStep) {
      float4 w[kFrontExperts][kFrontLoads];
#pragma unroll
      for (int i = 0; i < kFrontLoads; ++i) {
        const int c = h0 + 4 * (tid + i * kFrontThreads);
#pragma unroll
        for (int e = 0; e < kFrontExperts; ++e) {
          w[e][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < a.H && e0 + e < a.E)
            w[e][i] = __ldcs(reinterpret_cast<const float4*>(a.router_w + (size_t)(e0 + e) * a.H + c));
        }
      }
      // kFrontTokens at a time, their loads on the way together (32 tokens, 384 experts of
      // 7168: 23 us two at a time, 14 four)
#pragma unroll 1
      for (int t0 = 0; t0 < a.T; t0 += kFrontTokens) {
        float z[kFrontTokens * kFrontExperts] = {};
#pragma unroll
        for (int i = 0; i < kFrontLoads; ++i) {
          const int c = h0 + 4 * (tid + i * kFrontThreads);
          uint2 v[kFrontTokens];
#pragma unroll
          for (int t = 0; t < kFrontTokens; ++t) {
            v[t] = make_uint2(0u, 0u);
            if (c < a.H && t0 + t < a.T)
              v[t] = __ldg(reinterpret_cast<const uint2*>(a.x + (size_t)(t0 + t) * a.H + c));
          }
#pragma unroll
          for (int t = 0; t < kFrontTokens; ++t) {
            const float x0 = __uint_as_float(v[t].x << 16), x1 = __uint_as_float(v[t].x & 0xffff0000u);
            const float x2 = __uint_as_float(v[t].y << 16), x3 = __uint_as_float(v[t].y & 0xffff0000u);
#pragma unroll
            for (int e = 0; e < kFrontExperts; ++e) {
              float& to = z[t * kFrontExperts + e];
              to = fmaf(x0, w[e][i].x, to);
              to = fmaf(x1, w[e][i].y, to);
              to = fmaf(x2, w[e][i].z, to);
              to = fmaf(x3, w[e][i].w, to);
            }
          }
        }
        // sums over the warp, half of the values in each half of the lanes at every step:
        // lane 4 j gets value j
#pragma unroll
        for (int o = 16, n = kFrontTokens * kFrontExperts / 2; n > 0; o >>= 1, n >>= 1)
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const bool upper = lane & o;
            const float give = upper ? z[i] : z[i + n];
            z[i] = (upper ? z[i + n] : z[i]) + __shfl_xor_sync(0xffffffffu, give, o);
          }
        z[0] += __shfl_xor_sync(0xffffffffu, z[0], 2);
        z[0] += __shfl_xor_sync(0xffffffffu, z[0], 1);
        const int t = t0 + lane / 4 / kFrontExperts;
        if (!(lane & 3) && t < a.T) {
          float* to = &part[t][lane / 4 % kFrontExperts][warp];
          *to = h0 ? *to + z[0] : z[0];
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < a.T * kFrontExperts; i += kFrontThreads) {
      const int t = i / kFrontExperts, e = i % kFrontExperts;
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < kFrontThreads / 32; ++w) z += part[t][e][w];
      if (e0 + e < a.E) {
        const float score = 1.0f / (1.0f + expf(-z));
        const float key = score + __ldg(a.router_bias + e0 + e);
        const size_t at = (size_t)t * a.E + e0 + e;
        a.scores[at] = score;
        a.keys[at] = ordered(key != key ? -INFINITY : key);  // NaN ranks last
      }
    }
    return;
  }

  // x as fp16 in pair order, times the power of two that brings the token's
  // largest value to [2^14, 2^15): bf16's 8 bits stay whole down to 2^-29 of it
  const int t = static_cast<int>(blockIdx.x) - routers;
  if (t >= a.T || a.L > 0) return;
  __shared__ float top[kFrontThreads / 32];
  const uint16_t* row = a.x + (size_t)t * a.H;
  float m = 0.f;
  for (int c = 8 * tid; c < a.H; c += 8 * kFrontThreads) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + c));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i] << 16)),
                         fabsf(__uint_as_float(w[i] & 0xffff0000u))));
  }
  m = warp_max(m);
  if (lane == 0) top[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kFrontThreads / 32; ++w) m = fmaxf(m, top[w]);
  // exponent field of 2^(14 - floor(log2 m)), at most 2^126; 1 where m is 0 or not finite
  const int field = static_cast<int>(__float_as_uint(m) >> 23);
  const int up = m == 0.f || field == 255 ? 127 : min(127 + 14 + 127 - field, 253);
  const float by = __uint_as_float(static_cast<uint32_t>(up) << 23);
  if (tid == 0) a.x_unit[t] = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
  uint8_t* x16 = a.x16 + t * few_row_bytes(a.D);
  for (int c0 = 0; c0 < a.H; c0 += 8 * kFrontThreads) {
    const int c = c0 + 8 * tid;
    float start = 0.f;
    if (c < a.H) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      __half2 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // columns i and i + 4
        const uint32_t lo = (w[i >> 1] >> (16 * (i & 1))) << 16;
        const uint32_t hi = (w[2 + (i >> 1)] >> (16 * (i & 1))) << 16;
        p[i] = __floats2half2_rn(__uint_as_float(lo) * by, __uint_as_float(hi) * by);
        start += start_of(__low2float(p[i]) + __high2float(p[i]), i);
      }
      *reinterpret_cast<uint4*>(x16 + few_value_at(c)) = *reinterpret_cast<const uint4*>(p);
    }
    start += __shfl_xor_sync(0xffffffffu, start, 1);  // 16 columns
    if (c < a.H && !(tid & 1)) *reinterpret_cast<float*>(x16 + few_start_at(c)) = start;
  }
}

// ----------------------------------------------------------------- selection

// The chosen experts as lists in shared memory.  A row is one (token, expert) pair;
// the rows of a chunk follow one another.
struct Lists {
  float* row_weight;  // [T k] weight of a row's output
  uint32_t* tokens;   // [chunks] tokens, one bit each
  uint16_t* expert;   // [chunks]
  uint16_t* row0;     // [chunks] first row
  uint32_t* scaled;   // [T k] bits: a chunk's h has units of its own (the copying warp's)
};

// Ring and buffers of a CTA.
struct Ring {
  uint8_t* slots;
  int bytes;  // of a slot
  int n;      // slots
  Header* header;
  uint64_t* full;
  uint64_t* empty;
  uint64_t* named;  // header written
  __device__ __forceinline__ uint8_t* slot(uint32_t s) const { return slots + s * bytes; }
  __device__ __forceinline__ uint8_t* scales(uint32_t s) const { return slot(s) + kWeightBytes; }
  __device__ __forceinline__ uint8_t* rows(uint32_t s) const {
    return slot(s) + kWeightBytes + kScaleBytes;
  }
};

// Finished segments: partial sums [warp][block][token][16 rows] for each finishing
// warp, and its weighted sums [token][32 columns] over the segments of a unit.
struct Sums {
  float* part;
  float* unit;
  int tokens;
  Header* header;
  uint64_t* full;
  uint64_t* empty;
  __device__ __forceinline__ float* at(int buf, int warp, int block, int token) const {
    return part + (((buf * kMul + warp) * 2 + block) * tokens + token) * 16;
  }
};

// What the roles of a CTA share, at the start of its shared memory.  Each role is a
// function of its own that reads this: so each gets the registers it needs, and the
// compiler sees that everything lies in shared memory.
struct __align__(16) Context {
  FewArgs a;
  Header slot_header[kMaxSlots];
  Header sum_header[kFinish];
  uint64_t full[kMaxSlots], empty[kMaxSlots], named[kMaxSlots];
  uint64_t sum_full[kFinish], sum_empty[kFinish], listed;
  uint32_t in_group[kFewGroups];    // tokens of a group of chunks
  uint32_t groups_of[kFewTokens];   // groups of a token
  int scan[kMul];
  int units[kFewKinds], each[kFewKinds];  // units of a kind; of them for one tile or chunk
  int cta_abort, chunks, per_group, groups;
  int ring_at, slot, sums_at, unit_at, lists_at;  // offsets into shared memory
};
extern __shared__ __align__(16) uint8_t few_smem[];

__device__ __forceinline__ Context& context() { return *reinterpret_cast<Context*>(few_smem); }
__device__ __forceinline__ Ring ring_of(Context& c) {
  return Ring{few_smem + c.ring_at, c.slot, c.a.stages, c.slot_header, c.full, c.empty, c.named};
}
__device__ __forceinline__ Sums sums_of(Context& c) {
  return Sums{reinterpret_cast<float*>(few_smem + c.sums_at),
              reinterpret_cast<float*>(few_smem + c.unit_at), sum_tokens(c.a), c.sum_header,
              c.sum_full, c.sum_empty};
}
__device__ __forceinline__ Lists lists_of(Context& c) {
  const int pairs = c.a.T * c.a.k;
  Lists ls;
  ls.row_weight = reinterpret_cast<float*>(few_smem + c.lists_at);
  ls.tokens = reinterpret_cast<uint32_t*>(ls.row_weight + pairs);
  ls.expert = reinterpret_cast<uint16_t*>(ls.tokens + pairs);
  ls.row0 = ls.expert + pairs;
  ls.scaled = reinterpret_cast<uint32_t*>(ls.row0 + pairs);
  return ls;
}
__device__ __forceinline__ Waiter waiter_of(Context& c) {
  return Waiter{&c.cta_abort, c.a.status, c.a.wait_ns};
}

// mbar_wait with its slow part out of line (the code of all roles shares the instruction
// caches), and for the roles that run ahead or behind with a rest between two
// looks: seven warps that look all the time take as many issue slots as the
// products.
__device__ __noinline__ bool wait_slowly(uint64_t* bar, uint32_t parity, uint32_t rest_ns) {
  const Waiter w = waiter_of(context());
  uint64_t t0 = 0;
  for (int i = 0;; ++i) {
    if (rest_ns) __nanosleep(rest_ns);
    if (mbar_try_wait(bar, parity)) return true;
    if (i < 8) continue;  // reading the clock takes longer than most waits
    if (aborted(w)) return false;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (static_cast<int64_t>(now - t0) > w.limit_ns) {
      give_up(w);
      return false;
    }
  }
}
template <int REST = 0>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_slowly(bar, parity, REST));
}
constexpr int kRest = 100;  // ns

// Keys closer than this to the border `low` are compared again in 64 bits: it is far above
// what the fp32 logits and the sigmoid leave open, and where a large bias leaves the keys
// coarser steps, two of those or more.  With logits of std 1.7 and a bias of 0.01 one token
// in 135 has its k-th and next key as close (8 of 384 experts; 6 of 128: one in 360), so
// that a call of 32 tokens pays the second look one time in five.
constexpr float kNear = 2e-5f;
__device__ __forceinline__ float near_of(float low) { return fmaxf(kNear, 0x1p-22f * fabsf(low)); }

// One token's view of the router.  Passed by value: a reference to the kernel's arguments
// that leaves the kernel would turn every access to them into a load from memory.
struct Row {
  const uint16_t* x;     // [H]
  const uint32_t* key;   // [E]
  const float* w;        // [E, H]
  const float* bias;     // [E]
  int H, E, k;
};

// x . w_e to about 2^-44 of its terms' sum (every lane gets it): products and sums as pairs
// of fp32 values, as 64-bit arithmetic runs at a sixtieth of the rate, with eight
// loads on their way.  A close choice holds up every CTA: at H 2048 by 34 us in 64
// bits with one load at a time, by 18 with eight, so by 6; at H 7168 by 13.
__device__ __noinline__ double logit64(Row a, int e, int lane) {
  constexpr int kLoads = 8;
  const float* w = a.w + (size_t)e * a.H;
  float sum = 0.f, rest = 0.f;
  auto add = [&](float x, float wt) {
    const float p = x * wt, t = __fadd_rn(sum, p), q = __fsub_rn(t, sum);
    rest += __fadd_rn(__fsub_rn(sum, __fsub_rn(t, q)), __fsub_rn(p, q)) + fmaf(x, wt, -p);
    sum = t;
  };
#pragma unroll 1
  for (int c0 = 4 * lane; c0 < a.H; c0 += 128 * kLoads) {
    float4 wv[kLoads];
    uint2 xv[kLoads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int c = c0 + 128 * l;
      wv[l] = make_float4(0.f, 0.f, 0.f, 0.f);
      xv[l] = make_uint2(0u, 0u);
      if (c < a.H) {
        wv[l] = __ldg(reinterpret_cast<const float4*>(w + c));
        xv[l] = __ldg(reinterpret_cast<const uint2*>(a.x + c));
      }
    }
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      add(__uint_as_float(xv[l].x << 16), wv[l].x);
      add(__uint_as_float(xv[l].x & 0xffff0000u), wv[l].y);
      add(__uint_as_float(xv[l].y << 16), wv[l].z);
      add(__uint_as_float(xv[l].y & 0xffff0000u), wv[l].w);
    }
  }
  // a sum beyond fp32 has no remainder
  double z = static_cast<double>(sum) + static_cast<double>(isfinite(rest) ? rest : 0.f);
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}

// Experts near the k-th key `low`, decided in 64 bits: lane j < k holds
// choice j in descending order of fp32 keys and gets its final one.  More than 16
// of them (a router with no preference) stay as fp32 has them.
__device__ __noinline__ int select_near(Row a, int lane, int mine, float low) {
  int mine_near = 0, n = 0, sure = 0;
  const float above = low + near_of(low), below = low - near_of(low);
#pragma unroll 1
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    const float r = e < a.E ? unordered(__ldcg(a.key + e)) : -INFINITY;
    sure += __popc(__ballot_sync(0xffffffffu, r > above));
    uint32_t near = __ballot_sync(0xffffffffu, r <= above && r >= below);
#pragma unroll 1
    for (; near; near &= near - 1, ++n)
      if (lane == (n & 31)) mine_near = e0 + __ffs(near) - 1;
    if (n > 16) return mine;
  }
  double key = 0.0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const double z = logit64(a, __shfl_sync(0xffffffffu, mine_near, i), lane);
    if (lane == i) key = z;
  }
  key = 1.0 / (1.0 + exp(-key)) + static_cast<double>(a.bias[mine_near]);
  if (key != key) key = -INFINITY;  // NaN ranks last
  int rank = 0;  // ids ascend with the lane
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const double v = __shfl_sync(0xffffffffu, key, i);
    rank += v > key || (v == key && i < lane);
  }
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int e = __shfl_sync(0xffffffffu, mine_near, i);
    const int to = sure + __shfl_sync(0xffffffffu, rank, i);
    if (to < a.k && lane == to) mine = e;
  }
  return mine;
}

// The k experts with the largest keys (equal: the lower id); one warp, lane j < k gets
// choice j.
__device__ __noinline__ int select_token(Row a, int lane) {
  constexpr int NPL = 16;  // experts of a lane whose keys stay in registers
  uint32_t key[NPL];
  uint64_t gone = 0;  // chosen ones among the others
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    key[i] = lane + 32 * i < a.E ? __ldcg(a.key + lane + 32 * i) : 0u;
  uint32_t low = 0, next = 0;
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j <= a.k && j < a.E; ++j) {  // one more than k: the best that stays out
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
#pragma unroll 1
    for (int i = NPL; lane + 32 * i < a.E; ++i) {
      const uint32_t v = gone >> i & 1u ? 0u : __ldcg(a.key + lane + 32 * i);
      if (v > best) {
        best = v;
        at = i;
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (j == a.k) {
      next = top;
      break;
    }
    low = top;
    const uint32_t e =
        __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(lane + 32 * at) : ~0u);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (static_cast<uint32_t>(lane + 32 * i) == e) key[i] = 0u;
    if ((e & 31u) == static_cast<uint32_t>(lane)) gone |= 1ull << (e >> 5);
    if (lane == j) mine = static_cast<int>(e);
  }
  const float f_low = unordered(low), f_next = next ? unordered(next) : -INFINITY;
  if (f_next > -INFINITY && f_low - f_next <= near_of(f_low)) mine = select_near(a, lane, mine, f_low);
  return mine;
}

// Chunks of a group: at most kFewGroups groups; more chunks to a group, up to a slot of
// weights, as long as every CTA has four units.  Fewer and larger groups leave CTAs
// without work at the end (32 tokens of 7168, 8 groups: 95 of 890 us), more and smaller
// ones have more sums to store.
__device__ __forceinline__ int group_chunks(const FewArgs& a, int chunks) {
  const int least = max(1, (chunks + kFewGroups - 1) / kFewGroups);
  const int whole = min(kFewColumns / a.I, chunks * (a.D / 32) / (4 * static_cast<int>(gridDim.x)));
  return max(least, whole);
}

__device__ __forceinline__ void mul_sync() {
  __syncwarp();  // whose lanes come from loops of different lengths
  asm volatile("bar.sync 1, %0;" ::"n"(kMul * 32) : "memory");
}

// The lists of a call, by the multiplying warps of every CTA: each token's choice,
// a mask of tokens for each expert, chunks of at most kFewChunk tokens in the
// order of the experts.  The sums' memory holds E words and E halves meanwhile.
__device__ __noinline__ void build_lists(int tid) {
  Context& cx = context();
  const FewArgs& a = cx.a;
  const Lists ls = lists_of(cx);
  // tokens of an expert, weights of the choices, first row of an expert, rows of the
  // choices (0xffff: none)
  uint32_t* mask = reinterpret_cast<uint32_t*>(few_smem + cx.sums_at);
  float* weight = reinterpret_cast<float*>(mask + a.E);
  uint16_t* base = reinterpret_cast<uint16_t*>(weight + a.T * a.k);
  uint16_t* row = base + a.E;
  const int lane = tid & 31, warp = tid >> 5, k = a.k, pairs = a.T * k;
#pragma unroll 1
  for (int e = tid; e < a.E; e += kMul * 32) mask[e] = 0u;
#pragma unroll 1
  for (int p = tid; p < pairs; p += kMul * 32) {
    ls.row_weight[p] = 0.f;
    if (!(p & 31)) ls.scaled[p >> 5] = 0u;
  }
  if (tid < kFewGroups) cx.in_group[tid] = 0u;
  if (tid < kFewTokens) cx.groups_of[tid] = 0u;
  mul_sync();
  // a warp a token, lane j its choice j
#pragma unroll 1
  for (int t = warp; t < a.T; t += kMul) {
    int e = 0;
    float w = 0.f;
    if (a.router_w) {
      e = select_token(Row{a.x + (size_t)t * a.H, a.keys + (size_t)t * a.E, a.router_w,
                           a.router_bias, a.H, a.E, k}, lane);
      if (lane < k) w = __ldcg(a.scores + (size_t)t * a.E + e);
      if (a.renorm) w = __fdividef(w, warp_sum(w) + 1e-20f);
    } else if (lane < k) {
      e = a.topk_idx[t * k + lane];
      w = a.topk_w[t * k + lane];
    }
    if (lane < k) {
      const bool ok = e >= 0 && e < a.E;
      if (ok) atomicOr(&mask[e], 1u << t);
      else record_status(a.status, MOE_ERR_INVALID);
      weight[t * k + lane] = w;
      row[t * k + lane] = ok ? static_cast<uint16_t>(e) : 0xffffu;
    }
  }
  mul_sync();
  // rows and chunks before a thread's experts, both below 2^16
  const int each = (a.E + kMul * 32 - 1) / (kMul * 32), e0 = tid * each;
  int sum = 0;
#pragma unroll 1
  for (int e = e0; e < min(e0 + each, a.E); ++e) {
    const int n = __popc(mask[e]);
    sum += n | (n + kFewChunk - 1) / kFewChunk << 16;
  }
  int before = -sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  before += sum;
  if (lane == 31) cx.scan[warp] = sum;
  mul_sync();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kMul; ++w) {
    const int v = cx.scan[w];
    if (w < warp) before += v;
    all += v;
  }
  const int chunks = all >> 16, per = group_chunks(a, chunks);
  int at = before >> 16, r = before & 0xffff;
#pragma unroll 1
  for (int e = e0; e < min(e0 + each, a.E); ++e) {
    base[e] = static_cast<uint16_t>(r);
#pragma unroll 1
    for (uint32_t m = mask[e]; m; ++at) {
      const uint32_t first = m & (0u - m);
      m ^= first;
      const uint32_t second = m & (0u - m);
      m ^= second;
      ls.tokens[at] = first | second;
      ls.expert[at] = static_cast<uint16_t>(e);
      ls.row0[at] = static_cast<uint16_t>(r);
      r += second ? 2 : 1;
      const int group = at / per;
      atomicOr(&cx.in_group[group], first | second);
      atomicOr(&cx.groups_of[__ffs(first) - 1], 1u << group);
      if (second) atomicOr(&cx.groups_of[__ffs(second) - 1], 1u << group);
    }
  }
  if (tid == 0) {
    cx.chunks = chunks;
    cx.per_group = per;
    cx.groups = (chunks + per - 1) / per;
    cx.units[kFewGateUp] = chunks * (a.I / 16);
    cx.units[kFewDown] = cx.groups * (a.D / 32);
  }
  mul_sync();
  if (tid == 0) mbar_arrive(&cx.listed);  // the copies may start
  if (tid < a.T) {  // an expert that a token lists twice counts twice
#pragma unroll 1
    for (int p = tid * k; p < (tid + 1) * k; ++p) {
      const int e = row[p];
      if (e != 0xffff) ls.row_weight[base[e] + __popc(mask[e] & ((1u << tid) - 1u))] += weight[p];
    }
  }
  if (chunks == 0) {  // no valid choice at all: no unit will write the output
#pragma unroll 1
    for (int i = blockIdx.x * kMul * 32 + tid; i < a.T * a.H; i += gridDim.x * kMul * 32)
      a.out[i] = 0;
  }
  mul_sync();
}
static_assert(kFewChunk == 2, "the lists take two tokens at a time");

__device__ __forceinline__ int nth_token(uint32_t tokens, int i) {
  return 31 - __clz(i ? tokens : tokens & (0u - tokens));
}

// --------------------------------------------------------------------- units

// A role's place in the ring: slot, parity of its use, slots passed.  (A division by the
// number of slots would cost more than the rest of a role's turn.)
struct Place {
  uint32_t s = 0, parity = 0, n = 0;
  __device__ __forceinline__ void next(int slots) {
    ++n;
    if (++s == static_cast<uint32_t>(slots)) {
      s = 0;
      parity ^= 1u;
    }
  }
};

// Where a row's scales of groups 2 g2, 2 g2 + 1 lie in its row block: rows of 128 bytes
// whose 16-byte pieces are swizzled as TMA writes them.
__device__ __forceinline__ uint32_t scale_at(int row, int g2) {
  return row * 128 + (((g2 >> 2) ^ (row & 7)) << 4) + (g2 & 3) * 4;
}

// -------------------------------------------------------------------- copies

__device__ __noinline__ void copy_weights(const FewMaps* maps, int lane) {
  Context& cx = context();
  const FewArgs& a = cx.a;
  const Ring ring = ring_of(cx);
  const Lists ls = lists_of(cx);
  const uint64_t once = evict_first();
  Place at;
  bool ok = true, known = false;
  const int fixed = cx.units[kFewLatDown] + cx.units[kFewSharedUp];
  // kAhead tickets at a time, so that a unit does not wait for its own.  One thread takes
  // them all: its atomics on one address follow one another in program order, so the CTA
  // works on its units in ticket order.
  int ticket = lane == 0 ? atomicAdd(a.counters, kAhead) : 0, later = ticket + 1;
#pragma unroll 1
  while (ok) {
    int u = __shfl_sync(0xffffffffu, ticket, 0);
    ticket = later;
    if (lane == 0) later = atomicAdd(a.counters, 1);
    if (u >= fixed && !known) {
      known = true;
      ok = wait_for<kRest>(&cx.listed, 0);
      if (!ok) break;
    }
    int kind = 0;
#pragma unroll 1
    while (kind < kFewKinds && u >= cx.units[kind]) u -= cx.units[kind++];
    Header h{kFewEnd, 0, 0, 0};
    int end = 1;  // segments h.which .. end - 1
    const bool pair = kind == kFewGateUp || kind == kFewSharedUp;  // two matrices
    const bool four = is_int4(kind);
    int K = 1;
    if (kind < kFewKinds) {
      const int each = cx.each[kind], q = u / each, r = u - q * each;
      const int tile = pair ? 16 : 32;
      h = Header{kind, 0, four ? q : r, (four ? r : q) * tile};
      end = h.which + 1;
      if (kind == kFewDown) {
        h.which *= cx.per_group;
        end = min(h.which + cx.per_group, cx.chunks);
      }
      K = length_of(a, kind);
    }
    const int w0 = kFirstMatrix >> 4 * kind & 15, w1 = w0 + pair;
    const int row1 = h.n0 + (pair ? 0 : 16);
    const int step = four ? C : C / 4, wide = four ? 256 : 64;  // columns of 128 bytes
#pragma unroll 1
    for (; ok && h.which < end; ++h.which) {
      const int rows = few_rows_of(kind);
      const int mat = four ? ls.expert[h.which] : 0;
      const int size = four ? __popc(ls.tokens[h.which]) : min(rows, a.T - h.which * rows);
#pragma unroll 1
      for (int k0 = 0; k0 < K; k0 += step, at.next(ring.n)) {
        const uint32_t s = at.s;
        if (static_cast<int>(at.n) == a.stall_at) {  // tests only
          ok = false;
          break;
        }
        ok = wait_for<kRest>(&ring.empty[s], at.parity ^ 1u);
        if (!ok) break;
        if (lane == 0) {
          const int cols = min(step, K - k0);
          const bool last = k0 + step >= K;
          uint64_t* bar = &ring.full[s];
          ring.header[s] = Header{h.kind | (last ? kLastSlot : 0) |
                                      (last && h.which + 1 == end ? kLastSegment : 0),
                                  size | cols << 16, h.which, h.n0};
          mbar_arrive(&ring.named[s]);
          // one thread issues all copies: operands that differ between lanes would
          // be taken up one lane after another (200 cycles each)
          const int pieces = cols / wide;
          const bool tail = four && cols % wide != 0;
          mbar_arrive_expect_tx(bar, kind == kFewKinds ? 0 : (pieces + tail) * 2 * 2048);
          if (kind < kFewKinds) {
            uint8_t* dst = ring.slot(s);
            if (pieces > 0) {
              const CUtensorMap* m = cols == step ? maps->full : maps->rest;
              copy_once_4d(dst, m + w0, bar, h.n0, k0 / wide, mat, once);
              copy_once_4d(dst + kWeightBytes / 2, m + w1, bar, row1, k0 / wide, mat, once);
            }
            if (tail) {
              dst += pieces * 2048;
              const int word = (k0 + pieces * wide) / 8;
              copy_once_3d(dst, maps->tail + w0, bar, word, h.n0, mat, once);
              copy_once_3d(dst + kWeightBytes / 2, maps->tail + w1, bar, word, row1, mat, once);
            }
          }
        }
        __syncwarp();
      }
    }
    if (kind == kFewKinds) break;
  }
  // whatever ended the loop, no copy is still on its way when the CTA leaves
  drain_ring(ring.full, at.n, ring.n, a.status);
}
static_assert(kAhead == 2, "ticket and later");

// Waits until counter `c` has reached `n`; its value, or -1 when the time ran out.
__device__ __noinline__ int wait_count(const int32_t* c, int n) {
  int v = load_acquire(c);
  if ((v & kFewCount) >= n) return v;
  const Waiter wt = waiter_of(context());
  const uint64_t t0 = global_timer_ns();
  while (((v = load_acquire(c)) & kFewCount) < n) {
    if (aborted(wt)) return -1;
    if (static_cast<int64_t>(global_timer_ns() - t0) > wt.limit_ns) {
      give_up(wt);
      return -1;
    }
    __nanosleep(64);
  }
  return v;
}

// Scales and rows of tokens.
__device__ __noinline__ void copy_rest(const FewMaps* maps, int lane) {
  Context& cx = context();
  const FewArgs& a = cx.a;
  const Ring ring = ring_of(cx);
  const Lists ls = lists_of(cx);
  const uint64_t once = evict_first();
  const bool lanes = !(a.tma_scale[0] && a.tma_scale[1]);  // every lane arrives on a slot
  int known = 0;         // chunks whose h is known to be complete
  uint32_t others = a.L > 0 ? 0u : 1u << kFewGateUp;  // kinds whose rows are
  others |= 1u << kFewLatDown | 1u << kFewSharedUp;
  bool u_scaled = false, scaled = false;  // u, the segment: units of their own
  bool any_scaled = false;                // or any chunk
  int i = 0;  // slot of the segment
  int mat = 0, K = 0;
  int64_t pitch = 0;
  const uint8_t* src = nullptr;
#pragma unroll 1
  for (Place at;; at.next(ring.n)) {
    const uint32_t s = at.s;
    if (!wait_for<kRest>(&ring.named[s], at.parity)) break;
    const Header h = ring.header[s];
    __syncwarp();  // lane 0's arrivals let the slot and its header be written again
    const int kind = h.kind & 255;
    const bool four = is_int4(kind), down = kind == kFewDown;
    uint64_t* bar = &ring.full[s];
    if (four && i == 0) {
      mat = ls.expert[h.which];
      K = down ? a.I : a.D;
      pitch = few_row_bytes(K);
      src = down ? a.h16 + ls.row0[h.which] * pitch : a.x16;
    }
    // scales, which wait for nothing
    if (!four) {
      if (lanes || lane == 0) mbar_arrive(bar);
    } else {
      const int row1 = h.n0 + (down ? 16 : 0);
      uint8_t* dst = ring.scales(s);
      if (a.tma_scale[down] == kScalesDense) {
        // 16 whole rows at a time, one behind the other
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, 2 * K);
          const int N = down ? a.D : a.I, per_row = K / kGroup;
          const int64_t at = ((int64_t)mat * N + h.n0) * per_row;
          bulk_g2s(dst, a.scale[down ? 2 : 0] + at, K, bar);
          bulk_g2s(dst + kScaleBytes / 2, a.scale[down ? 2 : 1] + at + (down ? 16 * per_row : 0), K,
                   bar);
        } else if (lanes) {
          mbar_arrive(bar);
        }
      } else if (a.tma_scale[down]) {
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, kScaleBytes);
          const CUtensorMap* m = maps->scale + (down ? kFewDownW : kFewGateW);
          copy_once_3d(dst, m, bar, i * (C / kGroup), h.n0, mat, once);
          copy_once_3d(dst + kScaleBytes / 2, m + !down, bar, i * (C / kGroup), row1, mat, once);
        } else if (lanes) {
          mbar_arrive(bar);
        }
      } else {
        // rows of K / 16 bytes, not 16-byte aligned: 4 bytes (two groups) a lane, a row at
        // a time (D 5696, one token, 4 experts: 30 us; with the rows' pieces dealt out over
        // the lanes, which takes a division for each, 39)
        const int N = down ? a.D : a.I;
        const size_t row_bytes = K / 16;
        if (lane < h.cols() / 64) {
#pragma unroll 1
          for (int b = 0; b < 2; ++b) {
            const uint8_t* from = reinterpret_cast<const uint8_t*>(a.scale[down ? 2 : b]) +
                                  ((size_t)mat * N + (b ? row1 : h.n0)) * row_bytes + i * (C / 16) +
                                  4 * lane;
#pragma unroll 4
            for (int r = 0; r < 16; ++r, from += row_bytes)
              cp_async_4(dst + b * (kScaleBytes / 2) + scale_at(r, lane), from);
          }
        }
        cp_async_arrive_noinc(bar);
      }
    }
    if (kind == kFewEnd) {
      if (lane == 0) mbar_arrive(bar);
      return;
    }
    // the rows this segment reads have to be there
    if (i == 0 && (down ? h.which >= known : !(others >> kind & 1u))) {
      const int32_t* c = a.counters + (down ? kFewFixed + h.which
                                            : kind == kFewGateUp ? 1 : kind == kFewSharedDown ? 2 : 3);
      const int whole = few_chunks(a.T, kFewRows);
      const int n = down ? a.I / 16
                         : kind == kFewGateUp ? a.L / 32 * whole
                                              : kind == kFewSharedDown ? a.S / 16 * whole : a.L / 32;
      const int count = wait_count(c, n);
      if (down) {
        // and what a look at the next chunks shows at the same time
        const int chunk = h.which + lane, v = chunk < a.T * a.k ? load_acquire(c + lane) : 0;
        const bool there = (v & kFewCount) >= n;
        const uint32_t done = __ballot_sync(0xffffffffu, there);
        known = h.which + (~done ? __ffs(~done) - 1 : 32);
        if (there && (v & kFewScaled)) {
          any_scaled = true;
          atomicOr(&ls.scaled[chunk >> 5], 1u << (chunk & 31));
        }
      } else {
        others |= 1u << kind;
        if (kind == kFewGateUp && (count & kFewScaled)) u_scaled = any_scaled = true;
      }
      any_scaled = __any_sync(0xffffffffu, any_scaled);
      if (!__all_sync(0xffffffffu, count >= 0)) break;
      __syncwarp();  // what one lane has seen holds for all
      // written through the generic proxy, read by copies
      asm volatile("fence.proxy.async.global;" ::: "memory");
    }
    if (lane == 0) {
      uint8_t* dst = ring.rows(s);
      if (four) {
        const uint32_t tokens = ls.tokens[h.which];
        if (any_scaled) {
          if (i == 0) scaled = down ? ls.scaled[h.which >> 5] >> (h.which & 31) & 1u : u_scaled;
          if (scaled) ring.header[s].kind = h.kind | kScaled | i << kSlotShift;
        }
        mbar_arrive_expect_tx(bar, h.rows() * kFewBlock);
        const uint8_t* from = src + i * kFewBlock;
#pragma unroll 1
        for (int r = 0; r < h.rows(); ++r)
          bulk_g2s(dst + r * kPitch4, from + (down ? r : nth_token(tokens, r)) * pitch, kFewBlock,
                   bar);
      } else {
        const int most = few_rows_of(kind), bytes = min(a.T, most) * (C / 2);
        const int parts = most == kFewRows ? 1 : 2;
        const CUtensorMap* m = maps->rows + (parts == 1 ? 0 : kind == kFewSharedDown ? 1 : 2);
        mbar_arrive_expect_tx(bar, parts * bytes);
#pragma unroll 1
        for (int p = 0; p < parts; ++p)
          tma_g2s_4d(dst + p * bytes, m, bar, 0, h.which * most, i * (C / 256), p);
      }
    }
    __syncwarp();
    i = (h.kind & kLastSlot) ? 0 : i + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // a wait that ran out: nothing stays on its way
}

// ------------------------------------------------------------------ products

// Row of a block that lane (g, t) reads as rows g and (+ 8) g + 8 of an MMA: so the 8
// lanes of a 128-byte shared-memory access meet both halves of the swizzle.
__device__ __forceinline__ int row_of(int g) { return g >> 1 | (g & 1) << 2; }

// 128 columns (4 groups) of both row blocks and of up to 2 PAIRS tokens.
//
// A lane's 16-byte load of a row is one whole group, and the four lanes of a quad hold
// four groups.  An MMA adds over the quad, so the groups are kept apart on the
// other side: column n = 4 (token of the pair) + group of the B operand holds
// that token's values of that group, and zeros where the quad's other lanes
// hold another group.  Eight MMAs then give the partial sums of 16 rows, 4
// groups and 2 tokens, 8 of them in each accumulator column, with the words
// used as they were loaded and 4 scale products for 64 weights a lane.
//
// Columns of tokens that are not there hold whatever the slot does: no column reaches
// another.  Lanes that are off keep the zeros they were given.
struct Lane {
  int g, t, r;
  bool on;  // holds the B operand of its column's group
  __device__ __forceinline__ explicit Lane(int lane)
      : g(lane >> 2), t(lane & 3), r(row_of(lane >> 2)), on((lane >> 2 & 3) == (lane & 3)) {}
};

// One step: adds to acc[block][0, 1] (rows g and g + 8).  w, x, start, scale: where the lane
// reads; rows8: bytes between the scales of 8 rows; there: the lane's two columns are of
// groups that the row has.
__device__ __forceinline__ void multiply4(const uint8_t* w, const uint8_t* x, const uint8_t* start,
                                          const uint8_t* scale, int rows8, bool there, bool on,
                                          const Magic& magic, uint4 (&v)[4], float (&acc)[2][4]) {
  if (on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const uint4*>(x)[i];
  }
  // two start values (16 columns each) of groups 2 (t & 1) and + 1, token t >> 1
  const float4 s = *reinterpret_cast<const float4*>(start);
  const float start0 = s.x + s.y, start1 = s.z + s.w;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint4 q0 = *reinterpret_cast<const uint4*>(w + b * (kWeightBytes / 2));
    const uint4 q8 = *reinterpret_cast<const uint4*>(w + b * (kWeightBytes / 2) + 1024);
    const uint32_t w0[4] = {q0.x, q0.y, q0.z, q0.w}, w8[4] = {q8.x, q8.y, q8.z, q8.w};
    const uint32_t s0 = *reinterpret_cast<const uint32_t*>(scale + b * (kScaleBytes / 2));
    const uint32_t s8 = *reinterpret_cast<const uint32_t*>(scale + b * (kScaleBytes / 2) + rows8);
    float c[4] = {start0, start1, start0, start1};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo[4], hi[4];
      nibbles(w0[i], magic, lo);
      nibbles(w8[i], magic, hi);
      mma_f16(c, lo[0], hi[0], lo[1], hi[1], v[i].x, v[i].y, c[0], c[1], c[2], c[3]);
      mma_f16(c, lo[2], hi[2], lo[3], hi[3], v[i].z, v[i].w, c[0], c[1], c[2], c[3]);
    }
    if (there) {
      acc[b][0] = fmaf(__uint_as_float(s0 & 0xffff0000u), c[1],
                       fmaf(__uint_as_float(s0 << 16), c[0], acc[b][0]));
      acc[b][1] = fmaf(__uint_as_float(s8 & 0xffff0000u), c[3],
                       fmaf(__uint_as_float(s8 << 16), c[2], acc[b][1]));
    }
  }
}

// A multiplying warp's place in the ring and among the buffers of the finishing warps.
struct Turn {
  Place at;
  int buf = 0;         // the finishing warp of this unit
  uint32_t taken = 0;  // parity of its buffer, one bit a warp
  static_assert(kMaxSlots == 8 && kFinish == 2, "packing");
  __device__ __forceinline__ explicit Turn(int packed) {  // 0: the first
    at.s = packed & 7;
    at.parity = packed >> 3 & 1;
    buf = packed >> 4 & 1;
    taken = packed >> 5 & 3;
  }
  static __device__ __forceinline__ int pack(const Place& at, int buf, uint32_t taken) {
    return at.s | at.parity << 3 | buf << 4 | taken << 5;
  }
};

// A warp's steps through the slots of a segment in which 16 columns of a row have a unit of
// their own, from the slot where multiply() stopped, which has been waited for; where that
// goes on, or -1.  The products of a group's halves are made apart, and together too: with
// one unit for both halves a token gets the bits that it gets from multiply4, so that they
// do not depend on the other token.  Few calls come here, and the units come from L2 (one
// token of 8 experts, 7168 x 2048, all of h below 2^-11: 63 us, of ordinary size 48).
__device__ __noinline__ int multiply_scaled(int warp, int lane, int from) {
  Context& cx = context();
  const FewArgs& a = cx.a;
  const Ring ring = ring_of(cx);
  const Sums sums = sums_of(cx);
  const Lists ls = lists_of(cx);
  Turn m(from);
  const Lane l(lane);
  const Magic magic;
  const int token = l.t >> 1, room = min(a.T, kFewChunk) - 1;
  float acc[2][2] = {};  // [block][row g, g + 8]
#pragma unroll 1
  for (;;) {
    const Header h = ring.header[m.at.s];
    const uint8_t* slot = ring.slot(m.at.s);
    const bool down = (h.kind & (kScaled - 1)) == kFewDown;
    const int cols = h.cols();
    const float* units = nullptr;  // of the lane's two groups
    if (token < h.rows()) {
      const int row = down ? ls.row0[h.which] + token : nth_token(ls.tokens[h.which], token);
      units = (down ? a.h_unit + (size_t)row * (a.I / 16) : a.u_unit + (size_t)row * (a.L / 16)) +
              (h.kind >> kSlotShift) * (C / 16) + (l.t & 1) * 4;
    }
    const uint8_t* rows = slot + kWeightBytes + kScaleBytes;
    const bool dense = a.tma_scale[down] == kScalesDense;
#pragma unroll 1
    for (int c0 = 128 * warp; c0 < cols; c0 += 128 * kMul) {
      const bool there = c0 + 128 <= cols || !(l.t & 1);
      const float4 u = there && units ? __ldcg(reinterpret_cast<const float4*>(units + c0 / 16))
                                      : make_float4(1.f, 1.f, 1.f, 1.f);
      uint4 v[4];
      const uint8_t* x = rows + min(l.g >> 2, room) * kPitch4 + c0 * 2 + l.t * 64;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = l.on ? reinterpret_cast<const uint4*>(x)[i] : make_uint4(0u, 0u, 0u, 0u);
      const float4 start = *reinterpret_cast<const float4*>(
          rows + min(token, room) * kPitch4 + kStarts + c0 / 4 + (l.t & 1) * 16);
      const int piece = c0 / 256 * 2048 + ((((c0 / 128 & 1) << 2 | l.t) ^ (l.r & 7)) << 4);
      const int g2 = c0 / 64 + (l.t & 1);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint8_t* w = slot + b * (kWeightBytes / 2) + piece + l.r * 128;
        const uint8_t* scale = slot + kWeightBytes + b * (kScaleBytes / 2);
        const uint4 q0 = *reinterpret_cast<const uint4*>(w);
        const uint4 q8 = *reinterpret_cast<const uint4*>(w + 1024);
        const uint32_t w0[4] = {q0.x, q0.y, q0.z, q0.w}, w8[4] = {q8.x, q8.y, q8.z, q8.w};
        float all[4] = {start.x + start.y, start.z + start.w, start.x + start.y, start.z + start.w};
        float half[2][4] = {{start.x, start.z, start.x, start.z}, {start.y, start.w, start.y, start.w}};
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t lo[4], hi[4];
          nibbles(w0[i], magic, lo);
          nibbles(w8[i], magic, hi);
          float(&c)[4] = half[i >> 1];
          mma_f16(all, lo[0], hi[0], lo[1], hi[1], v[i].x, v[i].y, all[0], all[1], all[2], all[3]);
          mma_f16(all, lo[2], hi[2], lo[3], hi[3], v[i].z, v[i].w, all[0], all[1], all[2], all[3]);
          mma_f16(c, lo[0], hi[0], lo[1], hi[1], v[i].x, v[i].y, c[0], c[1], c[2], c[3]);
          mma_f16(c, lo[2], hi[2], lo[3], hi[3], v[i].z, v[i].w, c[0], c[1], c[2], c[3]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float first = u.x == u.y ? u.x * all[2 * r]
                                         : fmaf(u.x, half[0][2 * r], u.y * half[1][2 * r]);
          const float second = u.z == u.w ? u.z * all[2 * r + 1]
                                          : fmaf(u.z, half[0][2 * r + 1], u.w * half[1][2 * r + 1]);
          const uint32_t sc = *reinterpret_cast<const uint32_t*>(
              dense ? scale + (l.r + 8 * r) * (cols >> 4) + g2 * 4 : scale + scale_at(l.r + 8 * r, g2));
          if (there)
            acc[b][r] = fmaf(__uint_as_float(sc & 0xffff0000u), second,
                             fmaf(__uint_as_float(sc << 16), first, acc[b][r]));
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[m.at.s]);
    m.at.next(ring.n);
    if (h.kind & kLastSlot) {
      if (!wait_for(&sums.empty[m.buf], (m.taken >> m.buf & 1u) ^ 1u)) return -1;
      m.taken ^= 1u << m.buf;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int r = 0; r < 2; ++r) acc[b][r] += __shfl_xor_sync(0xffffffffu, acc[b][r], 1);
        if (!(l.t & 1) && token < h.rows()) {
          float* p = sums.at(m.buf, warp, b, token);
          p[l.r] = acc[b][0];
          p[l.r + 8] = acc[b][1];
        }
      }
      if (warp == 0 && lane == 0) {
        sums.header[m.buf] = h;
        sums.header[m.buf].kind = h.kind & ~kScaled;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums.full[m.buf]);
      if (h.kind & kLastSegment) m.buf ^= 1;
      return Turn::pack(m.at, m.buf, m.taken);
    }
    if (!wait_for(&ring.full[m.at.s], m.at.parity)) return -1;
  }
}

// Columns of bf16 weights, 16 at a time, and up to 8 tokens (in one or two parts).
__device__ __forceinline__ void multiply16(const uint8_t* slot, int cols, int tokens, int planes,
                                           int warp, int lane, const Lane& l, float (&acc)[2][4]) {
  const int li = lane & 7;
  // of the warp's first 16 columns; the next ones lie two pieces on, at the same place in them
  uint32_t w = smem_u32(slot) + (warp >> 2) * 2048 + ((lane & 8) + li) * 128 +
               ((((warp & 3) << 1 | lane >> 4) ^ li) << 4);
  // columns of tokens that are not there repeat the last one's
  int at = (warp >> 2) * tokens + min(l.g, tokens - 1);
  const uint8_t* rows = slot + kWeightBytes + kScaleBytes + l.t * 4;
  const int piece = (warp & 3) << 1;
#pragma unroll 1
  for (int c0 = 16 * warp; c0 < cols; c0 += 16 * kMul, w += kMul / 4 * 2048, at += kMul / 4 * tokens) {
    uint32_t wr[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) ldsm4(w + b * (kWeightBytes / 2), wr[b]);
    const uint8_t* x = rows + at * 128 + ((piece ^ (at & 6)) << 4);
    const int odd = (at & 1) << 4;
#pragma unroll
    for (int plane = 0; plane < 2; ++plane, x += tokens * (C / 2)) {
      if (plane == planes) break;
      const uint32_t b0 = *reinterpret_cast<const uint32_t*>(x + odd);
      const uint32_t b1 = *reinterpret_cast<const uint32_t*>(x + (odd ^ 16));
#pragma unroll
      for (int b = 0; b < 2; ++b) mma_bf16(acc[b], wr[b], b0, b1);
    }
  }
}

// Products of all slots; stops at a segment of multiply_scaled, and returns where, or -1.  (A
// call from inside the loop takes registers from it: 32 tokens 905 us, without 815 to 825.)
__device__ __noinline__ int multiply(int warp, int lane, int from) {
  Context& cx = context();
  const FewArgs& a = cx.a;
  const Ring ring = ring_of(cx);
  const Sums sums = sums_of(cx);
  // int4 units: [block][row g, g + 8], the groups of lane t odd and even still apart;
  // bf16 units: [block] MMA accumulator
  float acc[2][4] = {};
  const Magic magic;
  const Lane l(lane);
  const int room = min(a.T, kFewChunk) - 1, slots = ring.n;
  // Where the lane reads in a slot for its warp's first step, columns 128 warp and on; what
  // can be known before the slots: eight instructions more in a step are 8 % of a call.
  const int w_at =
      (warp >> 1) * 2048 + l.r * 128 + ((((warp & 1) << 2 | l.t) ^ (l.r & 7)) << 4);
  const int scales_at = kWeightBytes + static_cast<int>(scale_at(l.r, 2 * warp + (l.t & 1)));
  const int x_at =
      kWeightBytes + kScaleBytes + min(l.g >> 2, room) * kPitch4 + warp * 256 + l.t * 64;
  const int start_at = kWeightBytes + kScaleBytes + min(l.t >> 1, room) * kPitch4 + kStarts +
                       warp * 32 + (l.t & 1) * 16;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  Place at;
  int buf = 0;
  uint32_t taken = 0;
  if (from) {
    const Turn m(from);
    at = m.at;
    buf = m.buf;
    taken = m.taken;
  }
  for (;; at.next(slots)) {
    const uint32_t s = at.s;
    if (!wait_for(&ring.full[s], at.parity)) return -1;
    const Header h = ring.header[s];
    const int kind = h.kind & 255;
    const uint8_t* slot = ring.slot(s);
    if (is_int4(kind)) {
      const int cols = h.cols();
      const uint8_t *w = slot + w_at, *x = slot + x_at, *start = slot + start_at;
      const bool dense = a.tma_scale[kind - kFewGateUp] == kScalesDense;
      int scale = scales_at, rows8 = 1024;
      if (dense) {  // rows of cols / 16 bytes
        scale = kWeightBytes + l.r * (cols >> 4) + 8 * warp + (l.t & 1) * 4;
        rows8 = cols >> 1;
      }
#pragma unroll 1
      for (int c0 = 128 * warp; c0 < cols; c0 += 128 * kMul) {
        // the last step of a row may be half: its upper two groups add nothing
        multiply4(w, x, start, slot + scale, rows8, c0 + 128 <= cols || !(l.t & 1), l.on, magic, v,
                  acc);
        w += kMul / 2 * 2048;
        x += kMul * 256;
        start += kMul * 32;
        scale = dense ? scale + 8 * kMul : scale ^ 64;  // four pieces on, which are swizzled
      }
    } else {
      if (kind == kFewEnd) break;
      if (kind & kScaled) return Turn::pack(at, buf, taken);  // the first slot of a segment
      const int most = few_rows_of(kind);
      multiply16(slot, h.cols(), min(a.T, most), most == kFewRows ? 1 : 2, warp, lane, l, acc);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[s]);
    if (h.kind & kLastSlot) {
      if (!wait_for(&sums.empty[buf], (taken >> buf & 1u) ^ 1u)) return -1;
      taken ^= 1u << buf;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (is_int4(kind)) {
          acc[b][0] += __shfl_xor_sync(0xffffffffu, acc[b][0], 1);
          acc[b][1] += __shfl_xor_sync(0xffffffffu, acc[b][1], 1);
          if (!(l.t & 1) && (l.t >> 1) < h.rows()) {
            float* p = sums.at(buf, warp, b, l.t >> 1);
            p[l.r] = acc[b][0];
            p[l.r + 8] = acc[b][1];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (2 * l.t + i < h.rows()) {
              float* p = sums.at(buf, warp, b, 2 * l.t + i);
              p[l.g] = acc[b][i];
              p[l.g + 8] = acc[b][2 + i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;
      }
      if (warp == 0 && lane == 0) sums.header[buf] = h;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums.full[buf]);
      if (h.kind & kLastSegment) buf = (buf + 1) % kFinish;
    }
  }
  for (buf = 0; buf < kFinish; ++buf) {  // tell the finishing warps
    if (!wait_for(&sums.empty[buf], (taken >> buf & 1u) ^ 1u)) return -1;
    if (warp == 0 && lane == 0) sums.header[buf].kind = kFewEnd;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sums.full[buf]);
  }
  return -1;
}

// ----------------------------------------------------------------- finishing

// Adds one to a counter after the warp's stores; with `scaled` its bit is set first, so that
// whoever sees the count sees that too.
__device__ __forceinline__ void count_done(int32_t* c, int lane, bool scaled = false) {
  __syncwarp();
  if (lane == 0) {
    if (scaled) atomicOr(c, kFewScaled);
    add_release(c, 1);
  }
}

// 32 columns from n0 on of every token: the groups' sums, in order, whichever order they
// were computed in, and the shared expert's; for the latent path as two bf16 parts
// with the gain, and their squares summed over the 32 columns.  Eight lanes have a token,
// four columns each: what the last unit of a call is waited for by (32 tokens two at a
// time, a column a lane: 28 us at the end of a call, so 15; 16 tokens: 12 and 8).
__device__ __noinline__ void combine(int n0, int lane) {
  Context& cx = context();
  const FewArgs& a = cx.a;
  const bool latent = a.L > 0;
  const int n = n0 + 4 * (lane & 7);
  constexpr int kLoads = 8;  // on their way at a time
#pragma unroll 1
  for (int t0 = 0; t0 < a.T; t0 += 4) {
    const int t = t0 + (lane >> 3);
    const bool there = t < a.T;
    uint32_t m = there ? cx.groups_of[t] : 0u;
    const float* y = a.y + (size_t)t * a.D + n;
    const size_t next = (size_t)a.T * a.D;  // group
    float4 shared = make_float4(0.f, 0.f, 0.f, 0.f), sum = shared;
    if (there && !latent && a.S > 0)
      shared = __ldcg(reinterpret_cast<const float4*>(a.ys + (size_t)t * a.H + n));
#pragma unroll 1
    do {
      float4 v[kLoads];
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        v[l] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m) v[l] = __ldcg(reinterpret_cast<const float4*>(y + (__ffs(m) - 1) * next));
        m &= m - 1;
      }
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        sum.x += v[l].x;
        sum.y += v[l].y;
        sum.z += v[l].z;
        sum.w += v[l].w;
      }
    } while (__any_sync(0xffffffffu, m != 0u));
    float r[4] = {sum.x + shared.x, sum.y + shared.y, sum.z + shared.z, sum.w + shared.w};
    if (!latent) {
      if (there)
        *reinterpret_cast<uint2*>(a.out + (size_t)t * a.H + n) =
            make_uint2(f32_to_bf16_bits(r[0]) | static_cast<uint32_t>(f32_to_bf16_bits(r[1])) << 16,
                       f32_to_bf16_bits(r[2]) | static_cast<uint32_t>(f32_to_bf16_bits(r[3])) << 16);
      continue;
    }
    float q = fmaf(r[0], r[0], fmaf(r[1], r[1], fmaf(r[2], r[2], r[3] * r[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    if (!there) continue;
    if (!(lane & 7)) a.ssq[(size_t)(n0 / 32) * a.T + t] = q;
    uint32_t high[4], low[4];  // 16 bits of significand
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (a.norm) r[i] *= bf16_bits_to_f32(__ldg(a.lat_norm + n + i));
      high[i] = f32_to_bf16_bits(r[i]);
      low[i] = f32_to_bf16_bits(r[i] - bf16_bits_to_f32(static_cast<uint16_t>(high[i])));
    }
    uint16_t* z = a.z + (size_t)t * a.L + n;
    *reinterpret_cast<uint2*>(z) = make_uint2(high[0] | high[1] << 16, high[2] | high[3] << 16);
    *reinterpret_cast<uint2*>(z + (size_t)a.T * a.L) =
        make_uint2(low[0] | low[1] << 16, low[2] | low[3] << 16);
  }
  if (latent) count_done(a.counters + 3, lane);
}

// What the rows of the latent layer's norm are divided by: lane t gets token t's.
__device__ __noinline__ float norms(int lane) {
  const FewArgs& a = context().a;
  int lanes = 1;  // of a row of sums, a power of two: lane t has token t % lanes
  while (lanes < a.T) lanes *= 2;
  const int t = lane & (lanes - 1), step = 32 / lanes;
  constexpr int kLoads = 8;
  float q = 0.f;
#pragma unroll 1
  for (int j = lane / lanes; j < a.L / 32; j += kLoads * step) {
    float v[kLoads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l)
      v[l] = t < a.T && j + l * step < a.L / 32 ? __ldcg(a.ssq + (size_t)(j + l * step) * a.T + t) : 0.f;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) q += v[l];
  }
#pragma unroll 1
  for (int o = lanes; o < 32; o <<= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  return rsqrtf(q / static_cast<float>(a.L) + a.eps);
}

__device__ __noinline__ void finish(int buf, int lane) {
  Context& cx = context();
  const FewArgs& a = cx.a;
  const Sums sums = sums_of(cx);
  const Lists ls = lists_of(cx);
  const int halves = few_chunks(a.T, kFewRows / 2);
  int32_t* tile_done = a.counters + kFewFixed + a.T * a.k;
  int32_t* out_done = tile_done + a.D / 32;
  const int r16 = lane & 15, half = lane >> 4;
  float* unit = sums.unit + buf * a.T * 32 + lane;  // a token's 32 columns
  bool first = true;  // segment of a down projection's unit
  bool normed = false;
  float norm = 1.f;  // of token `lane`
  const float x_unit = a.L == 0 && lane < a.T ? __ldcg(a.x_unit + lane) : 1.f;  // of token `lane`
#pragma unroll 1
  for (uint32_t n = 0;; ++n) {
    if (!wait_for<kRest>(&sums.full[buf], n & 1u)) return;
    const Header h = sums.header[buf];
    const int kind = h.kind & 255;
    if (kind == kFewEnd) return;
    const bool four = is_int4(kind), pair = kind == kFewGateUp || kind == kFewSharedUp;
    const int c = h.n0 + (pair ? r16 : lane);
    const int token0 = h.which * few_rows_of(kind);
    const uint32_t tokens = four ? ls.tokens[h.which] : 0u;
    const int row0 = four ? ls.row0[h.which] : 0;
    if (kind == kFewLatUp && a.norm && !normed) {  // every sum of squares is there by now
      norm = norms(lane);
      normed = true;
    }
    if (kind == kFewDown && first) {
#pragma unroll 1
      for (int t = 0; t < a.T; ++t) unit[t * 32] = 0.f;
    }
    bool scaled = false;  // columns with a unit of their own
#pragma unroll 1
    for (int i = 0; i < h.rows(); ++i) {
      const int t = four ? nth_token(tokens, i) : token0 + i;
      float v = 0.f;
      const float* part = sums.at(buf, 0, half, i) + r16;
#pragma unroll
      for (int w = 0; w < kMul; ++w) v += part[w * 2 * sums.tokens * 16];
      const float other = __shfl_xor_sync(0xffffffffu, v, 16);  // of lanes below 16: up
      if (pair || kind == kFewLatDown) {
        // h, or u
        if (pair) {
          float g = v, u = other;
          if (kind == kFewGateUp && a.L == 0) {
            const float scale = __shfl_sync(0xffffffffu, x_unit, t);
            g *= scale;
            u *= scale;
          }
          v = g / (1.0f + expf(-g)) * u;
        }
        if (kind == kFewSharedUp) {
          // two bf16 parts: 16 bits of significand
          if (half == 0) {
            uint16_t* p = a.hs + (size_t)t * a.S + c;
            const uint16_t high = f32_to_bf16_bits(v);
            p[0] = high;
            p[(size_t)a.T * a.S] = f32_to_bf16_bits(v - bf16_bits_to_f32(high));
          }
        } else {
          // fp16 in pair order, and the unit and the start value of each 16 columns
          const bool mine = !pair || half == 0;
          if (mine && !(fabsf(v) <= 65504.0f)) record_status(a.status, MOE_ERR_UNSUPPORTED);
          const uint32_t top =
              __reduce_max_sync(0xffffffffu, mine ? __float_as_uint(fabsf(v)) : 0u);
          float by_one = 1.f;
          if (top > 0u && top < __float_as_uint(kFewSmallest)) {
            const uint32_t up = min(127u + 14u + 127u - (top >> 23), 253u);
            v *= __uint_as_float(up << 23);
            by_one = __uint_as_float((254u - up) << 23);
            scaled = true;
          }
          float* units = pair ? a.h_unit + (size_t)(row0 + i) * (a.I / 16)
                              : a.u_unit + (size_t)t * (a.L / 16);
          if (mine && r16 == 0) units[c / 16] = by_one;
          const __half f = __float2half_rn(v);
          uint8_t* row = pair ? a.h16 + (row0 + i) * few_row_bytes(a.I)
                              : a.x16 + t * few_row_bytes(a.L);
          if (mine)
            *reinterpret_cast<uint16_t*>(row + few_value_at(pair_pos(c))) = __half_as_ushort(f);
          float s = start_of(__half2float(f), c);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (mine && r16 == 0) *reinterpret_cast<float*>(row + few_start_at(c)) = s;
        }
      } else if (kind == kFewDown) {
        unit[t * 32] = fmaf(ls.row_weight[row0 + i], v, unit[t * 32]);
      } else {
        const size_t at = (size_t)t * a.H + c;
        if (kind == kFewLatUp) {
          if (a.norm) v *= __shfl_sync(0xffffffffu, norm, t);
          if (a.S == 0)
            a.out[at] = f32_to_bf16_bits(v);
          else
            a.yl[at] = v;
        } else {
          a.ys[at] = v;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sums.empty[buf]);  // the buffer has been read
    if (pair || kind == kFewLatDown) {
      count_done(a.counters + (kind == kFewGateUp ? kFewFixed + h.which : kind == kFewLatDown ? 1 : 2),
                 lane, scaled);
      continue;
    }
    if (kind == kFewDown) {
      first = (h.kind & kLastSegment) != 0;
      if (!first) continue;
      const int group = h.which / cx.per_group;
#pragma unroll 1
      for (uint32_t m = cx.in_group[group]; m; m &= m - 1) {
        const int t = __ffs(m) - 1;
        a.y[((size_t)group * a.T + t) * a.D + c] = unit[t * 32];
      }
    }
    if (kind == kFewLatUp && a.S == 0) continue;
    // whoever brings the last contribution to 32 columns reads them all
    const bool whole = a.L > 0 && kind != kFewDown;  // a tile of the latent layer's output
    int32_t* done = whole ? out_done + h.n0 / 32 * halves + h.which : tile_done + h.n0 / 32;
    const int all = whole ? 2
                          : cx.groups + (a.S > 0 && a.L == 0 ? halves : 0);
    __syncwarp();
    int old = 0;
    if (lane == 0) old = add_acq_rel(done, 1);
    old = __shfl_sync(0xffffffffu, old, 0);
    if (old != all - 1) continue;
    __threadfence();
    if (!whole) {
      combine(h.n0, lane);
      continue;
    }
#pragma unroll 1
    for (int i = 0; i < h.rows(); ++i) {
      const size_t at = (size_t)(token0 + i) * a.H + c;
      a.out[at] = f32_to_bf16_bits(__ldcg(a.yl + at) + __ldcg(a.ys + at));
    }
  }
}

// -------------------------------------------------------------------- kernel

// Offsets into a CTA's shared memory, behind the context.
struct Layout {
  int slot, sums, unit, lists;
  __host__ __device__ __forceinline__ explicit Layout(const FewArgs& a) {
    slot = slot_bytes(rows_bytes(a));
    sums = sums_bytes(a);
    unit = kFinish * a.T * 32 * 4;
    const int pairs = a.T * a.k;
    lists = (12 * pairs + (pairs + 31) / 32 * 4 + 15) / 16 * 16;
  }
  __host__ __device__ __forceinline__ int rest() const {
    return static_cast<int>(sizeof(Context)) + sums + unit + lists;
  }
};

__global__ void __launch_bounds__(kThreads, kCtas)
    few_kernel(const __grid_constant__ FewMaps maps, const FewArgs args) {
  Context& cx = context();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    const Layout lay(args);
    cx.a = args;
    // units in ticket order, as tiles of chunks of tokens, or chunks of experts by tiles
    const int whole = few_chunks(args.T, kFewRows), half = few_chunks(args.T, kFewRows / 2);
    cx.each[kFewLatDown] = cx.each[kFewSharedUp] = whole;
    cx.each[kFewSharedDown] = cx.each[kFewLatUp] = half;
    cx.each[kFewGateUp] = args.I / 16;
    cx.each[kFewDown] = args.D / 32;
    cx.units[kFewLatDown] = args.L / 32 * whole;
    cx.units[kFewSharedUp] = args.S / 16 * whole;
    cx.units[kFewGateUp] = cx.units[kFewDown] = 0;  // when the lists are made
    cx.units[kFewSharedDown] = args.S > 0 ? args.H / 32 * half : 0;
    cx.units[kFewLatUp] = args.L > 0 ? args.H / 32 * half : 0;
    cx.slot = lay.slot;
    cx.sums_at = sizeof(Context);
    cx.unit_at = cx.sums_at + lay.sums;
    cx.lists_at = cx.unit_at + lay.unit;
    const int end = lay.rest();
    cx.ring_at = end + (-(smem_u32(few_smem) + end) & 1023u);
    for (int s = 0; s < args.stages; ++s) {
      // the announcements of the weights, the rows and the scales (or of all its lanes)
      mbar_init(&cx.full[s], 2 + (args.tma_scale[0] && args.tma_scale[1] ? 1 : 32));
      mbar_init(&cx.empty[s], kMul);
      mbar_init(&cx.named[s], 1);
    }
    for (int b = 0; b < kFinish; ++b) {
      mbar_init(&cx.sum_full[b], kMul);
      mbar_init(&cx.sum_empty[b], 1);
    }
    mbar_init(&cx.listed, 1);
    cx.cta_abort = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  grid_wait();  // the prologue's logits, rows and cleared counters

  if (warp == 0) {
    copy_weights(&maps, lane);
  } else if (warp == 1) {
    copy_rest(&maps, lane);
  } else if (warp < kFirstMul) {
    finish(warp - kCopy, lane);
  } else {
    build_lists(threadIdx.x - 32 * kFirstMul);
    const int mul = warp - kFirstMul;
    for (int at = 0; at >= 0;) {
      at = multiply(mul, lane, at);
      if (at >= 0) at = multiply_scaled(mul, lane, at);
    }
  }
}

}  // namespace

// --------------------------------------------------------------------- launch

// Shared memory of a CTA when two, or when one, share an SM, less the ring's alignment.
constexpr int kRoomOfTwo = 113 * 1024 - 1024, kRoomOfOne = 227 * 1024 - 1024;

// Two slots at least; where two CTAs leave no room for that, one takes the SM.  With latent
// projections or a shared expert, whose units have the partial sums of 8 tokens, that is so
// from 12 tokens on at k = 16, 15 at k = 8, 16 at k = 6, 19 at k = 2: 8 of 384 experts, latent 3584 x 1024,
// 14 tokens 204 us, 15 tokens 248; 6 of 128, 4096 x 1408 and shared 2816, 15 tokens 156, 16
// tokens 201.
int few_stages(const FewArgs& a) {
  const Layout lay(a);
  int n = (kRoomOfTwo - lay.rest()) / lay.slot;
  if (n < 2) n = (kRoomOfOne - lay.rest()) / lay.slot;
  return n < kMaxSlots ? n : kMaxSlots;
}

static int launch_main(const FewArgs& a, const FewMaps& maps, cudaStream_t st) {
  MOE_TRY_CUDA(adapter_smem(reinterpret_cast<const void*>(few_kernel)));
  const Layout lay(a);
  const int smem = lay.rest() + lay.slot * a.stages;
  // no more CTAs than there can be units
  const int64_t tc = few_chunks(a.T, kFewRows / 2);
  const int64_t units = (a.L / 32 + a.S / 16 + a.H / 32 * 2) * tc +
                        static_cast<int64_t>(a.T) * a.k * (a.I / 16 + a.D / 32);
  const int64_t most = static_cast<int64_t>(num_sms()) * (smem <= kRoomOfTwo ? kCtas : 1);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units < most ? units : most));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  set_adapter_attrs(&cfg, attr, 0);
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, few_kernel, maps, a));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

int launch_few(const FewArgs& a, const FewMaps& maps, cudaStream_t st) {
  const int routers = a.router_w ? (a.E + kFrontExperts - 1) / kFrontExperts : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(routers + (a.L > 0 ? 1 : a.T));
  cfg.blockDim = dim3(kFrontThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  set_adapter_attrs(&cfg, attr, 0);
  MOE_TRY_CUDA(adapter_smem(reinterpret_cast<const void*>(few_front_kernel)));
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, few_front_kernel, a, routers));
  MOE_LAUNCH_CHECK();
  return launch_main(a, maps, st);
}

}  // namespace moe
