// The routed experts of a few tokens in two launches: a prologue and one
// persistent kernel (few.cu), shared with their entry points (few_api.cu).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

constexpr int kFewWidth = 1 << 20;  // largest width: units are counted in 32 bits
constexpr int kFewTokens = 32;  // tokens of a call: one bit each in an expert's mask
constexpr int kFewChunk = 2;    // tokens that share one pass over an expert's weights
constexpr int kFewRows = 8;     // tokens that share one pass over bf16 weights (4 in two parts)
constexpr int kFewColumns = 2048;  // int4 columns of a ring slot

constexpr int kFewGroups = 32;  // groups of chunks whose outputs are summed before they are stored

// Kinds of work units.  A unit is 32 weight rows (16 gate rows and the 16 up rows of
// the same columns) times the tokens of one chunk; a down projection's takes a group of chunks one after another.
// Units are taken in this order.
enum FewKind {
  kFewLatDown = 0,   // u = x lat_down^T           bf16 weights
  kFewSharedUp = 1,  // SiLU(x gate^T) * x up^T    bf16 weights
  kFewGateUp = 2,    // h of one expert            int4 weights
  kFewDown = 3,      // y of one expert            int4 weights
  kFewSharedDown = 4,
  kFewLatUp = 5,
  kFewKinds = 6,
  kFewEnd = 7
};

// Scales in 4-byte copies; by TMA (K a multiple of 256); or, of rows of at most a slot's
// columns, 16 whole rows in one bulk copy.
constexpr int kScalesWords = 0, kScalesTma = 1, kScalesDense = 2;

// Arguments of both kernels; pointers not used by a call are NULL.
struct FewArgs {
  // inputs
  const uint16_t* x;         // bf16 [T, H]
  const float* router_w;     // fp32 [E, H]; NULL: the choice is given
  const float* router_bias;  // fp32 [E]
  const int32_t* topk_idx;   // int32 [T, k], where the choice is given
  const float* topk_w;       // fp32 [T, k]
  const uint16_t* scale[3];  // bf16 scales of gate, up, down
  const uint16_t* lat_norm;  // bf16 [L] or NULL
  uint16_t* out;             // bf16 [T, H]
  // sizes: D is the width the experts see, L where the layer is latent (else 0)
  int T, H, E, k, I, L, D, S;
  int renorm, norm;
  float eps;
  int tma_scale[2];  // how the scales of gate/up and of down are copied, kScales*
  // workspace
  int32_t* counters;
  int n_counters;
  float* scores;     // fp32 [T, E] sigmoid of the logits
  uint32_t* keys;    // [T, E] order of score + bias
  uint8_t* x16;      // [T] rows of fp16 blocks (below): x times a power of two, or u
  float* x_unit;     // fp32 [T]: what one unit of x16 stands for
  float* u_unit;     // fp32 [T, L / 16]: what one unit of 16 columns of u stands for
  uint8_t* h16;      // [T k] rows of fp16 blocks
  float* h_unit;     // fp32 [T k, I / 16]: the same of h
  float* y;          // fp32 [groups, T, D]: weighted sums of the chunks of a group
  uint16_t* hs;      // bf16 [2, T, S]: high and low parts of the shared expert's h
  float* ys;         // fp32 [T, H] shared expert's output
  uint16_t* z;       // bf16 [2, T, L]: high and low parts of the combined rows times the gain
  float* ssq;        // fp32 [L / 32, T] sums of squares
  float* yl;         // fp32 [T, H] latent up-projection
  int* status;
  long long wait_ns;
  int stages;        // ring slots
  int stall_at;      // tests only: the weight copies stop before this stage (-1: never)
};

// counters: [0] ticket, [1] u tiles done, [2] shared h tiles done, [3] z tiles
// done, then one per chunk (T k), then one per 32 columns of D, then one per 32
// columns of H and kFewRows / 2 tokens.  Those of u and of the chunks keep in a bit
// of their own whether a tile has a unit other than 1.
constexpr int kFewFixed = 4;
constexpr int kFewScaled = 1 << 30, kFewCount = kFewScaled - 1;

// h and u are stored as fp16.  h goes as the square of x, and u has the size of its weights
// and x, so both may lie anywhere: 16 columns (32 of u) whose largest value is below this
// are stored times the power of two that brings it to [2^14, 2^15).  Others are stored
// as they are: fp16's step of 2^-24 below its normal range then costs 2^-12 of them at most.
constexpr float kFewSmallest = 0x1p-11f;

// Matrices with tensor maps; the first three are of packed int4.
enum FewMatrix {
  kFewGateW, kFewUpW, kFewDownW, kFewLatDownW, kFewLatUpW, kFewSharedGateW, kFewSharedUpW,
  kFewSharedDownW, kFewMatrices
};

// A ring slot takes 16 rows of a matrix in one copy: `full` of a whole slot's
// pieces of 128 bytes of K, `rest` of the whole pieces of the last slot of a row,
// `tail` of the columns behind them (K no multiple of 256).
struct FewMaps {
  CUtensorMap full[kFewMatrices], rest[kFewMatrices], tail[3], scale[3];
  CUtensorMap rows[3];  // tokens of the bf16 units: x, the shared expert's h, z
};

// A row of fp16 activations lies in blocks of kFewColumns columns in pair order, each
// followed by its start values (few.cu), one fp32 for 16 columns.
constexpr int kFewBlock = kFewColumns * 2 + kFewColumns / 16 * 4;
__host__ __device__ inline int64_t few_row_bytes(int K) {
  return static_cast<int64_t>((K + kFewColumns - 1) / kFewColumns) * kFewBlock;
}
// Row of column c and its 16-column group's start value.
__host__ __device__ inline int64_t few_value_at(int c) {
  return static_cast<int64_t>(c / kFewColumns) * kFewBlock + c % kFewColumns * 2;
}
__host__ __device__ inline int64_t few_start_at(int c) {
  return static_cast<int64_t>(c / kFewColumns) * kFewBlock + kFewColumns * 2 +
         c % kFewColumns / 16 * 4;
}

__host__ __device__ inline int few_chunks(int T, int rows) { return (T + rows - 1) / rows; }
// Tokens that share a pass over the weights of a bf16 kind.
__host__ __device__ inline int few_rows_of(int kind) {
  return kind == kFewSharedDown || kind == kFewLatUp ? kFewRows / 2 : kFewRows;
}

// Ring slots that fit into shared memory.
int few_stages(const FewArgs& a);

// Both launches (validated arguments, a workspace as few_api.cu carves it).
int launch_few(const FewArgs& a, const FewMaps& maps, cudaStream_t st);

}  // namespace moe
