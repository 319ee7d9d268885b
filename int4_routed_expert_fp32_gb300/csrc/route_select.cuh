// Selection of the grouped router (route_select.cu), over logits or over the
// router GEMM's partial logits.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Host checks of a moe_route_config; MOE_OK or the error to return.
int check_route_config(const moe_route_config* cfg);

// topk_idx / topk_w [T, k] from the logits z of expert e of token t,
//   z = sum over p < S, in order, of in[t * ld + p * sp + e]
// (logits given by the caller: S = 1).  Validated arguments.
int launch_route_select(const moe_route_config& cfg, const void* in, bool bf16, size_t ld, int S,
                        size_t sp, const float* bias, int T, int32_t* topk_idx, float* topk_w,
                        cudaStream_t s);

}  // namespace moe
