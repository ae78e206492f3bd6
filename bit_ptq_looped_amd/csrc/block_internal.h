// Shared by the translation units of the block's parts between its linears and
// the attention.  Not part of the public C ABI (include/loopq_block.h).
#pragma once

#include "../../include/loopq_block.h"
#include "kv_internal.h"

namespace loopq {

constexpr int kNormMaxK = 32768;

struct NormArgs {
  const void* x;
  const void* res;    // null: none
  const float* w;     // null: none
  void* sum;          // null: not wanted
  void* y;            // null: not wanted
  int8_t* codes;      // null: not wanted
  float* steps;
  int64_t ldx, ldr, lds, ldy;  // elements
  int64_t row0;       // first row of the launch
  int rows, K;        // rows: all of the call's
  int x_bf16, res_bf16, y_bf16;
  int per_token;
  float eps, clip, qmax;
};
hipError_t launch_rms_norm(NormArgs a, hipStream_t s);

}  // namespace loopq
