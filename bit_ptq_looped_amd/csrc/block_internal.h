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
  int rows, K;
  int x_bf16, res_bf16, y_bf16;
  int per_token;
  float eps, clip, qmax;
  double inv_k;       // 1 / K
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);

// One tensor of a rotary call: [tokens][heads][dim], heads side by side.
struct RopePart {
  const void* in;
  void* out;          // null for the keys and values of a cache write
  int64_t ld_in, ld_out;  // elements
  int heads;
  int out_bf16;
};

// Rotary positions of up to three tensors: q (turned, to out), k (turned) and v
// (as it is) to the slab.  Without a cache, part[0] alone at given positions.
struct RopeArgs {
  RopePart part[3];
  int in_bf16;
  int tokens, head_dim, rot, pairs;
  const double* inv_freq;
  float magnitude;
  const int32_t* positions;  // given positions, or null: from the table
  const int32_t* cu;
  KvTable t;
  uint16_t* pool;            // at the slab's keys of page 0
  int64_t page_stride, plane;
  int page_shift;
  int heads;                 // of all parts
  int split, per;            // waves a token, heads each of them takes
};
hipError_t launch_rope(RopeArgs a, hipStream_t s);

constexpr int kAdapterMaxRank = 128;
constexpr int kAdapterMaxRows = 1 << 20;
// bytes between rows: 64 rows of x, or 32 of y, lie within 2^31 bytes
constexpr int64_t kAdapterMaxLdx = 1 << 25, kAdapterMaxLdy = 1 << 26;
struct AdapterArgs {
  const void* x;
  int64_t ldx;           // elements
  int x_bf16, rows, K, N;
  const int32_t* ids;    // [rows]
  const uint16_t* A;     // bf16 [adapters][R][K]
  const uint16_t* B;     // bf16 [adapters][N][R]
  const float* scales;   // [adapters]
  const int32_t* ranks;  // [adapters], or null: all R
  int adapters, R;
  float* y;
  int64_t ldy;
  bool sort;             // (by the launcher) tokens of a segment may be put in order
  float* z;              // workspace: [splits][rows][R]
  uint16_t* planes;      // behind it: bf16 [rows][R / 8][3][8] (by the launcher)
  int2* order;           // behind them: row and adapter (or -1) of each place [rows] (by the launcher)
};
size_t adapter_workspace_bytes(int64_t rows, int max_rank);
hipError_t launch_adapter(AdapterArgs a, hipStream_t s);

}  // namespace loopq
