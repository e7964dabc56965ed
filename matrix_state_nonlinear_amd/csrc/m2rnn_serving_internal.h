// Host-side interface of the carried convolution and of group norm with a gate for the C ABI
// (m2rnn_api.hip).
#pragma once

#include "m2rnn_internal.h"

namespace m2rnn {

// The convolution with a carried history (m2rnn_carry.hip).
struct CarryArgs {
  int64_t B, T, C;
  const void* x;       // [B, T, C] io type
  const float* w;      // [C, 4]
  const float* bias;   // [C] or null
  const void* hist;    // [B, 3, C] io type or null: the inputs before x
  void* out;           // [B, T, C] io type
  void* hist_out;      // [B, 3, C] io type or null; the single-token form's history, in place
  const int* lens;     // [B] or null: inputs of each sequence that count for hist_out
  const void* dout;    // backward: [B, T, C] io type
  void* dx;            // [B, T, C] io type
  float* dw;           // [C, 4]
  float* dbias;        // [C] or null
  void* dhist;         // [B, 3, C] io type or null
  float* ws;
};
size_t conv_carry_workspace_floats(int64_t B, int64_t T, int64_t C);
// what: 0 forward, 1 backward, 2 one token
hipError_t launch_conv_carry(const CarryArgs& a, int io_dtype, int what, hipStream_t stream);

// Group norm with a SiLU gate (m2rnn_groupnorm.hip): rows of G groups of S channels.
struct GroupNormArgs {
  int64_t rows, G, S;
  float eps;
  const void* y;       // [rows, G S] io type
  const void* g_pre;   // [rows, G S] io type
  const float* gamma;  // [G S]
  const float* beta;   // [G S]
  void* out;           // forward: [rows, G S] io type
  const void* dout;    // backward: [rows, G S] io type
  void* dy;            // [rows, G S] io type
  void* dg_pre;        // [rows, G S] io type
  float* dgamma;       // [G S]
  float* dbeta;        // [G S]
  float* ws;
  int lg, gw;          // lanes per group and groups per wave, set by the launcher
  int64_t rows_per;    // rows per wave
};
size_t groupnorm_workspace_floats(int64_t rows, int64_t G, int64_t S, int io_dtype);
// Whether the grids of either direction stay below 2^32 threads.
bool groupnorm_grid_ok(int64_t rows, int64_t G, int64_t S, int io_dtype);
hipError_t launch_groupnorm_gate(const GroupNormArgs& a, int io_dtype, bool bwd, hipStream_t stream);

}  // namespace m2rnn
