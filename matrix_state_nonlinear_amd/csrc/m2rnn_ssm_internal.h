// Host-side interface of the selective state-space scan (m2rnn_ssm_*.hip) for
// the C ABI (m2rnn_api.hip), and the argument blocks of its kernels.
#pragma once

#include "m2rnn_internal.h"

namespace m2rnn {

// One pass of the decayed linear attention that the scan and its gradients
// consist of (m2rnn_ssm_sweep.h): for a head, over the tokens p in walking order,
//     out_p = rho_p (sum_{p' <= p} D_{pp'} g_{p'} (a_p . b_p') c_p' + R_p S^T a_p) [+ skip (.) c_p]
// from the state S [DA, DC] carried in.
struct SsmSweepArgs {
  const void* a;        // [B, T, N / a_grp, DA]: head n reads head n / a_grp
  const void* b;        // [B, T, N / b_grp, DA]
  const void* c;        // [B, T, N / c_grp, DC]
  const void* e;        // [B, T, N / e_grp, DC] (dk, dq): rowdot_p = e_p . (R_p S^T a_p)
  const double* cum;    // [B, N, T] sums of log2 f over each chunk (ssm_chunk tokens) up to a token
  const float* d;       // [B, N, T] step sizes
  const float* skip;    // [N, DC] or null
  void* out;            // [B, T, N, DC], input type, or fp32 when out_f32
  float* rowdot;        // [slabs, B, N, T] (dk, dq)
  float* pairs;         // [slabs, B, N, T] (dq): with M_ij = g_j D_ij (e_i . c_j)(a_i . b_j),
                        // the sum of M over the chunk's pairs i >= p > j
  float* colpairs;      // (dq) the sum of M_ip / g_p over the chunk's i >= p
  float* colsum;        // [B, N, nseg, DA] (dq): sum_p a_p (.) b_p
  const float* state0;  // [B, N, nseg, *] segment starts (or [B, N, *] when nseg = 1), or null = 0
  float* stateT;        // [B, N, *] or null: the state after the last token (nseg = 1 only)
  const float* hend;    // base only: [B, N, nseg, *], the other state at each segment's end is
                        // entry s + 1, and hend_last [B, N, *] for the last one
  const float* hend_last;
  double* base;         // [slabs, B, N, nseg] or null: <state0, hend> of every segment
  int64_t B, T, N, nseg, seglen, slabs;
  int a_grp, b_grp, c_grp, e_grp;
  int DA, DC;
  int a_stride, c_stride;  // element strides of a state along DA and DC
  int mode;                // which of the sweeps (kY .. kDq of m2rnn_ssm_sweep.h): the direction, and
                           // whether d_p multiplies the inputs (g) or the outputs (rho)
  int out_f32;
  int vec;                 // 16-byte accesses of a, b, c, e and 4-element ones of out allowed
};

// State that each segment of T adds to a zero start, and its decay.
struct SsmContribArgs {
  const void* b;        // [B, T, N / b_grp, DA]
  const void* c;        // [B, T, N / c_grp, DC]
  const double* cum;    // as above
  const float* d;
  float* contrib;       // [B, N, nseg, DA, DC]
  float* fseg;          // [B, N, nseg] decay over a segment, or null
  int64_t B, T, N, nseg, seglen, slabs;
  int b_grp, c_grp;
  int DA, DC;
  int rev, w_in;
  int vec;
};

// One token of every sequence.
struct SsmStepArgs {
  const void* k;        // [B, NQ, K]
  const void* v;        // [B, N, V]
  const void* q;        // [B, NQ, K]
  const float* logit;   // [B, N]
  const float* alpha;   // [N]
  const float* beta;    // [N]
  const float* w_r;     // [N, V]
  float* H;             // [B, N, K, V], updated in place
  void* y;              // [B, N, V]
  int64_t B, N, NQ, K, V;
  int lanes_v;          // lanes along V, set by the launcher
};
hipError_t launch_ssm_step(const SsmStepArgs& a, int in_dtype, hipStream_t stream);

// Whole-call arguments (device pointers checked by the ABI).
struct SsmArgs {
  const void* k;
  const void* v;
  const void* q;
  const float* logit;
  const float* alpha;
  const float* beta;
  const float* w_r;
  const float* H0;      // may be null
  void* y;              // forward
  float* HT;            // forward, may be null
  const void* dy;       // backward
  const float* dHT;     // may be null
  void* dk;
  void* dv;
  void* dq;
  float* dlogit;
  float* dw_r;
  float* dalpha;
  float* dbeta;
  float* dH0;           // may be null
  float* ws;
  int64_t B, T, N, NQ, K, V;
};

// Columns of the output (DC of the sweep, contracting over DA) per workgroup: up to 128, or 64
// where a 128-column state would not leave registers for two workgroups per CU.  Four prompts of
// 4096 tokens, 16 heads, K = 64, V = 128: 94 us with 128 columns, 106 with 64 (each slab reads the
// other tensors again); one of 16384 tokens, 32 heads, K = V = 128: the sweep takes 230 us with 128
// columns, 213 with 64.
inline int ssm_columns(int64_t DA, int64_t DC) { return DC > 64 && DA <= 64 ? 128 : 64; }
inline int64_t ssm_slabs(int64_t DA, int64_t DC) {
  const int c = ssm_columns(DA, DC);
  return (DC + c - 1) / c;
}

// Workspace of a call: offsets in floats (64-float aligned) and the split of T
// into nseg segments of seglen tokens.
struct SsmLayout {
  int64_t nseg, seglen;
  size_t cum, d;                           // [B, N, T] double, float
  size_t hseg, fseg;                       // [B, N, nseg, K, V], [B, N, nseg] (nseg > 1 or backward)
  size_t gseg, hT, base, adot, bdot, pairs, colpairs;  // backward
  size_t colsum, gatepart, dqp, dkp;
  size_t total_floats;
};
SsmLayout ssm_fwd_layout(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V, int in_dtype);
SsmLayout ssm_bwd_layout(int64_t B, int64_t T, int64_t N, int64_t NQ, int64_t K, int64_t V);
hipError_t launch_ssm_fwd(const SsmArgs& a, int in_dtype, hipStream_t stream);
hipError_t launch_ssm_bwd(const SsmArgs& a, int in_dtype, hipStream_t stream);

// The sweep's instances, by input type, and by whether 16-byte accesses are allowed (not: _any),
// each in a file of its own (they compile in parallel).
hipError_t launch_ssm_sweep_bf16(const SsmSweepArgs& a, hipStream_t stream);
hipError_t launch_ssm_sweep_bf16_any(const SsmSweepArgs& a, hipStream_t stream);
hipError_t launch_ssm_sweep_f32(const SsmSweepArgs& a, hipStream_t stream);
hipError_t launch_ssm_sweep_f32_any(const SsmSweepArgs& a, hipStream_t stream);
hipError_t launch_ssm_sweep(const SsmSweepArgs& a, int in_dtype, hipStream_t stream);
hipError_t launch_ssm_contrib(const SsmContribArgs& a, int in_dtype, hipStream_t stream);
// The step sizes and, per chunk of the sweeps, the running sums of log2 f.
hipError_t launch_ssm_decays(const SsmArgs& a, int in_dtype, double* cum, float* d,
                             hipStream_t stream);
// Whether rows of `heads` x `D` elements at p can be accessed in 16-byte pieces with 32-bit offsets
// within a chunk.  Element accesses otherwise (670 us instead of 234 for four prompts of 16384
// tokens, 16 heads, K = V = 64).
bool ssm_vec_rows(const void* p, int64_t heads, int64_t D, int elem_bytes);
// Scans over the segments, one or two in a launch: seg [units, nseg, KV] (what a segment adds)
// becomes the state each starts from (rev: ends at), `first` [units, KV] or null = 0 the first
// one's, and `last` [units, KV] or null gets the state behind the last.
struct SsmSegScan {
  float* seg;
  const float* first;
  float* last;
  bool rev;
};
struct SsmSegScans {
  SsmSegScan s[2];
};
hipError_t launch_ssm_segscan(const SsmSegScans& scans, const float* fseg, int64_t units,
                              int64_t nseg, int64_t KV, hipStream_t stream);

}  // namespace m2rnn
