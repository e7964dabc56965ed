// Instances of the state-space scan's sweep kernel (m2rnn_ssm_sweep.h) and their dispatch.
#include "m2rnn_ssm_sweep.h"

namespace m2rnn {
namespace {

#ifndef M2RNN_SSM_IN
#define M2RNN_SSM_IN uint16_t
#define M2RNN_SSM_VEC true
#define M2RNN_SSM_NAME launch_ssm_sweep_bf16
#endif

template <typename InT, int AT, int NT, int RS, int MODE>
hipError_t run(const SsmSweepArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.B * a.N * a.nseg * a.slabs));
  if constexpr (sizeof(InT) == 2 && (MODE == ssm::kY || MODE == ssm::kDv))
    if (a.nseg > 1) {  // the last state comes from the segments' scan (asked for or not, so that the
                       // other results do not depend on it)
      hipLaunchKernelGGL((ssm::m2rnn_ssm_sweep_kernel<InT, AT, NT, RS, MODE, false, M2RNN_SSM_VEC>),
                         grid, dim3(256), 0, stream, a);
      return hipGetLastError();
    }
  hipLaunchKernelGGL((ssm::m2rnn_ssm_sweep_kernel<InT, AT, NT, RS, MODE, true, M2RNN_SSM_VEC>), grid,
                     dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Columns per workgroup (ssm_columns), and how many waves share them when there are few: two or
// four waves split the chunk's rows instead of repeating them (two prompts of 4096 tokens, 64 heads
// on one q and k, K = 64: V = 16 takes 74 us shared and 86 not; four of 8192, 16 heads, V = 32 84
// and 92); dq contracts over the columns in blocks of 32, so four would have nothing to share.
template <typename InT, int AT, int MODE>
hipError_t pick_nt(const SsmSweepArgs& a, hipStream_t stream) {
  if constexpr (AT <= 2)
    if (ssm_columns(a.DA, a.DC) == 128) return run<InT, AT, 2, 1, MODE>(a, stream);
  if constexpr (MODE != ssm::kDq)
    if (a.DC <= 16) return run<InT, AT, 1, 4, MODE>(a, stream);
  if (a.DC <= 32) return run<InT, AT, 1, 2, MODE>(a, stream);
  return run<InT, AT, 1, 1, MODE>(a, stream);
}

template <typename InT, int MODE>
hipError_t pick_at(const SsmSweepArgs& a, hipStream_t stream) {
  if (a.DA <= 32) return pick_nt<InT, 1, MODE>(a, stream);
  if (a.DA <= 64) return pick_nt<InT, 2, MODE>(a, stream);
  if (a.DA <= 128) return pick_nt<InT, 4, MODE>(a, stream);
  // only y and dv contract over K; dq and dk contract over V <= 128
  if constexpr (MODE == ssm::kY || MODE == ssm::kDv) return pick_nt<InT, 8, MODE>(a, stream);
  return hipErrorInvalidValue;
}

template <typename InT>
hipError_t pick_mode(const SsmSweepArgs& a, hipStream_t stream) {
  switch (a.mode) {
    case ssm::kY: return pick_at<InT, ssm::kY>(a, stream);
    case ssm::kDv: return pick_at<InT, ssm::kDv>(a, stream);
    case ssm::kDk: return pick_at<InT, ssm::kDk>(a, stream);
    default: return pick_at<InT, ssm::kDq>(a, stream);
  }
}

}  // namespace

hipError_t M2RNN_SSM_NAME(const SsmSweepArgs& a, hipStream_t stream) {
  return pick_mode<M2RNN_SSM_IN>(a, stream);
}

}  // namespace m2rnn
