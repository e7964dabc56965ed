// Instances of the state-space scan's sweep kernel (m2rnn_ssm_sweep.h) and their dispatch.
#include "m2rnn_ssm_sweep.h"

namespace m2rnn {
namespace {

#ifndef M2RNN_SSM_IN
#define M2RNN_SSM_IN uint16_t
#define M2RNN_SSM_VEC true
#define M2RNN_SSM_NAME launch_ssm_sweep_bf16
#endif

template <typename InT, int AT, int NT, int MODE>
hipError_t run(const SsmSweepArgs& a, hipStream_t stream) {
  const int64_t grid = a.B * a.N * a.nseg * a.slabs;
  hipLaunchKernelGGL((ssm::m2rnn_ssm_sweep_kernel<InT, AT, NT, MODE, M2RNN_SSM_VEC>), dim3((unsigned)grid),
                     dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename InT, int AT, int MODE>
hipError_t pick_nt(const SsmSweepArgs& a, hipStream_t stream) {
  return a.DC <= 64 ? run<InT, AT, 1, MODE>(a, stream) : run<InT, AT, 2, MODE>(a, stream);
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
