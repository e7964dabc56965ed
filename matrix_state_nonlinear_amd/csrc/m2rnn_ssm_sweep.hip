// Instances of the state-space scan's sweep kernel (m2rnn_ssm_sweep.h) and their dispatch.
#include "m2rnn_ssm_sweep.h"

namespace m2rnn {
namespace {

template <typename InT, int AT, int NT, int MODE>
hipError_t run(const SsmSweepArgs& a, hipStream_t stream) {
  const int64_t grid = a.B * a.N * a.nseg * a.slabs;
  hipLaunchKernelGGL((ssm::m2rnn_ssm_sweep_kernel<InT, AT, NT, MODE>), dim3((unsigned)grid),
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
  if constexpr (MODE == ssm::kPlain) return pick_nt<InT, 8, MODE>(a, stream);
  return hipErrorInvalidValue;
}

template <typename InT>
hipError_t pick_mode(const SsmSweepArgs& a, hipStream_t stream) {
  if (a.pairs) return pick_at<InT, ssm::kPairs>(a, stream);
  if (a.e) return pick_at<InT, ssm::kRowdot>(a, stream);
  return pick_at<InT, ssm::kPlain>(a, stream);
}

}  // namespace

#ifdef M2RNN_SSM_F32
hipError_t launch_ssm_sweep_f32(const SsmSweepArgs& a, hipStream_t stream) {
  return pick_mode<float>(a, stream);
}
#else
hipError_t launch_ssm_sweep_bf16(const SsmSweepArgs& a, hipStream_t stream) {
  return pick_mode<uint16_t>(a, stream);
}
#endif

}  // namespace m2rnn
