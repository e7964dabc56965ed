// One token of every sequence through the selective state-space scan:
//     d = softplus(logit + beta),  H <- exp(-alpha d) H + d k v^T,  y = H^T q + w_r (.) v.
// The state is read and written once, 8 K V bytes a head against 4 K V multiply-adds, so the
// step is bound by HBM.  A wave (W = 1) or a workgroup of four takes a head: lanes run along V in
// 16-byte pieces and then along K, four pieces per lane in flight; the columns' sums are
// joined by lane exchanges and, for four waves, through LDS.  512 sequences of 16 heads, K = V = 64:
// 46.6 us for 273 MB (5.9 TB/s, part of the state still in the memory-side cache from the step
// before); 58 us after other work has emptied it (4.7 TB/s; 63 with the state's loads behind the decay
// instead of before it); sixteen pieces in flight took 87.
#include "m2rnn_io.h"
#include "m2rnn_ssm_internal.h"
#include "m2rnn_ssm_sweep.h"

namespace m2rnn {

namespace {

// W waves per head; VEC columns per lane; NB column blocks per lane (V > 64 VEC).
template <typename InT, int W, int VEC, int NB>
__global__ void __launch_bounds__(256) m2rnn_ssm_step_kernel(const SsmStepArgs g) {
  constexpr int HEADS = 4 / W;  // heads per workgroup
  __shared__ float red[W > 1 ? W : 1][64 * VEC * NB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t unit = (int64_t)blockIdx.x * HEADS + wave / W;
  const int wh = wave % W;
  const bool live = unit < g.B * g.N;  // whole waves; with W = 4, whole workgroups
  if (W == 1 && !live) return;
  const int64_t b = unit / g.N, n = unit % g.N;
  const int K = (int)g.K, V = (int)g.V;
  const int64_t qk = (b * g.NQ + n / (g.N / g.NQ)) * K;
  const InT* kp = (const InT*)g.k + qk;
  const InT* qp = (const InT*)g.q + qk;
  const InT* vp = (const InT*)g.v + unit * V;
  float* H = g.H + unit * (int64_t)K * V;

  // lv lanes along V (a power of two), 64 / lv rows per pass of a wave
  const int lv = g.lanes_v, rows = 64 / lv;
  const int cl = lane & (lv - 1), r0 = wh * rows + lane / lv;
  // the first rows of the state are on their way while the decay is made
  constexpr int U = 4;
  const float logit = g.logit[unit], beta = g.beta[n], alpha = g.alpha[n];
  io::Vals<VEC> h[U][NB];
  float k[U], q[U];
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int row = r + i * rows * W;
      const bool ok = row < K;
      k[i] = ok ? load_in(kp + row) : 0.0f;
      q[i] = ok ? load_in(qp + row) : 0.0f;
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        const int col = (c * lv + cl) * VEC;
        if (ok && col < V) h[i][c] = io::load<VEC>(H + (int64_t)row * V + col);
      }
    }
  };
  load(r0);
  float v[NB][VEC], acc[NB][VEC];
#pragma unroll
  for (int c = 0; c < NB; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int col = (c * lv + cl) * VEC + j;
      v[c][j] = col < V ? load_in(vp + col) : 0.0f;
      acc[c][j] = 0.0f;
    }
  const float d = ssm::softplus(logit + beta);
  const float f = ssm::pow2(ssm::log2_decay(alpha, d));
  for (int r = r0; r < K; r += rows * W * U) {
    if (r != r0) load(r);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int row = r + i * rows * W;
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        const int col = (c * lv + cl) * VEC;
        if (row < K && col < V) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float x = __builtin_fmaf(f, h[i][c].x[j], k[i] * d * v[c][j]);
            h[i][c].x[j] = x;
            acc[c][j] = __builtin_fmaf(x, q[i], acc[c][j]);
          }
          io::store<VEC>(H + (int64_t)row * V + col, h[i][c]);
        }
      }
    }
  }
  for (int s = lv; s < 64; s *= 2)
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[c][j] += __shfl_xor(acc[c][j], s);
  if constexpr (W > 1) {
    if (lane < lv)
#pragma unroll
      for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) red[wh][(c * lv + cl) * VEC + j] = acc[c][j];
    __syncthreads();
    if (wh != 0) return;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int i = (c * lv + cl) * VEC + j;
        acc[c][j] = (red[0][i] + red[1][i]) + (red[W - 2][i] + red[W - 1][i]);
      }
  }
  if (lane < lv) {
    InT* y = (InT*)g.y + unit * V;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int col = (c * lv + cl) * VEC + j;
        if (col < V)
          io::store<1>(y + col, io::Vals<1>{__builtin_fmaf(g.w_r[n * V + col], v[c][j], acc[c][j])});
      }
  }
}

template <typename InT, int W>
hipError_t run(SsmStepArgs g, bool vec, hipStream_t stream) {
  const int vec_n = vec ? 4 : 1;
  int lv = 1;
  while (lv < 64 && lv * vec_n < g.V) lv *= 2;
  g.lanes_v = lv;
  const dim3 grid((unsigned)((g.B * g.N + 4 / W - 1) / (4 / W)));
  if (vec)
    hipLaunchKernelGGL((m2rnn_ssm_step_kernel<InT, W, 4, 1>), grid, dim3(256), 0, stream, g);
  else if (g.V <= 64)
    hipLaunchKernelGGL((m2rnn_ssm_step_kernel<InT, W, 1, 1>), grid, dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL((m2rnn_ssm_step_kernel<InT, W, 1, 2>), grid, dim3(256), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_step(const SsmStepArgs& g, int in_dtype, hipStream_t stream) {
  const bool vec = g.V % 4 == 0 && aligned16(g.H);
  // a wave holds 4 x 64 x 4 elements in flight: larger heads are shared by four waves (2048 heads of
  // 128 x 128: 43.8 us shared, 46.9 not; 8192 of 64 x 64: 46.6 both; 8192 of 32 x 64: 31.4 and 24.1; 32768
  // of 64 x 16: 81 and 48)
  const bool split = g.K * g.V >= 4096;
  if (in_dtype == kBF16)
    return split ? run<uint16_t, 4>(g, vec, stream) : run<uint16_t, 1>(g, vec, stream);
  return split ? run<float, 4>(g, vec, stream) : run<float, 1>(g, vec, stream);
}

}  // namespace m2rnn
