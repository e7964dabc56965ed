// The selective state-space scan: segments of T, the pass between them, and the host side of
// the forward (the sweep kernel itself is in m2rnn_ssm_sweep.h).
//
// A head's tokens can be split into segments that run at the same time: a first pass
// computes what each segment adds to a zero state, a scan over the segments turns these into
// every segment's starting state, and the sweep then runs all segments from theirs.  The
// first pass costs about half a sweep again, so T is only split as far as it takes to occupy the
// device.
#include "m2rnn_ssm_sweep.h"

namespace m2rnn {

namespace {

template <typename InT, int AT, int NT>
hipError_t run(const SsmContribArgs& a, hipStream_t stream) {
  const int64_t grid = a.B * a.N * a.nseg * a.slabs;
  hipLaunchKernelGGL((ssm::m2rnn_ssm_contrib_kernel<InT, AT, NT>), dim3((unsigned)grid),
                     dim3(256), 0, stream, a);
  return hipGetLastError();
}
template <typename InT, int AT>
hipError_t pick_nt(const SsmContribArgs& a, hipStream_t stream) {
  return a.DC <= 64 ? run<InT, AT, 1>(a, stream) : run<InT, AT, 2>(a, stream);
}
template <typename InT>
hipError_t pick_at(const SsmContribArgs& a, hipStream_t stream) {
  if (a.DA <= 32) return pick_nt<InT, 1>(a, stream);
  if (a.DA <= 64) return pick_nt<InT, 2>(a, stream);
  if (a.DA <= 128) return pick_nt<InT, 4>(a, stream);
  return pick_nt<InT, 8>(a, stream);
}

// seg[u][s] (what segment s adds) -> the state at its start (rev: at its end, from later
// segments); last[u] the state after all of them.  One thread per state element.
__global__ void __launch_bounds__(256)
    m2rnn_ssm_segscan_kernel(float* __restrict__ seg, const float* __restrict__ fseg,
                             const float* __restrict__ first, float* __restrict__ last,
                             int64_t total, int64_t nseg, int64_t KV, int rev) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t u = i / KV, x = i % KV;
  float cur = first ? first[i] : 0.0f;
  float* p = seg + u * nseg * KV + x;
  const float* f = fseg + u * nseg;
#pragma unroll 4
  for (int64_t s = 0; s < nseg; ++s) {
    const int64_t j = rev ? nseg - 1 - s : s;
    const float add = p[j * KV];
    p[j * KV] = cur;
    cur = __builtin_fmaf(f[j], cur, add);
  }
  if (last) last[i] = cur;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t pad64(size_t x) { return align_up(x, 64); }

}  // namespace

hipError_t launch_ssm_contrib(const SsmContribArgs& a, int in_dtype, hipStream_t stream) {
  return in_dtype == kBF16 ? pick_at<uint16_t>(a, stream) : pick_at<float>(a, stream);
}

hipError_t launch_ssm_segscan(float* seg, const float* fseg, const float* first, float* last,
                              int64_t units, int64_t nseg, int64_t KV, bool rev,
                              hipStream_t stream) {
  const int64_t total = units * KV;
  hipLaunchKernelGGL(m2rnn_ssm_segscan_kernel, dim3((unsigned)ceil_div(total, 256)), dim3(256), 0,
                     stream, seg, fseg, first, last, total, nseg, KV, rev ? 1 : 0);
  return hipGetLastError();
}

// Segments of the forward: as many as bring the grid to two workgroups per CU, of at
// least 128 tokens.
SsmLayout ssm_fwd_layout(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V, int in_dtype) {
  SsmLayout L{};
  const int64_t units = B * N;
  int64_t nseg = units > 0 ? ceil_div(512, units) : 1;
  const int64_t most = T / 128 > 1 ? T / 128 : 1;
  if (nseg > most) nseg = most;
  L.seglen = align_up((size_t)ceil_div(T > 0 ? T : 1, nseg), 64);
  L.nseg = ceil_div(T > 0 ? T : 1, L.seglen);
  size_t off = 0;
  if (L.nseg > 1) {
    L.hseg = off;
    off += pad64((size_t)units * L.nseg * K * V);
    L.fseg = off;
    off += pad64((size_t)units * L.nseg);
  }
  L.total_floats = off;
  return L;
}

hipError_t launch_ssm_sweep(const SsmSweepArgs& a, int in_dtype, hipStream_t stream) {
  return in_dtype == kBF16 ? launch_ssm_sweep_bf16(a, stream) : launch_ssm_sweep_f32(a, stream);
}

namespace {
// Whether rows of `D` elements at p can be read in 16-byte pieces.
int vec16(const void* p, int64_t D, int in_dtype) {
  return aligned16(p) && D % (in_dtype == kBF16 ? 8 : 4) == 0;
}
}  // namespace

hipError_t launch_ssm_fwd(const SsmArgs& a, int in_dtype, hipStream_t stream) {
  const SsmLayout L = ssm_fwd_layout(a.B, a.T, a.N, a.K, a.V, in_dtype);
  const int grp = (int)(a.N / a.NQ);
  const float* start = a.H0;
  hipError_t err;
  if (L.nseg > 1) {
    float* hseg = a.ws + L.hseg;
    float* fseg = a.ws + L.fseg;
    SsmContribArgs c{};
    c.b = a.k; c.c = a.v; c.b_grp = grp; c.c_grp = 1;
    c.logit = a.logit; c.alpha = a.alpha; c.beta = a.beta;
    c.contrib = hseg; c.fseg = fseg;
    c.B = a.B; c.T = a.T; c.N = a.N; c.nseg = L.nseg; c.seglen = L.seglen; c.slabs = 1;
    c.DA = (int)a.K; c.DC = (int)a.V; c.w_in = 1;
    c.vb = vec16(a.k, a.K, in_dtype);
    c.vc = vec16(a.v, a.V, in_dtype);
    if ((err = launch_ssm_contrib(c, in_dtype, stream)) != hipSuccess) return err;
    err = launch_ssm_segscan(hseg, fseg, a.H0, a.HT, a.B * a.N, L.nseg, a.K * a.V, false, stream);
    if (err != hipSuccess) return err;
    start = hseg;
  }
  SsmSweepArgs s{};
  s.a = a.q; s.b = a.k; s.c = a.v;
  s.a_grp = grp; s.b_grp = grp; s.c_grp = 1; s.e_grp = 1;
  s.logit = a.logit; s.alpha = a.alpha; s.beta = a.beta; s.skip = a.w_r;
  s.out = a.y;
  s.state0 = start;
  s.stateT = L.nseg > 1 ? nullptr : a.HT;
  s.B = a.B; s.T = a.T; s.N = a.N; s.nseg = L.nseg; s.seglen = L.seglen; s.slabs = 1;
  s.DA = (int)a.K; s.DC = (int)a.V;
  s.a_stride = (int)a.V; s.c_stride = 1;
  s.w_in = 1;
  s.va = vec16(a.q, a.K, in_dtype);
  s.vb = vec16(a.k, a.K, in_dtype);
  s.vc = vec16(a.v, a.V, in_dtype);
  s.vo = a.V % 4 == 0 && aligned16(a.y);
  return launch_ssm_sweep(s, in_dtype, stream);
}

}  // namespace m2rnn
