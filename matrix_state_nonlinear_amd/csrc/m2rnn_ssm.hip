// The selective state-space scan: segments of T, the pass between them, and the host side of
// the forward (the sweep kernel itself is in m2rnn_ssm_sweep.h).
//
// A first kernel makes every token's step size and the running sums of its chunk's decays, which
// all later passes read.
//
// A head's tokens can be split into segments that run at the same time: a first pass
// computes what each segment adds to a zero state, a scan over the segments turns these into
// every segment's starting state, and the sweep then runs all segments from theirs.  The
// first pass costs almost half a sweep again, so T is only split as far as it takes to occupy the
// device.  Four prompts of 16384 tokens, 16 heads, K = V = 64: sweep 144 us, first pass 66, decays 11,
// scan over the segments 8.
#include "m2rnn_ssm_sweep.h"

namespace m2rnn {

namespace {

template <typename InT, int AT, int NT, int RS>
hipError_t run(const SsmContribArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.B * a.N * a.nseg * a.slabs));
  const auto kernel = a.rev ? (a.vec ? ssm::m2rnn_ssm_contrib_kernel<InT, AT, NT, RS, true, true>
                                     : ssm::m2rnn_ssm_contrib_kernel<InT, AT, NT, RS, true, false>)
                            : (a.vec ? ssm::m2rnn_ssm_contrib_kernel<InT, AT, NT, RS, false, true>
                                     : ssm::m2rnn_ssm_contrib_kernel<InT, AT, NT, RS, false, false>);
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}
template <typename InT, int AT>
hipError_t pick_nt(const SsmContribArgs& a, hipStream_t stream) {
  if constexpr (AT <= 2)
    if (ssm_columns(a.DA, a.DC) == 128) return run<InT, AT, 2, 1>(a, stream);
  if constexpr (AT > 1)  // a wave keeps at least one 16-row tile of the state
    if (a.DC <= 16) return run<InT, AT, 1, 4>(a, stream);
  if (a.DC <= 32) return run<InT, AT, 1, 2>(a, stream);
  return run<InT, AT, 1, 1>(a, stream);
}
template <typename InT>
hipError_t pick_at(const SsmContribArgs& a, hipStream_t stream) {
  if (a.DA <= 32) return pick_nt<InT, 1>(a, stream);
  if (a.DA <= 64) return pick_nt<InT, 2>(a, stream);
  if (a.DA <= 128) return pick_nt<InT, 4>(a, stream);
  return pick_nt<InT, 8>(a, stream);
}

// Step sizes and chunk sums of log2 f for a workgroup's 64 tokens x 16 heads: logits come in
// rows of heads and the results go out in rows of tokens, through LDS.  A wave sums four
// heads, a lane per token; L = 32 has two chunks to a wave.  11 us for a million tokens x heads
// (17 MB, 1.5 TB/s): the logarithm and the double sums bound it, not the memory.
template <int L>
__global__ void __launch_bounds__(256)
    m2rnn_ssm_decays_kernel(int64_t T, int64_t N, const float* __restrict__ logit,
                            const float* __restrict__ alpha, const float* __restrict__ beta,
                            double* __restrict__ cum, float* __restrict__ d) {
  __shared__ float x[64][17];
  const int64_t hb = (N + 15) / 16, tb = (T + 63) / 64;
  const int64_t n0 = blockIdx.x % hb * 16, t0 = blockIdx.x / hb % tb * 64, b = blockIdx.x / hb / tb;
  for (int i = threadIdx.x; i < 64 * 16; i += 256) {
    const int64_t t = t0 + i / 16, n = n0 + i % 16;
    x[i / 16][i % 16] = t < T && n < N ? logit[(b * T + t) * N + n] : 0.0f;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float dt[4];
  double sum[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int64_t n = n0 + 4 * w + h < N ? n0 + 4 * w + h : N - 1;
    dt[h] = ssm::softplus(x[lane][4 * w + h] + beta[n]);
    sum[h] = t0 + lane < T ? ssm::log2_decay(alpha[n], dt[h]) : 0.0;
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) sum[h] = ssm::lane_sums<L>(sum[h]);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int64_t n = n0 + 4 * w + h;
    if (n < N && t0 + lane < T) {
      const int64_t at = (b * N + n) * T + t0 + lane;
      cum[at] = sum[h];
      d[at] = dt[h];
    }
  }
}

// One thread per state element; blockIdx.y the scan.  Loads run four segments ahead of the sums: 7 us
// for 12 segments of 64 heads of 64 x 64 states (25 MB, each read and written; a launch's latency).
__global__ void __launch_bounds__(256)
    m2rnn_ssm_segscan_kernel(const SsmSegScans scans, const float* __restrict__ fseg, int64_t total,
                             int64_t nseg, int64_t KV) {
  const SsmSegScan sc = scans.s[blockIdx.y];
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t u = i / KV, x = i % KV;
  float cur = sc.first ? sc.first[i] : 0.0f;
  float* p = sc.seg + u * nseg * KV + x;
  const float* f = fseg + u * nseg;
  for (int64_t s = 0; s < nseg; s += 4) {
    float add[4], fs[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t q = s + k < nseg ? s + k : nseg - 1, j = sc.rev ? nseg - 1 - q : q;
      add[k] = p[j * KV];
      fs[k] = f[j];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < nseg) {
        p[(sc.rev ? nseg - 1 - (s + k) : s + k) * KV] = cur;
        cur = __builtin_fmaf(fs[k], cur, add[k]);
      }
  }
  if (sc.last) sc.last[i] = cur;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t pad64(size_t x) { return align_up(x, 64); }

}  // namespace

hipError_t launch_ssm_contrib(const SsmContribArgs& a, int in_dtype, hipStream_t stream) {
  return in_dtype == kBF16 ? pick_at<uint16_t>(a, stream) : pick_at<float>(a, stream);
}

hipError_t launch_ssm_segscan(const SsmSegScans& scans, const float* fseg, int64_t units,
                              int64_t nseg, int64_t KV, hipStream_t stream) {
  const int64_t total = units * KV;
  hipLaunchKernelGGL(m2rnn_ssm_segscan_kernel,
                     dim3((unsigned)ceil_div(total, 256), scans.s[1].seg ? 2 : 1), dim3(256), 0,
                     stream, scans, fseg, total, nseg, KV);
  return hipGetLastError();
}

// Workgroups of the forward's sweep that a CU holds (LDS and registers of m2rnn_ssm_sweep.h).
int64_t ssm_per_cu(int64_t K, int64_t V, int in_dtype) {
  return in_dtype == kBF16 && K <= 64 && V <= 64 ? 3 : 2;
}

// Segments of the forward: as many as fill every CU once, of at least 64 tokens.  Four prompts of
// 16384 tokens, 16 heads, K = V = 64: 236 us (12 segments); unsplit 884 us, 24 segments 246.  One of
// 2048 tokens: 35 us, unsplit 109.
SsmLayout ssm_fwd_layout(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V, int in_dtype) {
  SsmLayout L{};
  const int64_t units = B * N, wgs = units * ssm_slabs(K, V);
  const int64_t want = 256 * ssm_per_cu(K, V, in_dtype);
  int64_t nseg = wgs > 0 ? ceil_div(want, wgs) : 1;
  const int64_t most = T / 64 > 1 ? T / 64 : 1;
  if (nseg > most) nseg = most;
  L.seglen = align_up((size_t)ceil_div(T > 0 ? T : 1, nseg), 64);
  L.nseg = ceil_div(T > 0 ? T : 1, L.seglen);
  size_t off = pad64((size_t)units * T * 2);  // cum, at 0
  L.d = off;
  off += pad64((size_t)units * T);
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
  if (in_dtype == kBF16)
    return a.vec ? launch_ssm_sweep_bf16(a, stream) : launch_ssm_sweep_bf16_any(a, stream);
  return a.vec ? launch_ssm_sweep_f32(a, stream) : launch_ssm_sweep_f32_any(a, stream);
}

bool ssm_vec_rows(const void* p, int64_t heads, int64_t D, int elem_bytes) {
  return aligned16(p) && D * elem_bytes % 16 == 0 && (double)heads * (double)D * elem_bytes < 16777216.0;
}

hipError_t launch_ssm_decays(const SsmArgs& a, int in_dtype, double* cum, float* d,
                             hipStream_t stream) {
  const dim3 grid((unsigned)(a.B * ceil_div(a.T, 64) * ceil_div(a.N, 16)));
  if (in_dtype == kBF16)
    hipLaunchKernelGGL(m2rnn_ssm_decays_kernel<ssm::Cfg<uint16_t>::L>, grid, dim3(256), 0, stream,
                       a.T, a.N, a.logit, a.alpha, a.beta, cum, d);
  else
    hipLaunchKernelGGL(m2rnn_ssm_decays_kernel<ssm::Cfg<float>::L>, grid, dim3(256), 0, stream, a.T,
                       a.N, a.logit, a.alpha, a.beta, cum, d);
  return hipGetLastError();
}

hipError_t launch_ssm_fwd(const SsmArgs& a, int in_dtype, hipStream_t stream) {
  const SsmLayout L = ssm_fwd_layout(a.B, a.T, a.N, a.K, a.V, in_dtype);
  const int grp = (int)(a.N / a.NQ), E = in_dtype == kBF16 ? 2 : 4;
  const float* start = a.H0;
  double* cum = (double*)(a.ws + L.cum);
  float* d = a.ws + L.d;
  hipError_t err = launch_ssm_decays(a, in_dtype, cum, d, stream);
  if (err != hipSuccess) return err;
  const bool vk = ssm_vec_rows(a.k, a.NQ, a.K, E), vv = ssm_vec_rows(a.v, a.N, a.V, E);
  if (L.nseg > 1) {
    float* hseg = a.ws + L.hseg;
    float* fseg = a.ws + L.fseg;
    SsmContribArgs c{};
    c.b = a.k; c.c = a.v; c.b_grp = grp; c.c_grp = 1;
    c.cum = cum; c.d = d;
    c.contrib = hseg; c.fseg = fseg;
    c.B = a.B; c.T = a.T; c.N = a.N; c.nseg = L.nseg; c.seglen = L.seglen;
    c.slabs = ssm_slabs(a.K, a.V);
    c.DA = (int)a.K; c.DC = (int)a.V; c.w_in = 1;
    c.vec = vk && vv;
    if ((err = launch_ssm_contrib(c, in_dtype, stream)) != hipSuccess) return err;
    err = launch_ssm_segscan({{{hseg, a.H0, a.HT, false}, {}}}, fseg, a.B * a.N, L.nseg, a.K * a.V,
                             stream);
    if (err != hipSuccess) return err;
    start = hseg;
  }
  SsmSweepArgs s{};
  s.a = a.q; s.b = a.k; s.c = a.v;
  s.a_grp = grp; s.b_grp = grp; s.c_grp = 1; s.e_grp = 1;
  s.cum = cum; s.d = d; s.skip = a.w_r;
  s.out = a.y;
  s.state0 = start;
  s.stateT = L.nseg > 1 ? nullptr : a.HT;
  s.B = a.B; s.T = a.T; s.N = a.N; s.nseg = L.nseg; s.seglen = L.seglen;
  s.slabs = ssm_slabs(a.K, a.V);
  s.DA = (int)a.K; s.DC = (int)a.V;
  s.a_stride = (int)a.V; s.c_stride = 1;
  s.mode = ssm::kY;
  s.vec = vk && vv && ssm_vec_rows(a.q, a.NQ, a.K, E) && ssm_vec_rows(a.y, a.N, a.V, E);
  return launch_ssm_sweep(s, in_dtype, stream);
}

}  // namespace m2rnn
