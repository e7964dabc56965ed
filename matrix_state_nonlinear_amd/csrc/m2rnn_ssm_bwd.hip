// Backward of the selective state-space scan: the host side of the sweeps for dq, dv
// and dk (m2rnn_ssm_sweep.h), and the kernels for what is left.
//
// The sweeps return, per token, the parts of the decays' gradient inside a chunk (X_t, the sum of
// M over the pairs around t) and those of the carried states (a_t, b_t; m2rnn_ssm_sweep.h has
// the definitions).  The part g = 2^{c_L} <H0, G> that passes through the whole chunk follows from
// w = <state, state gradient> at the chunk's end, w_end = sum b + g, or its start, w_start = sum a +
// g: from the segment's end, where w is a dot product, backwards, and from its start, the end of
// the segment before, forwards.  Each chunk adds the rounding of its sums to the one and the other;
// g is their mean weighted against that (dalpha 3.0e-6 off from the end alone, 1.2e-6 so).  Then
//     dl_t = X_t + sum_{i >= t} a_i + sum_{j < t} b_j + g,
//     dlogit = sigmoid(x) (dd - alpha dl),  d dd = sum_i M_it + b_t.
// These sums are kept in double.  Where the chunk's decay is below kNoPass, g is below what
// w_end - sum b is rounded by, and is left out: the difference would add the same error to all the
// chunk's tokens (with it dalpha at B = 16, T = 4096, 16 heads was more than twice as far off).
//
// B = 16, T = 4096, 16 heads, K = 32, V = 128, bf16: the call takes 0.9 ms; under the profiler, which
// stretches them by a tenth, decays 12 us, the states' two first passes 82 and 84, their scans 28, dq 315,
// dv 244, dk 264, the decays' gradient 27, parameters 7.
#include "m2rnn_ssm_sweep.h"

namespace m2rnn {

namespace {

// Tokens per segment at most: the decays' gradient carries w from chunk to chunk inside a segment,
// and its error with it (at B = 16, T = 4096, 16 heads, K = 32, V = 128 dalpha and dbeta are 1.2e-6
// and 3e-7 off with 512, 2.5e-6 and 8e-7 with 1024; forward and backward take 1.19 and 1.13 ms).
constexpr int64_t kMaxSeg = 512;
constexpr int kMaxChunks = 16;  // of 32 tokens
constexpr double kNoPass = 15.0;  // -log of 3e-7

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t pad64(size_t x) { return align_up(x, 64); }

// One workgroup per (b, n, segment), a wave per chunk of `L` tokens (as in the sweeps): the sums
// inside the chunks all at once, then every wave follows w from the segment's end to its chunk.
// Bound by the latency of its few loads per thread (27 us for 25 MB at the size above).
__global__ void __launch_bounds__(64 * kMaxChunks)
    m2rnn_ssm_dgate_kernel(int64_t B, int64_t T, int64_t N, int64_t nseg, int64_t seglen, int L,
                           int slabs, int vslabs, const float* __restrict__ adot,
                           const float* __restrict__ bdot, const float* __restrict__ pairs,
                           const float* __restrict__ colpairs, const double* __restrict__ base,
                           bool from_zero, const float* __restrict__ logit,
                           const float* __restrict__ alpha, const float* __restrict__ beta,
                           float* __restrict__ dlogit, float* __restrict__ part) {
  __shared__ double tot[3][kMaxChunks];  // per chunk: sums of a and b, and its -log f in all
  __shared__ double red[2][kMaxChunks];
  // heads fastest: neighbouring workgroups share lines of logit and dlogit
  const int64_t unit = blockIdx.x;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = unit % N, seg = unit / N % nseg, b = unit / N / nseg;
  const int64_t bn = b * N + n;
  const int64_t t0 = seg * seglen, t1 = t0 + seglen < T ? t0 + seglen : T;
  const int nch = (int)((t1 - t0 + L - 1) / L);
  const int64_t c = t0 + (int64_t)w * L;
  // lane 0 has the chunk's last token
  const int len = c < t1 ? (int)(t1 - c < L ? t1 - c : L) : 0;
  const int64_t t = c + len - 1 - lane;
  const bool ok = lane < len;
  const double al = (double)alpha[n];
  double a = 0.0, dd = 0.0, bs = 0.0, X = 0.0;
  float x = 0.0f;
  if (ok) {
    for (int s = 0; s < slabs; ++s) {
      const int64_t o = ((int64_t)s * B * N + bn) * T + t;
      a += (double)adot[o];
      bs += (double)bdot[o];
      dd += (double)colpairs[o];
      X += (double)pairs[o];
    }
    x = logit[(b * T + t) * N + n] + beta[n];
  }
  const float d = ok ? ssm::softplus(x) : 0.0f;
  dd += bs;
  // asum: a from this token on; bsum: b before this token; decay: the chunk's -log f in all
  double asum = a, bsum = bs * (double)d, decay = al * (double)d;
  const double b_own = bsum;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const double oa = __shfl_up(asum, s), ob = __shfl_down(bsum, s);
    if (lane >= s) asum += oa;
    if (lane + s < 64) bsum += ob;
    decay += __shfl_xor(decay, s);
  }
  if (lane == 0) {
    tot[1][w] = bsum;
    tot[2][w] = decay;
  }
  if (lane == 63) tot[0][w] = asum;
  bsum -= b_own;
  __syncthreads();
  double w_end = 0.0, w_start = 0.0, g = 0.0, g_left = 0.0;
  if (base)
    for (int s = 0; s < vslabs; ++s) {
      const double* p = base + ((int64_t)s * B * N + bn) * nseg + seg;
      w_end += p[0];
      if (seg > 0) w_start += p[-1];
    }
  for (int k = nch - 1; k >= w; --k) {
    g = tot[2][k] > kNoPass ? 0.0 : w_end - tot[1][k];
    w_end = tot[0][k] + g;
  }
  if (seg > 0 || from_zero) {  // (w at the first token's start is not known with an initial state)
    for (int k = 0; k <= w; ++k) {
      g_left = tot[2][k] > kNoPass ? 0.0 : w_start - tot[0][k];
      w_start = tot[1][k] + g_left;
    }
    const double share = ((double)w + 0.5) / (double)nch;
    g = g * share + g_left * (1.0 - share);
  }
  double sa = 0.0, sb = 0.0;
  if (ok) {
    const double dl = X + asum + (bsum + g);
    const float ex = expf(-fabsf(x));
    const float sig = x >= 0.0f ? 1.0f / (1.0f + ex) : ex / (1.0f + ex);
    sb = (double)sig * (dd - al * dl);
    sa = -(double)d * dl;
    dlogit[(b * T + t) * N + n] = (float)sb;
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    sa += __shfl_xor(sa, s);
    sb += __shfl_xor(sb, s);
  }
  if (lane == 0) {
    red[0][w] = sa;
    red[1][w] = sb;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    double sum = 0.0;
    for (int k = 0; k < nch; ++k) sum += red[threadIdx.x][k];
    part[(bn * nseg + seg) * 2 + threadIdx.x] = (float)sum;
  }
}

// dw_r[n][x] = sum over (b, segment) of colsum[b][n][seg][x], x < V, and dalpha, dbeta from
// part[b][n][seg][2] as columns V and V + 1.  64 columns of a head per workgroup, its sixteen
// waves taking every sixteenth (b, segment), joined in a fixed order (7 us for 16 heads of 128
// (b, segment); with four waves 15).
__global__ void __launch_bounds__(1024)
    m2rnn_ssm_params_kernel(int64_t B, int64_t N, int64_t nseg, int64_t V,
                            const float* __restrict__ colsum, const float* __restrict__ part,
                            float* __restrict__ dw_r, float* __restrict__ dalpha,
                            float* __restrict__ dbeta) {
  __shared__ double red[16][64];
  const int64_t cb = (V + 2 + 63) / 64;
  const int64_t n = blockIdx.x / cb;
  const int64_t x = (blockIdx.x % cb) * 64 + (threadIdx.x & 63);
  const int grp = threadIdx.x >> 6;
  double sum = 0.0;
  if (x < V + 2) {
#pragma unroll 4
    for (int64_t r = grp; r < B * nseg; r += 16) {
      const int64_t row = (r / nseg * N + n) * nseg + r % nseg;
      sum += (double)(x < V ? colsum[row * V + x] : part[row * 2 + (x - V)]);
    }
  }
  red[grp][threadIdx.x & 63] = sum;
  __syncthreads();
  if (grp != 0 || x >= V + 2) return;
  double all = 0.0;
#pragma unroll
  for (int k = 0; k < 16; ++k) all += red[k][threadIdx.x];
  const float total = (float)all;
  if (x < V) dw_r[n * V + x] = total;
  else if (x == V) dalpha[n] = total;
  else dbeta[n] = total;
}

// Sums of shared heads: out[b t][nq][k] = sum over the group's heads of part[b t][n][k], in
// head order, for dq (blockIdx.y = 0) and dk (1).  Reads each partial once: 60 us for 270 MB
// (4.5 TB/s) at B = 2, T = 4096, 64 heads on one q and k, K = 64.
template <typename InT>
__global__ void __launch_bounds__(256)
    m2rnn_ssm_group_kernel(int64_t total, int64_t K, int grp, const float* __restrict__ part0,
                           const float* __restrict__ part1, InT* __restrict__ out0,
                           InT* __restrict__ out1) {
  const float* part = blockIdx.y ? part1 : part0;
  InT* out = blockIdx.y ? out1 : out0;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const float* p = part + i / K * grp * K + i % K;
  float sum = 0.0f;
#pragma unroll 8
  for (int h = 0; h < grp; ++h) sum += p[(int64_t)h * K];
  if constexpr (sizeof(InT) == 2) out[i] = (uint16_t)ssm::pack_rne(sum, 0.0f);
  else out[i] = sum;
}

}  // namespace

// Segments of the backward: at most kMaxSeg tokens, and as many as bring each of the three sweeps
// to about 512 workgroups, of at least 64 tokens.  Forward and backward of one window of 4096 tokens,
// 16 heads, K = V = 64: 147 us; with 256 workgroups 157, with 1024 179.
SsmLayout ssm_bwd_layout(int64_t B, int64_t T, int64_t N, int64_t NQ, int64_t K, int64_t V) {
  SsmLayout L{};
  const int64_t units = B * N, tok = T > 0 ? T : 1;
  int64_t nseg = units > 0 ? ceil_div(512, units) : 1;
  const int64_t most = tok / 64 > 1 ? tok / 64 : 1;
  if (nseg > most) nseg = most;
  if (nseg < ceil_div(tok, kMaxSeg)) nseg = ceil_div(tok, kMaxSeg);
  L.seglen = (int64_t)align_up((size_t)ceil_div(tok, nseg), 64);
  L.nseg = ceil_div(tok, L.seglen);
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off += pad64(n);
    return at;
  };
  const size_t KV = (size_t)K * V, U = (size_t)units;
  L.cum = take(U * T * 2);
  L.d = take(U * T);
  L.hseg = take(U * L.nseg * KV);
  L.gseg = take(U * L.nseg * KV);
  L.hT = take(U * KV);
  L.fseg = take(U * L.nseg);
  L.base = take(U * L.nseg * ssm_slabs(K, V) * 2);
  L.adot = take(U * T * ssm_slabs(V, K));
  L.bdot = take(U * T * ssm_slabs(V, K));
  L.pairs = take(U * T * ssm_slabs(V, K));
  L.colpairs = take(U * T * ssm_slabs(V, K));
  L.colsum = take(U * L.nseg * V);
  L.gatepart = take(U * L.nseg * 2);
  if (NQ < N) {
    L.dqp = take(U * T * K);
    L.dkp = take(U * T * K);
  }
  L.total_floats = off;
  return L;
}

hipError_t launch_ssm_bwd(const SsmArgs& a, int in_dtype, hipStream_t stream) {
  const SsmLayout L = ssm_bwd_layout(a.B, a.T, a.N, a.NQ, a.K, a.V);
  const int grp = (int)(a.N / a.NQ);
  const int64_t units = a.B * a.N, KV = a.K * a.V;
  const int E = in_dtype == kBF16 ? 2 : 4;
  const bool vk = ssm_vec_rows(a.k, a.NQ, a.K, E) && ssm_vec_rows(a.q, a.NQ, a.K, E),
             vv = ssm_vec_rows(a.v, a.N, a.V, E) && ssm_vec_rows(a.dy, a.N, a.V, E), vec = vk && vv;
  // the gradients' rows: of the input's type, or a shared head's fp32 parts
  const bool vdv = ssm_vec_rows(a.dv, a.N, a.V, E),
             vdq = grp > 1 ? ssm_vec_rows(a.ws, a.N, a.K, 4) : ssm_vec_rows(a.dq, a.N, a.K, E),
             vdk = grp > 1 ? ssm_vec_rows(a.ws, a.N, a.K, 4) : ssm_vec_rows(a.dk, a.N, a.K, E);
  double* cum = (double*)(a.ws + L.cum);
  float* d = a.ws + L.d;
  float* hseg = a.ws + L.hseg;
  float* gseg = a.ws + L.gseg;
  float* fseg = a.ws + L.fseg;
  float* hT = a.ws + L.hT;
  hipError_t err = launch_ssm_decays(a, in_dtype, cum, d, stream);
  if (err != hipSuccess) return err;

  // the state at each segment's start, and the state gradient at its end; a single segment
  // starts from H0 and, without dHT, ends at zero
  const bool passes = L.nseg > 1 || a.dHT;
  if (passes) {
    SsmContribArgs c{};
    c.cum = cum; c.d = d; c.vec = vec;
    c.B = a.B; c.T = a.T; c.N = a.N; c.nseg = L.nseg; c.seglen = L.seglen;
    c.slabs = ssm_slabs(a.K, a.V);
    c.DA = (int)a.K; c.DC = (int)a.V;
    c.b = a.k; c.c = a.v; c.b_grp = grp; c.c_grp = 1;
    c.contrib = hseg; c.fseg = fseg; c.w_in = 1;
    if ((err = launch_ssm_contrib(c, in_dtype, stream)) != hipSuccess) return err;
    c.b = a.q; c.c = a.dy;
    c.contrib = gseg; c.fseg = nullptr; c.w_in = 0; c.rev = 1;
    if ((err = launch_ssm_contrib(c, in_dtype, stream)) != hipSuccess) return err;
    err = launch_ssm_segscan({{{hseg, a.H0, hT, false}, {gseg, a.dHT, a.dH0, true}}}, fseg, units,
                             L.nseg, KV, stream);
    if (err != hipSuccess) return err;
  }

  SsmSweepArgs s{};
  s.cum = cum; s.d = d;
  s.B = a.B; s.T = a.T; s.N = a.N; s.nseg = L.nseg; s.seglen = L.seglen;

  // dq: over dy and v, from the states
  SsmSweepArgs dq = s;
  dq.a = a.dy; dq.b = a.v; dq.c = a.k; dq.e = a.q;
  dq.a_grp = 1; dq.b_grp = 1; dq.c_grp = grp; dq.e_grp = grp;
  dq.DA = (int)a.V; dq.DC = (int)a.K; dq.slabs = ssm_slabs(a.V, a.K);
  dq.a_stride = 1; dq.c_stride = (int)a.V;
  dq.state0 = passes ? hseg : a.H0;
  dq.rowdot = a.ws + L.adot;
  dq.pairs = a.ws + L.pairs;
  dq.colpairs = a.ws + L.colpairs;
  dq.colsum = a.ws + L.colsum;
  dq.mode = ssm::kDq;
  dq.out = grp > 1 ? (void*)(a.ws + L.dqp) : a.dq;
  dq.out_f32 = grp > 1;
  dq.vec = vec && vdq;
  if ((err = launch_ssm_sweep(dq, in_dtype, stream)) != hipSuccess) return err;

  // dv: over k and q in reverse, from the state gradients
  SsmSweepArgs dv = s;
  dv.a = a.k; dv.b = a.q; dv.c = a.dy;
  dv.a_grp = grp; dv.b_grp = grp; dv.c_grp = 1; dv.e_grp = 1;
  dv.DA = (int)a.K; dv.DC = (int)a.V; dv.slabs = ssm_slabs(a.K, a.V);
  dv.a_stride = (int)a.V; dv.c_stride = 1;
  dv.state0 = passes ? gseg : nullptr;
  dv.stateT = passes ? nullptr : a.dH0;
  if (passes) {
    dv.base = (double*)(a.ws + L.base);
    dv.hend = hseg;
    dv.hend_last = hT;
  }
  dv.skip = a.w_r;
  dv.mode = ssm::kDv;
  dv.out = a.dv;
  dv.vec = vec && vdv;
  if ((err = launch_ssm_sweep(dv, in_dtype, stream)) != hipSuccess) return err;

  // dk: over v and dy in reverse, from the transposed state gradients
  SsmSweepArgs dk = s;
  dk.a = a.v; dk.b = a.dy; dk.c = a.q; dk.e = a.k;
  dk.a_grp = 1; dk.b_grp = 1; dk.c_grp = grp; dk.e_grp = grp;
  dk.DA = (int)a.V; dk.DC = (int)a.K; dk.slabs = ssm_slabs(a.V, a.K);
  dk.a_stride = 1; dk.c_stride = (int)a.V;
  dk.state0 = passes ? gseg : nullptr;
  dk.rowdot = a.ws + L.bdot;
  dk.mode = ssm::kDk;
  dk.out = grp > 1 ? (void*)(a.ws + L.dkp) : a.dk;
  dk.out_f32 = grp > 1;
  dk.vec = vec && vdk;
  if ((err = launch_ssm_sweep(dk, in_dtype, stream)) != hipSuccess) return err;

  const int chunk = in_dtype == kBF16 ? ssm::Cfg<uint16_t>::L : ssm::Cfg<float>::L;
  hipLaunchKernelGGL(m2rnn_ssm_dgate_kernel, dim3((unsigned)(units * L.nseg)),
                     dim3((unsigned)(64 * ceil_div(L.seglen, chunk))), 0, stream, a.B, a.T, a.N,
                     L.nseg, L.seglen, chunk, (int)ssm_slabs(a.V, a.K), (int)ssm_slabs(a.K, a.V),
                     a.ws + L.adot, a.ws + L.bdot, a.ws + L.pairs, a.ws + L.colpairs,
                     passes ? (const double*)(a.ws + L.base) : nullptr, a.H0 == nullptr, a.logit,
                     a.alpha, a.beta, a.dlogit, a.ws + L.gatepart);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  hipLaunchKernelGGL(m2rnn_ssm_params_kernel, dim3((unsigned)(a.N * ceil_div(a.V + 2, 64))),
                     dim3(1024), 0, stream, a.B, a.N, L.nseg, a.V, a.ws + L.colsum,
                     a.ws + L.gatepart, a.dw_r, a.dalpha, a.dbeta);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  if (grp > 1) {
    const int64_t total = a.B * a.T * a.NQ * a.K;
    const dim3 grid((unsigned)ceil_div(total, 256), 2);
    if (in_dtype == kBF16)
      hipLaunchKernelGGL(m2rnn_ssm_group_kernel<uint16_t>, grid, dim3(256), 0, stream, total, a.K,
                         grp, a.ws + L.dqp, a.ws + L.dkp, (uint16_t*)a.dq, (uint16_t*)a.dk);
    else
      hipLaunchKernelGGL(m2rnn_ssm_group_kernel<float>, grid, dim3(256), 0, stream, total, a.K,
                         grp, a.ws + L.dqp, a.ws + L.dkp, (float*)a.dq, (float*)a.dk);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace m2rnn
