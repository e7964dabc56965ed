// The short causal convolution with a history that is carried between calls (prompts in
// pieces, truncated training windows, single tokens):
//     u_t[c] = bias[c] + sum_{i<4} w[c][i] x_{t-3+i}[c],  out = SiLU(u),  x_{-3..-1} = hist.
// All kernels are bound by HBM: threads take four consecutive channels (one where C or an address
// does not allow it), slide the last inputs through registers over a run of time steps, fetch them a
// group of steps ahead, and read and write each tensor once (runs overlap by three steps, the
// backward's by six).  At B = 4, T = 16384, C = 1024 in bf16 the forward takes 50 us (268 MB, 5.3
// TB/s, what a copy reaches) and the backward 84 us (403 MB, 4.8 TB/s); one token of 512 sequences 4 us.
// Eight channels (16 bytes of bf16) took 56 us forward, 104 backward and 4.7 us for the token: taps,
// sums and sliding inputs take up to 24 registers a channel, and half the waves are there to wait.
#include <type_traits>

#include "m2rnn_io.h"
#include "m2rnn_serving_internal.h"

namespace m2rnn {

namespace {

constexpr int kRunFwd = 16;  // time steps per thread, forward
constexpr int kRunBwd = 32;  // and backward
constexpr int kGroup = 4;    // of them fetched at a time
constexpr int kRunsPerGroup = 4;  // runs (one per wave) whose sums a backward workgroup joins

template <int VEC>
struct Taps {
  float w[4][VEC], bias[VEC];
  __device__ __forceinline__ void load(const float* wp, const float* bp, int64_t c) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i][k] = wp[(c + k) * 4 + i];
      bias[k] = bp ? bp[c + k] : 0.0f;
    }
  }
  __device__ __forceinline__ float u(int k, float m3, float m2, float m1, float x) const {
    return __builtin_fmaf(w[3][k], x, __builtin_fmaf(w[2][k], m1, __builtin_fmaf(w[1][k], m2,
                          __builtin_fmaf(w[0][k], m3, bias[k]))));
  }
};

// x_t of a sequence for t >= -3: the history holds t = -3 .. -1 (zero without one)
template <typename IoT, int VEC>
__device__ __forceinline__ io::Vals<VEC> at(const IoT* x, const IoT* hist, int64_t t, int64_t C) {
  if (t >= 0) return io::load<VEC>(x + t * C);
  if (hist) return io::load<VEC>(hist + (t + 3) * C);
  io::Vals<VEC> z;
#pragma unroll
  for (int k = 0; k < VEC; ++k) z.x[k] = 0.0f;
  return z;
}

// A wave per run of 16 steps and 256 channels.  Runs of 32 take 49 us at the size above, but 9.3
// instead of 6.9 at B = 1, T = 4096; without the fetch a group ahead 58 and 11.
template <typename IoT, int VEC>
__global__ void __launch_bounds__(256) m2rnn_conv_carry_kernel(const CarryArgs g, int64_t runs) {
  const int64_t Cv = g.C / VEC, cblocks = (Cv + 63) / 64;
  // a wave per (b, run, 64 pieces of channels), channels fastest
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t row = wid / cblocks;
  const int64_t cv = wid % cblocks * 64 + (threadIdx.x & 63);
  if (row >= g.B * runs || cv >= Cv) return;
  const int64_t c = cv * VEC, b = row / runs, t0 = row % runs * kRunFwd;
  const int64_t t1 = t0 + kRunFwd < g.T ? t0 + kRunFwd : g.T;
  Taps<VEC> tp;
  tp.load(g.w, g.bias, c);
  const IoT* x = (const IoT*)g.x + b * g.T * g.C + c;
  const IoT* hist = g.hist ? (const IoT*)g.hist + b * 3 * g.C + c : nullptr;
  IoT* out = (IoT*)g.out + b * g.T * g.C + c;
  io::Vals<VEC> m3 = at<IoT, VEC>(x, hist, t0 - 3, g.C), m2 = at<IoT, VEC>(x, hist, t0 - 2, g.C),
                m1 = at<IoT, VEC>(x, hist, t0 - 1, g.C);
  auto step = [&](int64_t t, const io::Vals<VEC>& xt) {
    io::Vals<VEC> o;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float u = tp.u(k, m3.x[k], m2.x[k], m1.x[k], xt.x[k]);
      o.x[k] = u * io::sigmoid(u);
    }
    io::store<VEC>(out + t * g.C, o);
    m3 = m2;
    m2 = m1;
    m1 = xt;
  };
  // groups of steps, fetched one group ahead, without branches (a load in a branch would be waited
  // for at its end; rows past the sequence's end are its last row's)
  const int64_t last = g.T - 1;
  io::Raw<IoT, VEC> xr[kGroup];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) xr[i].load(x + (t + i < last ? t + i : last) * g.C);
  };
  fetch(t0);
  int64_t t = t0;
  for (; t + kGroup <= t1; t += kGroup) {
    io::Vals<VEC> xv[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) xv[i] = xr[i].vals();
    fetch(t + kGroup);
#pragma unroll
    for (int i = 0; i < kGroup; ++i) step(t + i, xv[i]);
  }
  for (; t < t1; ++t) step(t, io::load<VEC>(x + t * g.C));
  if (g.hist_out && t0 == 0) {  // the last three inputs of the first len ones (bf16 widens and
                                // rounds back exactly)
    int64_t len = g.lens ? (int64_t)g.lens[b] : g.T;
    len = len < 0 ? 0 : len > g.T ? g.T : len;
    IoT* ho = (IoT*)g.hist_out + b * 3 * g.C + c;
#pragma unroll
    for (int i = 0; i < 3; ++i) io::store<VEC>(ho + i * g.C, at<IoT, VEC>(x, hist, len - 3 + i, g.C));
  }
}

// du_t = dout_t SiLU'(u_t) for the run and the three steps after it; dx_s = sum_i w[i] du_{s+3-i}
// follows three steps behind.  The run that starts a sequence also gives dhist (s < 0).  Sums of
// du_t x_{t-3+i} and du_t over the four waves' runs go to part[group][5][C].  Runs of 64 steps instead
// of 32 take 90 us at the size above and 23 instead of 16 at B = 1, T = 4096; without the fetch a
// group ahead (and with eight channels) it was 114.
template <typename IoT, int VEC>
__global__ void __launch_bounds__(256)
    m2rnn_conv_carry_bwd_kernel(const CarryArgs g, int64_t runs, float* __restrict__ part) {
  __shared__ float red[kRunsPerGroup][64 * VEC];
  const int64_t Cv = g.C / VEC, cblocks = (Cv + 63) / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t grp = blockIdx.x / cblocks;
  const int64_t row = grp * kRunsPerGroup + wave;
  const int64_t cv = blockIdx.x % cblocks * 64 + lane;
  const bool live = row < g.B * runs && cv < Cv;
  float s[5][VEC];
#pragma unroll
  for (int i = 0; i < 5; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[i][k] = 0.0f;
  if (live) {
    const int64_t c = cv * VEC, b = row / runs, t0 = row % runs * kRunBwd;
    const int64_t t1 = t0 + kRunBwd < g.T ? t0 + kRunBwd : g.T;
    Taps<VEC> tp;
    tp.load(g.w, g.bias, c);
    const IoT* x = (const IoT*)g.x + b * g.T * g.C + c;
    const IoT* hist = g.hist ? (const IoT*)g.hist + b * 3 * g.C + c : nullptr;
    const IoT* dout = (const IoT*)g.dout + b * g.T * g.C + c;
    IoT* dx = (IoT*)g.dx + b * g.T * g.C + c;
    IoT* dh = g.dhist ? (IoT*)g.dhist + b * 3 * g.C + c : nullptr;
    io::Vals<VEC> m3 = at<IoT, VEC>(x, hist, t0 - 3, g.C), m2 = at<IoT, VEC>(x, hist, t0 - 2, g.C),
                  m1 = at<IoT, VEC>(x, hist, t0 - 1, g.C);
    float d3[VEC], d2[VEC], d1[VEC];  // du_{t-3}, du_{t-2}, du_{t-1}
#pragma unroll
    for (int k = 0; k < VEC; ++k) d3[k] = d2[k] = d1[k] = 0.0f;
    // One step: of the run (OWN), or behind it, where du is zero past the sequence's end; FIRST: of
    // the first three, whose dx is another run's or the history's
    auto step = [&](auto own, auto first, int64_t t, const io::Vals<VEC>& xt, const io::Vals<VEC>& go) {
      float du[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float u = tp.u(k, m3.x[k], m2.x[k], m1.x[k], xt.x[k]);
        const float sg = io::sigmoid(u);
        du[k] = go.x[k] * sg * __builtin_fmaf(u, 1.0f - sg, 1.0f);
        if constexpr (decltype(own)::value) {
          s[0][k] = __builtin_fmaf(du[k], m3.x[k], s[0][k]);
          s[1][k] = __builtin_fmaf(du[k], m2.x[k], s[1][k]);
          s[2][k] = __builtin_fmaf(du[k], m1.x[k], s[2][k]);
          s[3][k] = __builtin_fmaf(du[k], xt.x[k], s[3][k]);
          s[4][k] += du[k];
        } else {
          du[k] = t < g.T ? du[k] : 0.0f;
        }
      }
      m3 = m2;
      m2 = m1;
      m1 = xt;
      // dx_{t-3} = w3 du_{t-3} + w2 du_{t-2} + w1 du_{t-1} + w0 du_t
      io::Vals<VEC> o;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        o.x[k] = __builtin_fmaf(tp.w[0][k], du[k], __builtin_fmaf(tp.w[1][k], d1[k],
                 __builtin_fmaf(tp.w[2][k], d2[k], tp.w[3][k] * d3[k])));
        d3[k] = d2[k];
        d2[k] = d1[k];
        d1[k] = du[k];
      }
      const int64_t sx = t - 3;
      if constexpr (decltype(first)::value) {
        if (sx >= t0) io::store<VEC>(dx + sx * g.C, o);
        else if (t0 == 0 && dh) io::store<VEC>(dh + (sx + 3) * g.C, o);
      } else {
        io::store<VEC>(dx + sx * g.C, o);
      }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    static_assert(kGroup >= 3, "the first group holds all steps whose dx is not the run's");
    // groups of steps, fetched one group ahead as in the forward
    const int64_t last = g.T - 1;
    io::Raw<IoT, VEC> xr[kGroup], gr[kGroup];
    auto fetch = [&](int64_t t) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int64_t r = (t + i < last ? t + i : last) * g.C;
        xr[i].load(x + r);
        gr[i].load(dout + r);
      }
    };
    auto group = [&](auto first, int64_t t) {
      io::Vals<VEC> xv[kGroup], gv[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        xv[i] = xr[i].vals();
        gv[i] = gr[i].vals();
      }
      fetch(t + kGroup);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) step(Yes{}, first, t + i, xv[i], gv[i]);
    };
    fetch(t0);
    int64_t t = t0;
    if (t + kGroup <= t1) {
      group(Yes{}, t);
      for (t += kGroup; t + kGroup <= t1; t += kGroup) group(No{}, t);
    }
    for (; t < t1; ++t)  // what a sequence's last run has left
      step(Yes{}, Yes{}, t, io::load<VEC>(x + t * g.C), io::load<VEC>(dout + t * g.C));
    for (; t < t1 + 3; ++t) {
      const int64_t r = (t < last ? t : last) * g.C;
      step(No{}, Yes{}, t, io::load<VEC>(x + r), io::load<VEC>(dout + r));
    }
  }
  const int64_t c0 = blockIdx.x % cblocks * 64 * VEC;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int k = 0; k < VEC; ++k) red[wave][lane * VEC + k] = s[i][k];
    __syncthreads();
    for (int col = threadIdx.x; col < 64 * VEC; col += 256)
      if (c0 + col < g.C)
        part[(grp * 5 + i) * g.C + c0 + col] = (red[0][col] + red[1][col]) + (red[2][col] + red[3][col]);
  }
}

// Sums over the groups: dw[c][i] and dbias[c].  64 columns per workgroup of sixteen waves, each
// taking every sixteenth row of part, joined in order.
__global__ void __launch_bounds__(1024)
    m2rnn_conv_carry_sum_kernel(int64_t P, int64_t C, const float* __restrict__ part,
                                float* __restrict__ dw, float* __restrict__ dbias) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;  // k C + c
  float sum = 0.0f;
  if (col < 5 * C) {
#pragma unroll 8
    for (int64_t p = wave; p < P; p += 16) sum += part[p * 5 * C + col];
  }
  red[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || col >= 5 * C) return;
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) total += (double)red[i][lane];
  const int64_t k = col / C, c = col % C;
  if (k < 4) dw[c * 4 + k] = (float)total;
  else if (dbias) dbias[c] = (float)total;
}

// One token of every sequence: the history shifts by one in place.
template <typename IoT, int VEC>
__global__ void __launch_bounds__(256) m2rnn_conv_step_kernel(const CarryArgs g) {
  const int64_t Cv = g.C / VEC;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= g.B * Cv) return;
  const int64_t b = i / Cv, c = i % Cv * VEC;
  IoT* h = (IoT*)g.hist_out + b * 3 * g.C + c;
  const io::Vals<VEC> m3 = io::load<VEC>(h), m2 = io::load<VEC>(h + g.C), m1 = io::load<VEC>(h + 2 * g.C),
                      x = io::load<VEC>((const IoT*)g.x + b * g.C + c);
  Taps<VEC> tp;
  tp.load(g.w, g.bias, c);
  io::Vals<VEC> o;
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const float u = tp.u(k, m3.x[k], m2.x[k], m1.x[k], x.x[k]);
    o.x[k] = u * io::sigmoid(u);
  }
  io::store<VEC>((IoT*)g.out + b * g.C + c, o);
  io::store<VEC>(h, m2);
  io::store<VEC>(h + g.C, m1);
  io::store<VEC>(h + 2 * g.C, x);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename IoT, int VEC>
hipError_t fwd(const CarryArgs& g, hipStream_t stream) {
  const int64_t runs = ceil_div(g.T, kRunFwd), waves = g.B * runs * ceil_div(g.C / VEC, 64);
  hipLaunchKernelGGL((m2rnn_conv_carry_kernel<IoT, VEC>), dim3((unsigned)ceil_div(waves, 4)),
                     dim3(256), 0, stream, g, runs);
  return hipGetLastError();
}
template <typename IoT, int VEC>
hipError_t bwd(const CarryArgs& g, hipStream_t stream) {
  const int64_t runs = ceil_div(g.T, kRunBwd), groups = ceil_div(g.B * runs, kRunsPerGroup);
  hipLaunchKernelGGL((m2rnn_conv_carry_bwd_kernel<IoT, VEC>),
                     dim3((unsigned)(groups * ceil_div(g.C / VEC, 64))), dim3(256), 0, stream, g,
                     runs, g.ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(m2rnn_conv_carry_sum_kernel, dim3((unsigned)ceil_div(5 * g.C, 64)), dim3(1024),
                     0, stream, groups, g.C, g.ws, g.dw, g.dbias);
  return hipGetLastError();
}
template <typename IoT, int VEC>
hipError_t one(const CarryArgs& g, hipStream_t stream) {
  hipLaunchKernelGGL((m2rnn_conv_step_kernel<IoT, VEC>),
                     dim3((unsigned)ceil_div(g.B * (g.C / VEC), 256)), dim3(256), 0, stream, g);
  return hipGetLastError();
}
template <typename IoT>
hipError_t pick(const CarryArgs& g, int what, hipStream_t stream) {
  uintptr_t all = 0;
  for (const void* p : {g.x, g.hist, (const void*)g.out, (const void*)g.hist_out, g.dout,
                        (const void*)g.dx, (const void*)g.dhist})
    all |= (uintptr_t)p;
  const bool vec = g.C % 4 == 0 && all % (4 * sizeof(IoT)) == 0;
  if (what == 0) return vec ? fwd<IoT, 4>(g, stream) : fwd<IoT, 1>(g, stream);
  if (what == 1) return vec ? bwd<IoT, 4>(g, stream) : bwd<IoT, 1>(g, stream);
  return vec ? one<IoT, 4>(g, stream) : one<IoT, 1>(g, stream);
}

}  // namespace

size_t conv_carry_workspace_floats(int64_t B, int64_t T, int64_t C) {
  return (size_t)ceil_div(B * ceil_div(T, kRunBwd), kRunsPerGroup) * 5 * (size_t)C;
}

hipError_t launch_conv_carry(const CarryArgs& g, int io_dtype, int what, hipStream_t stream) {
  return io_dtype == kBF16 ? pick<uint16_t>(g, what, stream) : pick<float>(g, what, stream);
}

}  // namespace m2rnn
