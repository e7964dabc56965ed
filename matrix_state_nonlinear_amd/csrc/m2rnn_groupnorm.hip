// Group norm with a SiLU gate over the channels of a token:
//     out = (gamma (.) z + beta) (.) SiLU(g_pre),  z = (y - mean) / sqrt(var + eps),
// mean and variance over each of the G groups of S = D / G consecutive channels, and its
// backward.  A row of D channels is G groups in memory order, so the tensors are [rows G, S].
// Bound by HBM: each tensor is read and written once.  A group is held by a few lanes (LG, a power
// of two, each with NCH pieces of VEC elements), mean and centred variance are exchanged between
// them, and a wave holds several groups, of several rows where a row has too few.  The backward
// keeps a wave on its columns over a run of rows, so dgamma and dbeta are sums in
// registers; their partials are joined by a second kernel in a fixed order.  65536 rows of 16 groups
// of 64 channels in bf16: forward 86 us (403 MB, 4.7 TB/s), backward 136 us (671 MB, 4.9 TB/s; a copy
// reaches 5.2) and 7 us for the partials; 512 rows 4 us.
#include "m2rnn_io.h"
#include "m2rnn_serving_internal.h"

namespace m2rnn {

namespace {

__device__ __forceinline__ float group_sum(float x, int lg) {
  for (int s = 1; s < lg; s *= 2) x += __shfl_xor(x, s);
  return x;
}

// Where a wave's lanes sit: lane = (row of the pass, group, lane of the group).
struct Place {
  int l, grp, row;
  __device__ __forceinline__ Place(const GroupNormArgs& g) {
    const int lane = threadIdx.x & 63;
    l = lane & (g.lg - 1);
    grp = lane / g.lg & (g.gw - 1);
    row = lane / (g.lg * g.gw);
  }
};

template <typename IoT, int VEC, int NCH>
struct Piece {
  io::Vals<VEC> v[NCH];
  __device__ __forceinline__ void load(const IoT* p, int l, int lg, int S) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * lg + l) * VEC;
      if (j < S) v[c] = io::load<VEC>(p + j);
    }
  }
};

// mean and 1 / sqrt(var + eps) of a group, and y centred in place
template <typename IoT, int VEC, int NCH>
__device__ __forceinline__ float normalise(Piece<IoT, VEC, NCH>& y, const GroupNormArgs& g, int l) {
  const int S = (int)g.S;
  const float inv = 1.0f / (float)S;
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
    if ((c * g.lg + l) * VEC < S)
#pragma unroll
      for (int k = 0; k < VEC; ++k) sum += y.v[c].x[k];
  const float mean = group_sum(sum, g.lg) * inv;
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
    if ((c * g.lg + l) * VEC < S)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        y.v[c].x[k] -= mean;
        sq = __builtin_fmaf(y.v[c].x[k], y.v[c].x[k], sq);
      }
  return 1.0f / sqrtf(group_sum(sq, g.lg) * inv + g.eps);
}

// blockIdx.x * 4 + wave = (row block, column block of gw groups), columns fastest
template <typename IoT, int VEC, int NCH>
__global__ void __launch_bounds__(256) m2rnn_groupnorm_gate_kernel(const GroupNormArgs g) {
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t cblocks = (g.G + g.gw - 1) / g.gw;
  const Place p(g);
  const int64_t grp = wid % cblocks * g.gw + p.grp;
  const int rp = 64 / (g.lg * g.gw);  // rows per pass
  const int64_t r0 = wid / cblocks * g.rows_per;
  const int64_t r1 = r0 + g.rows_per < g.rows ? r0 + g.rows_per : g.rows;
  const int S = (int)g.S;
  if (grp >= g.G || r0 >= g.rows) return;  // whole groups of lanes
  Piece<float, VEC, NCH> gam, bet;
  gam.load(g.gamma + grp * S, p.l, g.lg, S);
  bet.load(g.beta + grp * S, p.l, g.lg, S);
  for (int64_t r = r0 + p.row; r < r1; r += rp) {
    const int64_t at = (r * g.G + grp) * S;
    Piece<IoT, VEC, NCH> y, gp;
    y.load((const IoT*)g.y + at, p.l, g.lg, S);
    gp.load((const IoT*)g.g_pre + at, p.l, g.lg, S);
    const float rs = normalise(y, g, p.l);
    IoT* o = (IoT*)g.out + at;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * g.lg + p.l) * VEC;
      if (j < S) {
        io::Vals<VEC> x;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float a = __builtin_fmaf(gam.v[c].x[k], y.v[c].x[k] * rs, bet.v[c].x[k]);
          x.x[k] = a * gp.v[c].x[k] * io::sigmoid(gp.v[c].x[k]);
        }
        io::store<VEC>(o + j, x);
      }
    }
  }
}

// With a = gamma z + beta, da = dout SiLU(g_pre), dz = da gamma:
//     dy = rs (dz - mean(dz) - z mean(dz z)),  dg_pre = dout a SiLU'(g_pre),
//     dgamma = sum_rows da z,  dbeta = sum_rows da.
// The four waves of a workgroup take the same columns of four neighbouring row blocks.
template <typename IoT, int VEC, int NCH>
__global__ void __launch_bounds__(256) m2rnn_groupnorm_gate_bwd_kernel(const GroupNormArgs g) {
  __shared__ float red[4][2][64 * VEC * NCH];
  const int wave = threadIdx.x >> 6;
  const int64_t cblocks = (g.G + g.gw - 1) / g.gw;
  const Place p(g);
  const int64_t grp = blockIdx.x % cblocks * g.gw + p.grp, quad = blockIdx.x / cblocks;
  const int64_t rb = quad * 4 + wave;
  const int rp = 64 / (g.lg * g.gw);
  const int64_t r0 = rb * g.rows_per;
  const int64_t r1 = r0 + g.rows_per < g.rows ? r0 + g.rows_per : g.rows;
  const int S = (int)g.S;
  const bool live = grp < g.G;  // (a wave behind the last row has nothing to add)
  const float inv = 1.0f / (float)S;
  Piece<float, VEC, NCH> gam, bet;
  if (live) {
    gam.load(g.gamma + grp * S, p.l, g.lg, S);
    bet.load(g.beta + grp * S, p.l, g.lg, S);
  }
  float sg[NCH][VEC], sb[NCH][VEC];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int k = 0; k < VEC; ++k) sg[c][k] = sb[c][k] = 0.0f;
  for (int64_t r = r0 + p.row; live && r < r1; r += rp) {
    const int64_t at = (r * g.G + grp) * S;
    Piece<IoT, VEC, NCH> y, gp, go;
    y.load((const IoT*)g.y + at, p.l, g.lg, S);
    gp.load((const IoT*)g.g_pre + at, p.l, g.lg, S);
    go.load((const IoT*)g.dout + at, p.l, g.lg, S);
    const float rs = normalise(y, g, p.l);
    IoT* dg = (IoT*)g.dg_pre + at;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * g.lg + p.l) * VEC;
      if (j < S) {
        io::Vals<VEC> x;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float z = y.v[c].x[k] * rs, gv = gp.v[c].x[k], d = go.v[c].x[k];
          const float a = __builtin_fmaf(gam.v[c].x[k], z, bet.v[c].x[k]);
          const float sig = io::sigmoid(gv);
          const float da = d * gv * sig;
          x.x[k] = d * a * sig * __builtin_fmaf(gv, 1.0f - sig, 1.0f);
          sg[c][k] = __builtin_fmaf(da, z, sg[c][k]);
          sb[c][k] += da;
          const float dz = da * gam.v[c].x[k];
          s1 += dz;
          s2 = __builtin_fmaf(dz, z, s2);
          y.v[c].x[k] = z;
          go.v[c].x[k] = dz;
        }
        io::store<VEC>(dg + j, x);
      }
    }
    s1 = group_sum(s1, g.lg) * inv;
    s2 = group_sum(s2, g.lg) * inv;
    IoT* dy = (IoT*)g.dy + at;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * g.lg + p.l) * VEC;
      if (j < S) {
        io::Vals<VEC> x;
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          x.x[k] = rs * (go.v[c].x[k] - s1 - y.v[c].x[k] * s2);
        io::store<VEC>(dy + j, x);
      }
    }
  }
  // join the pass's rows, then the four waves: one partial per workgroup, part[quad][2][D]
  const int lanes = g.lg * g.gw;  // that hold different columns
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      for (int s = lanes; s < 64; s *= 2) {
        sg[c][k] += __shfl_xor(sg[c][k], s);
        sb[c][k] += __shfl_xor(sb[c][k], s);
      }
      const int i = ((threadIdx.x & 63) * NCH + c) * VEC + k;
      red[wave][0][i] = sg[c][k];
      red[wave][1][i] = sb[c][k];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < lanes * NCH * VEC; i += 256) {
    const int lane = i / (NCH * VEC), c = i / VEC % NCH, k = i % VEC;
    const int64_t gr = blockIdx.x % cblocks * g.gw + lane / g.lg;
    const int j = (c * g.lg + lane % g.lg) * VEC + k;
    if (gr < g.G && j < S) {
      float* o = g.ws + quad * 2 * g.G * S + gr * S + j;
      o[0] = (red[0][0][i] + red[1][0][i]) + (red[2][0][i] + red[3][0][i]);
      o[g.G * S] = (red[0][1][i] + red[1][1][i]) + (red[2][1][i] + red[3][1][i]);
    }
  }
}

// Groups too wide for a wave's registers: one workgroup per (group, run of rows), each
// tensor read again for each of the passes over a row.  Backward sums are kept in the partial.
template <typename IoT, bool BWD>
__global__ void __launch_bounds__(256) m2rnn_groupnorm_wide_kernel(const GroupNormArgs g) {
  __shared__ float red[2][4];
  const int64_t grp = blockIdx.x % g.G, rb = blockIdx.x / g.G;
  const int64_t S = g.S, r0 = rb * g.rows_per;
  const int64_t r1 = r0 + g.rows_per < g.rows ? r0 + g.rows_per : g.rows;
  const float inv = 1.0f / (float)S;
  const float* gam = g.gamma + grp * S;
  const float* bet = g.beta + grp * S;
  float* pg = g.ws + rb * 2 * g.G * S + grp * S;
  float* pb = pg + g.G * S;
  auto both = [&](float a, float b, float& A, float& B) {
    for (int s = 1; s < 64; s *= 2) {
      a += __shfl_xor(a, s);
      b += __shfl_xor(b, s);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      red[0][threadIdx.x >> 6] = a;
      red[1][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    A = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
    B = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  };
  for (int64_t r = r0; r < r1; ++r) {
    const int64_t at = (r * g.G + grp) * S;
    const IoT* y = (const IoT*)g.y + at;
    const IoT* gp = (const IoT*)g.g_pre + at;
    const IoT* go = BWD ? (const IoT*)g.dout + at : nullptr;
    float sum = 0.0f, mean, sq = 0.0f, var, none;
    for (int64_t j = threadIdx.x; j < S; j += 256) sum += load_in(y + j);
    both(sum, 0.0f, mean, none);
    mean *= inv;
    for (int64_t j = threadIdx.x; j < S; j += 256) {
      const float c = load_in(y + j) - mean;
      sq = __builtin_fmaf(c, c, sq);
    }
    both(sq, 0.0f, var, none);
    const float rs = 1.0f / sqrtf(var * inv + g.eps);
    if constexpr (!BWD) {
      for (int64_t j = threadIdx.x; j < S; j += 256) {
        const float gv = load_in(gp + j);
        const float a = __builtin_fmaf(gam[j], (load_in(y + j) - mean) * rs, bet[j]);
        io::store<1>((IoT*)g.out + at + j, io::Vals<1>{a * gv * io::sigmoid(gv)});
      }
    } else {
      float s1 = 0.0f, s2 = 0.0f, S1, S2;
      for (int64_t j = threadIdx.x; j < S; j += 256) {
        const float z = (load_in(y + j) - mean) * rs, gv = load_in(gp + j), d = load_in(go + j);
        const float a = __builtin_fmaf(gam[j], z, bet[j]), sig = io::sigmoid(gv), da = d * gv * sig;
        io::store<1>((IoT*)g.dg_pre + at + j,
                     io::Vals<1>{d * a * sig * __builtin_fmaf(gv, 1.0f - sig, 1.0f)});
        pg[j] = (r == r0 ? 0.0f : pg[j]) + da * z;
        pb[j] = (r == r0 ? 0.0f : pb[j]) + da;
        s1 = __builtin_fmaf(da, gam[j], s1);
        s2 = __builtin_fmaf(da * gam[j], z, s2);
      }
      both(s1, s2, S1, S2);
      for (int64_t j = threadIdx.x; j < S; j += 256) {
        const float z = (load_in(y + j) - mean) * rs, gv = load_in(gp + j), d = load_in(go + j);
        const float dz = d * gv * io::sigmoid(gv) * gam[j];
        io::store<1>((IoT*)g.dy + at + j, io::Vals<1>{rs * (dz - S1 * inv - z * (S2 * inv))});
      }
    }
  }
}

// dgamma and dbeta: sums over the row blocks of part[rb][2 D], sixteen waves each taking
// every sixteenth block, joined in order.
__global__ void __launch_bounds__(1024)
    m2rnn_groupnorm_sum_kernel(int64_t P, int64_t D, const float* __restrict__ part,
                               float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (col < 2 * D) {
#pragma unroll 8
    for (int64_t p = wave; p < P; p += 16) sum += part[p * 2 * D + col];
  }
  red[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || col >= 2 * D) return;
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) total += (double)red[i][lane];
  if (col < D) dgamma[col] = (float)total;
  else dbeta[col - D] = (float)total;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes, groups and rows of a wave for pieces of `vec` elements; pieces per lane (0: too wide).
struct Plan {
  int lg, gw, nch;
  int64_t rows_per, blocks;  // rows per wave (per workgroup when too wide), row blocks
  int64_t parts;             // partials of the backward
};
Plan plan(int64_t rows, int64_t G, int64_t S, int vec, bool bwd) {
  Plan p{1, 1, 0, 1, 1, 1};
  const int64_t pieces = ceil_div(S, vec);
  while (p.lg < 64 && p.lg < pieces) p.lg *= 2;
  const int64_t nch = ceil_div(pieces, p.lg);
  int64_t waves;  // that work on one row block
  if (nch <= 4) {
    p.nch = nch == 1 ? 1 : nch == 2 ? 2 : 4;
    while (p.gw * p.lg < 64 && p.gw < G) p.gw *= 2;
    waves = ceil_div(G, p.gw);
  } else {
    waves = G;
  }
  const int rp = p.nch ? 64 / (p.lg * p.gw) : 1;
  // the forward amortises gamma and beta over a few rows, the backward its partials over more: as
  // many rows per wave as leave 8192 waves (8 per SIMD), within these limits
  const int64_t most = bwd ? 128 : 8;
  int64_t per = ceil_div(rows * waves, 8192 * (int64_t)rp);
  per = per < 1 ? 1 : per > most ? most : per;
  p.rows_per = per * rp;
  p.blocks = ceil_div(rows, p.rows_per);
  p.parts = p.nch ? ceil_div(p.blocks, 4) : p.blocks;
  return p;
}

template <typename IoT, int VEC, int NCH>
hipError_t run(const GroupNormArgs& g, bool bwd, int64_t blocks, hipStream_t stream) {
  const int64_t cblocks = ceil_div(g.G, g.gw);
  if (bwd)
    hipLaunchKernelGGL((m2rnn_groupnorm_gate_bwd_kernel<IoT, VEC, NCH>),
                       dim3((unsigned)(ceil_div(blocks, 4) * cblocks)), dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL((m2rnn_groupnorm_gate_kernel<IoT, VEC, NCH>),
                       dim3((unsigned)ceil_div(blocks * cblocks, 4)), dim3(256), 0, stream, g);
  return hipGetLastError();
}
template <typename IoT, int VEC>
hipError_t pick(GroupNormArgs g, bool bwd, hipStream_t stream) {
  const Plan p = plan(g.rows, g.G, g.S, VEC, bwd);
  g.lg = p.lg;
  g.gw = p.gw;
  g.rows_per = p.rows_per;
  hipError_t e;
  if (p.nch == 1) e = run<IoT, VEC, 1>(g, bwd, p.blocks, stream);
  else if (p.nch == 2) e = run<IoT, VEC, 2>(g, bwd, p.blocks, stream);
  else if (p.nch == 4) e = run<IoT, VEC, 4>(g, bwd, p.blocks, stream);
  else {
    const dim3 grid((unsigned)(p.blocks * g.G));
    if (bwd)
      hipLaunchKernelGGL((m2rnn_groupnorm_wide_kernel<IoT, true>), grid, dim3(256), 0, stream, g);
    else
      hipLaunchKernelGGL((m2rnn_groupnorm_wide_kernel<IoT, false>), grid, dim3(256), 0, stream, g);
    e = hipGetLastError();
  }
  if (e != hipSuccess || !bwd) return e;
  hipLaunchKernelGGL(m2rnn_groupnorm_sum_kernel, dim3((unsigned)ceil_div(2 * g.G * g.S, 64)),
                     dim3(1024), 0, stream, p.parts, g.G * g.S, g.ws, g.dgamma, g.dbeta);
  return hipGetLastError();
}
template <typename IoT>
hipError_t pick(const GroupNormArgs& g, bool bwd, hipStream_t stream) {
  const bool vec = g.S % io::kVec<IoT> == 0 && aligned16(g.y) && aligned16(g.g_pre) &&
                   aligned16(g.gamma) && aligned16(g.beta) && aligned16(g.out) &&
                   aligned16(g.dout) && aligned16(g.dy) && aligned16(g.dg_pre);
  return vec ? pick<IoT, io::kVec<IoT>>(g, bwd, stream) : pick<IoT, 1>(g, bwd, stream);
}

}  // namespace

// The larger of the plans for 16-byte pieces and for single elements (the call's addresses are
// not known here).
size_t groupnorm_workspace_floats(int64_t rows, int64_t G, int64_t S, int io_dtype) {
  const int vec = io_dtype == kBF16 ? io::kVec<uint16_t> : io::kVec<float>;
  const int64_t a = plan(rows, G, S, 1, true).parts;
  const int64_t b = S % vec == 0 ? plan(rows, G, S, vec, true).parts : 0;
  return (size_t)(a > b ? a : b) * 2 * (size_t)(G * S);
}

bool groupnorm_grid_ok(int64_t rows, int64_t G, int64_t S, int io_dtype) {
  const int vec = io_dtype == kBF16 ? io::kVec<uint16_t> : io::kVec<float>;
  for (int v : {1, vec})
    for (bool bwd : {false, true}) {
      const Plan p = plan(rows, G, S, v, bwd);
      const double wgs = p.nch ? ((double)p.blocks / 4.0 + 1.0) * (double)ceil_div(G, p.gw)
                               : (double)p.blocks * (double)G;
      if (wgs >= (double)(1 << 24)) return false;
    }
  return 2.0 * (double)G * (double)S / 64.0 + 1.0 < (double)(1 << 22);
}

hipError_t launch_groupnorm_gate(const GroupNormArgs& g, int io_dtype, bool bwd, hipStream_t stream) {
  return io_dtype == kBF16 ? pick<uint16_t>(g, bwd, stream) : pick<float>(g, bwd, stream);
}

}  // namespace m2rnn
