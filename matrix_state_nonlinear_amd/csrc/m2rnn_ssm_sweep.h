// The selective state-space scan as a chunked sweep on the matrix cores.
//
// Per head, H_t = f_t H_{t-1} + d_t k_t v_t^T and y_t = H_t^T q_t.  Over a chunk of
// L tokens that starts from the state S (c_p the sum of log2 f up to token p of
// the chunk, all exponents <= 0):
//     y_p  = sum_{p' <= p} 2^{c_p - c_p'} d_p' (q_p . k_p') v_p' + 2^{c_p} S^T q_p
//     S   <- 2^{c_L} S + sum_p 2^{c_L - c_p} d_p k_p v_p^T
// which is four matrix products a chunk instead of L dependent steps.  The three
// gradients of the sequence tensors are the same sum with the tensors in other
// places (R the state gradient, walked from the last token to the first):
//     dq: a = dy, b = v,  c = k, forward,  state H^T
//     dv: a = k,  b = q,  c = dy, reverse, state R,   d_p on the output
//     dk: a = v,  b = dy, c = q,  reverse, state R^T, d_p on the output
// so one kernel computes all four.
//
// The gradient of the decays is taken from the same passes.  With M_ij = d_j 2^{c_i - c_j}
// (q_i . k_j)(dy_i . v_j), H0 the state at the chunk's start and G the state gradient at its end,
//     dl_t = f_t <H_{t-1}, R_t> = sum_{i >= t > j} M_ij + sum_{i >= t} a_i + sum_{j < t} b_j + 2^{c_L} <H0, G>,
//     a_i = 2^{c_i} q_i^T H0 dy_i,   b_j = d_j 2^{c_L - c_j} k_j^T G v_j,   d_j dd_j = sum_{i >= j} M_ij + b_j:
// the dq pass has the second factor of M and the parts a, and forms the first factor next to it
// (its c and e tiles are k and q); the dk pass has b.  Nothing is subtracted inside a chunk, so a strong
// decay does not cost precision.
//
// A workgroup (4 waves) walks one segment of one head, the state in MFMA
// accumulators throughout: a wave owns 16 NT columns of it, all DA rows.  Where there are fewer
// than 64 columns, RS waves own the same ones and share the chunk's output rows.  All
// products use the 16x16x32 bf16 MFMA (16 times the rate of the fp32 one); bf16
// inputs are exact operands, and every fp32 operand (the decayed scores, the state,
// the decayed inputs of the state update, and fp32 inputs) is split into bf16
// terms whose sum is the fp32 value: three for what is summed into the state (24
// bits, exact), two for the scores and the state's readout when the inputs and
// outputs are bf16 (relative error 2^-15 at most against the output's 2^-8), three of them for
// fp32 inputs and where the readout goes into the decays' fp32 gradient.  Operands are taken so
// that an accumulator layout is the next product's operand layout: the state's accumulators are
// the readout's operand without a move, and an output lane holds four consecutive columns.
//
// What bounds it.  A token and head takes about 2 L (DA + DC) + 4 DA DC operations in chunks of L
// tokens, far below the matrix cores' rate for the bytes it reads: the forward sweep is bound by how
// fast the tiles come in.  Four prompts of 16384 tokens, 16 heads, K = V = 64, bf16: 144 us for 562 MB
// (3.9 TB/s; the same kernel without its products took nine tenths of that; a copy reaches 5.2 TB/s
// on rows that lie together, these are 128 bytes every 2 KB).  The dq and dk sweeps (315 and 264 us
// at B = 16, T = 4096, 16 heads, K = 32, V = 128, 800 MB each) also issue on 52 to 57 % of the
// cycles: two score products, the pair sums and the splits.  Loads run a chunk ahead in registers and cross
// the barriers (lds_barrier); with __syncthreads and branches around them the prompt took 311 us.
#pragma once

#include <type_traits>

#include "m2rnn_device.h"
#include "m2rnn_ssm_internal.h"

namespace m2rnn {
namespace ssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Tokens per chunk: 64 for bf16 inputs, 32 for fp32 ones (three bf16 planes each in LDS).
template <typename InT>
struct Cfg;
template <>
struct Cfg<uint16_t> {
  static constexpr int L = 64, planes = 1, score_terms = 2, state_terms = 2, epc = 8;
};
template <>
struct Cfg<float> {
  static constexpr int L = 32, planes = 3, score_terms = 3, state_terms = 3, epc = 4;
};

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// acc += (sum of a's terms) (sum of b's terms), leaving out the products below the
// last term kept (2^-24 of the result).
template <int PA, int PB>
__device__ __forceinline__ f32x4 mfma_terms(const bf16x8 (&a)[PA], const bf16x8 (&b)[PB], f32x4 c) {
#pragma unroll
  for (int i = PA - 1; i >= 0; --i)
#pragma unroll
    for (int j = PB - 1; j >= 0; --j)
      if (i + j <= 2) c = mfma_bf16(a[i], b[j], c);
  return c;
}

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
// (by value: a bit cast of a vector's element in place reads element 0)
__device__ __forceinline__ float as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ float hi_part(float x) {  // x truncated to bf16
  return __builtin_bit_cast(float, bits(x) & 0xFFFF0000u);
}
// two values truncated to bf16, the first in the low half
__device__ __forceinline__ uint32_t pack_trunc(float x0, float x1) {
  return __builtin_amdgcn_perm(bits(x1), bits(x0), 0x07060302u);
}
// two values rounded to nearest even
__device__ __forceinline__ uint32_t pack_rne(float x0, float x1) {
  const bf16x2 p{(__bf16)x0, (__bf16)x1};
  return __builtin_bit_cast(uint32_t, p);
}
// x0, x1 as P bf16 terms: truncation for all but the last of two, which is rounded;
// three truncated terms hold all 24 bits.
template <int P>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t (&t)[P]) {
  static_assert(P == 2 || P == 3, "");
  t[0] = pack_trunc(x0, x1);
  const float r0 = x0 - hi_part(x0), r1 = x1 - hi_part(x1);
  if constexpr (P == 2) {
    t[1] = pack_rne(r0, r1);
  } else {
    t[1] = pack_trunc(r0, r1);
    t[2] = pack_trunc(r0 - hi_part(r0), r1 - hi_part(r1));
  }
}
template <int P>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&f)[P]) {
  uint32_t w[P][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t[P];
    split2<P>(x[2 * i], x[2 * i + 1], t);
#pragma unroll
    for (int p = 0; p < P; ++p) w[p][i] = t[p];
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
    f[p] = __builtin_bit_cast(bf16x8, u32x4{w[p][0], w[p][1], w[p][2], w[p][3]});
}
__device__ __forceinline__ float lo_half(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float hi_half(uint32_t u) {
  return __builtin_bit_cast(float, u & 0xFFFF0000u);
}
// sums of the terms of eight values (exact: largest first, 24 bits in all)
template <int P>
__device__ __forceinline__ void widen8(const bf16x8 (&f)[P], float (&x)[8]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const u32x4 u = __builtin_bit_cast(u32x4, f[p]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = p ? x[2 * i] + lo_half(u[i]) : lo_half(u[i]);
      x[2 * i + 1] = p ? x[2 * i + 1] + hi_half(u[i]) : hi_half(u[i]);
    }
  }
}

// ------------------------------------------------------------- LDS operands
// Eight values of one row that are consecutive along it.
__device__ __forceinline__ bf16x8 row8(const uint16_t* p) {
  return __builtin_bit_cast(bf16x8, *(const u32x4*)p);
}
// Columns 4 g .. 4 g + 3 and 16 + 4 g .. of a 32-column block (p at the block's column
// 4 g): the order in which two 16-row accumulator tiles hold their rows.
__device__ __forceinline__ bf16x8 row4x2(const uint16_t* p) {
  const u32x2 x = *(const u32x2*)p, y = *(const u32x2*)(p + 16);
  return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
}
// Eight consecutive rows of one column per lane: the transposing read gives lane l of a
// 16-lane group column l of four rows whose 16 columns the group's lanes address
// in pieces of four (lane s: row s / 4, columns 4 (s % 4)).  p: the group's first row at the
// block's first column; stride in elements.
__device__ __forceinline__ bf16x8 col8(const uint16_t* p, int stride, int m) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const uint16_t* s = p + (m >> 2) * stride + (m & 3) * 4;
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)s);
  const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(s + 4 * stride));
  const u32x2 xx = __builtin_bit_cast(u32x2, x), yy = __builtin_bit_cast(u32x2, y);
  return __builtin_bit_cast(bf16x8, u32x4{xx[0], xx[1], yy[0], yy[1]});
}

// A workgroup barrier that orders LDS accesses only: global loads issued ahead and output
// stores stay in flight across it (__syncthreads waits for them).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ int wave_index() {  // uniform
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
}

// The same value, but unknown to the compiler to be it: addresses formed from it are not kept in
// registers across the sweep's other phases.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// ------------------------------------------------------------- staging
// A [tokens, stride] array as a sweep walks it: `base` is at the current chunk's lowest token
// (and the first column wanted), and row p of a chunk of `len` tokens in walking order is token p,
// in reverse (REV) len - 1 - p.
//
// Accesses go through a buffer descriptor whose extent ends with the last row's columns: what lies
// outside reads as zero and is not written, so no access needs a branch (a branch that
// zeroes the register of a load in flight has to wait for it).  Offsets: kOut for columns that
// do not exist; row p of a full chunk otherwise.  A short chunk walked in reverse shifts by the
// missing rows, and rows that do not exist wrap below zero; a chunk has less than
// 2^30 bytes (ssm_vec_rows), so neither can come back into the extent.
template <int L, bool REV, bool VEC>
struct Walk {
  const char* base;                             // uniform
  std::conditional_t<VEC, int, int64_t> stride; // bytes
  int bytes;                                    // of a row, from base

  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int len) const {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (len - 1) * (int)stride + bytes,
                                             0x00020000);
  }
  __device__ __forceinline__ uint32_t shift(int len) const {
    return REV ? (uint32_t)((L - len) * (int)stride) : 0u;
  }
  __device__ __forceinline__ const char* row(int p, int len) const {
    return base + (REV ? len - 1 - p : p) * (int64_t)stride;
  }
  __device__ __forceinline__ void next() { base += (REV ? -L : L) * (int64_t)stride; }
};
constexpr uint32_t kOut = 0x80000000u;

// A tile of L rows (tokens) x W columns: 16-byte pieces, N of them per thread, fetched
// into registers while the chunk before is worked on and written to LDS after it.
template <typename InT, int W, bool REV, bool VEC>
struct Tile {
  using Rows = Walk<Cfg<InT>::L, REV, VEC>;
  static constexpr int L = Cfg<InT>::L, EPC = Cfg<InT>::epc, CPR = W / EPC, RP = 256 / CPR,
                       N = (L * CPR + 255) / 256, STRIDE = W + 8, PLANE = L * STRIDE;
  static_assert((L * CPR % 256 == 0 || L * CPR < 256) && 256 % CPR == 0, "");
  u32x4 r[N];

  // this thread's offset in a full chunk of rows of which D columns exist
  static __device__ __forceinline__ uint32_t offset(const Rows& c, int D) {
    const int row = (int)threadIdx.x / CPR, col = ((int)threadIdx.x % CPR) * EPC;
    return col < D && row < L ? (uint32_t)((REV ? L - 1 - row : row) * (int)c.stride) +
                         (uint32_t)(col * sizeof(InT))
                   : kOut;
  }
  // rows p < len come from the chunk; columns >= D and rows >= len are zero
  __device__ __forceinline__ void fetch(const Rows& c, uint32_t off, int len, int D) {
    if constexpr (VEC) {
      const auto rs = c.rsrc(len);
      const uint32_t v = off - c.shift(len);
      const uint32_t pass = (uint32_t)((REV ? -RP : RP) * c.stride);
#pragma unroll
      for (int i = 0; i < N; ++i)
        r[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(v + i * pass), 0, 0);
    } else {
      const int row0 = (int)threadIdx.x / CPR, col = ((int)threadIdx.x % CPR) * EPC;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = row0 + RP * i;
        u32x4 x{0, 0, 0, 0};
        if (row < len && col < D) {
          const InT* p = (const InT*)c.row(row, len) + col;
#pragma unroll
          for (int j = 0; j < EPC; ++j) {
            if (col + j < D) {
              if constexpr (EPC == 8)
                x[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
              else
                x[j] = bits(p[j]);
            }
          }
        }
        r[i] = x;
      }
    }
  }
  __device__ __forceinline__ void put(uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = (int)threadIdx.x + 256 * i;
      if (L * CPR < 256 && id >= L * CPR) break;
      uint16_t* p = lds + (id / CPR) * STRIDE + (id % CPR) * EPC;
      if constexpr (EPC == 8) {
        *(u32x4*)p = r[i];
      } else {
        uint32_t t0[3], t1[3];
        split2<3>(as_float(r[i][0]), as_float(r[i][1]), t0);
        split2<3>(as_float(r[i][2]), as_float(r[i][3]), t1);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) *(u32x2*)(p + pl * PLANE) = u32x2{t0[pl], t1[pl]};
      }
    }
  }
  // acc[j] += x[j] y[j] over this thread's pieces (its columns are the same in every piece)
  static __device__ __forceinline__ void dot_cols(const Tile& x, const Tile& y, float (&acc)[EPC]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < EPC; ++j) {
        if constexpr (EPC == 8) {
          const uint32_t u = x.r[i][j / 2], w = y.r[i][j / 2];
          acc[j] += (j & 1) ? hi_half(u) * hi_half(w) : lo_half(u) * lo_half(w);
        } else {
          acc[j] += as_float(x.r[i][j]) * as_float(y.r[i][j]);
        }
      }
  }
};

// ------------------------------------------------------------- decays of a chunk
// Per token p of the chunk, from the exact (double) prefix sums c_p of log2 f: every power has
// an exponent <= 0 and is rounded once.
template <int L>
struct Gates {
  float R[L];      // 2^{c_p}: from the carried state to p
  float W[L];      // 2^{c_end - c_p} g_p: from p to the state carried on
  float et[L];     // 2^{c_tile_end - c_p} (tiles of 16 tokens)
  float eg[L];     // the same times g_p
  float rr[L / 16 - 1][L];  // 2^{c_p - c_end(tile j)}, j below p's tile
  float chi[L], clo[L];     // c_p in two parts, for the tiles on the diagonal
  float g[L];      // input weight
  float rho[L];    // output weight
  float total;     // 2^{c_end}
};

__device__ __forceinline__ float pow2(double c) {
  const double n = __builtin_rint(c);
  return __builtin_ldexpf(__builtin_amdgcn_exp2f((float)(c - n)), (int)n);
}
__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}
// log2 f, held at -2048 or more: 2^-2048 is already zero in fp32, and the sums of a chunk
// then keep their low bits.
__device__ __forceinline__ double log2_decay(float alpha, float d) {
  return fmax(-(double)alpha * (double)d * 1.4426950408889634, -2048.0);
}

// x of the lane that CTRL names, 0 where there is none or the row is not in MASK
template <int CTRL, int MASK>
__device__ __forceinline__ double dpp_or_zero(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, MASK, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, MASK, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)(uint32_t)hi << 32) | (uint64_t)(uint32_t)lo);
}
// Inclusive sums over the lanes of a wave, or of each half (L = 32): shifts within the 16-lane
// rows, then each row's last lane added to the row (L = 64: two rows) behind it.  No LDS exchange.
template <int L>
__device__ __forceinline__ double lane_sums(double x) {
  x += dpp_or_zero<0x111, 0xF>(x);  // row_shr:1
  x += dpp_or_zero<0x112, 0xF>(x);
  x += dpp_or_zero<0x114, 0xF>(x);
  x += dpp_or_zero<0x118, 0xF>(x);
  x += dpp_or_zero<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
  if constexpr (L == 64) x += dpp_or_zero<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
  return x;
}

// The prefix sums and step sizes of a chunk as one lane per token sees them, fetched a chunk ahead:
// wave 0 makes R and the diagonal's parts from them, wave 1 W, wave 2 the tiles' input factors, wave
// 3 the tiles' output factors.  Going forward the decay into p counts at p (the inclusive sums of
// the chunk's tokens); in reverse the decay between p and p + 1 is p's own, which is the
// chunk's total less the inclusive sum.
template <int L, bool REV>
struct GateRegs {
  double c, total, end[3];  // end: the sums at the tiles' last tokens (wave 2: of the token's own tile)
  float d;

  // No branch and no scalar load: the loads stay in flight like the tiles' (kept in a wave's
  // own branch, they would be waited for at its end).
  __device__ __forceinline__ void fetch(const double* cum, const float* dt, int len) {
    const int lane = threadIdx.x & 63, w = wave_index();
    const auto rc = __builtin_amdgcn_make_buffer_rsrc((void*)cum, 0, len * 8, 0x00020000);
    const auto rd = __builtin_amdgcn_make_buffer_rsrc((void*)dt, 0, len * 4, 0x00020000);
    auto at = [&](int p) {
      p = p < len ? p : len - 1;
      return REV ? len - 1 - p : p;
    };
    auto sum = [&](int i) {
      return __builtin_bit_cast(double, __builtin_amdgcn_raw_buffer_load_b64(rc, i * 8, 0, 0));
    };
    c = sum(at(lane));
    total = sum(len - 1);
    d = as_float(__builtin_amdgcn_raw_buffer_load_b32(rd, at(lane) * 4, 0, 0));
#pragma unroll
    for (int j = 0; j < L / 16 - 1; ++j) end[j] = sum(at(w == 2 ? lane | 15 : 16 * j + 15));
  }
  __device__ __forceinline__ void put(Gates<L>& G, bool w_in, bool w_out) const {
    const int lane = threadIdx.x & 63, w = wave_index();
    const double x = REV ? total - c : c;
    const float g = w_in ? d : 1.0f;
    if (lane < L) {
      if (w == 0) {
        G.R[lane] = pow2(x);
        const float hi = (float)x;
        G.chi[lane] = hi;
        G.clo[lane] = (float)(x - (double)hi);
        G.g[lane] = g;
      } else if (w == 1) {
        G.W[lane] = pow2(total - x) * g;
        G.rho[lane] = w_out ? d : 1.0f;
        if (lane == 0) G.total = pow2(total);
      } else if (w == 2) {
        const float et = pow2((REV ? total - end[0] : end[0]) - x);
        G.et[lane] = et;
        G.eg[lane] = et * g;
      } else {
#pragma unroll
        for (int j = 0; j < L / 16 - 1; ++j)
          G.rr[j][lane] = lane >= 16 * (j + 1) ? pow2(x - (REV ? total - end[j] : end[j])) : 0.0f;
      }
    }
  }
};

// ------------------------------------------------------------- the sweep
// The four sweeps.  kDk also returns the dot products of e with the state's part of the output (b /
// d), kDq these (a) and the sums over the pairs of a chunk.
enum : int { kY = 0, kDv = 1, kDk = 2, kDq = 3 };

// Sums over the pairs of a chunk, by 16 x 16 tile (it, jt) of M
template <int L>
struct PairSums {
  alignas(16) float rs[L / 16][L];  // [jt][i] sum over the tile's j of M_ij, jt < i's tile
  alignas(16) float cs[L / 16][L];  // [it][j] sum over the tile's i of M_ij / d_j, it >= j's tile
  alignas(16) float xd[L];          // [t] sum over i >= t > j of t's own tile
};
struct NoSums {};

template <typename InT, int AT, int NT, int RS, int MODE, bool VEC>
struct SweepShared {
  using C = Cfg<InT>;
  static constexpr int L = C::L;
  static constexpr bool REV = MODE == kDv || MODE == kDk;
  using TA = Tile<InT, 32 * AT, REV, VEC>;
  using TC = Tile<InT, 64 * NT / RS, REV, VEC>;
  static constexpr int PSTRIDE = L + 8;
  alignas(16) uint16_t a[C::planes * TA::PLANE];
  alignas(16) uint16_t b[C::planes * TA::PLANE];
  alignas(16) uint16_t c[C::planes * TC::PLANE];
  alignas(16) uint16_t e[MODE == kDq ? C::planes * TC::PLANE : 8];
  alignas(16) uint16_t p[C::score_terms][L * PSTRIDE];
  alignas(16) Gates<L> g;
  alignas(16) float red[4][L];
  std::conditional_t<MODE == kDq, PairSums<L>, NoSums> sums;
};

// Shifts within the 16-lane rows, zero beyond their ends: lane l reads lane l + N (l - N).
template <int N>
__device__ __forceinline__ float row_down(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x100 + N, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ float row_up(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x110 + N, 0xF, 0xF, true));
}
// sum over the row's lanes from this one on
__device__ __forceinline__ float row_suffix(float x) {
  x += row_down<1>(x);
  x += row_down<2>(x);
  x += row_down<4>(x);
  x += row_down<8>(x);
  return x;
}
// sum over the row's lanes before this one
__device__ __forceinline__ float row_prefix_excl(float x) {
  x = row_up<1>(x);
  x += row_up<1>(x);
  x += row_up<2>(x);
  x += row_up<4>(x);
  x += row_up<8>(x);
  return x;
}
// the sum of x over the four 16-lane rows, in every lane
__device__ __forceinline__ float rows_sum(float x) {
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

// Four consecutive columns of row p of a chunk: `off` as Tile::offset's for this lane's row and
// columns, `it` 16-row tiles further on.  Without VEC: `left` of the columns exist.
template <int L, bool REV, bool VEC>
__device__ __forceinline__ int place4(const Walk<L, REV, VEC>& c, uint32_t off, int it, int len) {
  const uint32_t tile = (uint32_t)((REV ? -16 : 16) * (int)c.stride) * (uint32_t)it;
  return (int)(off - c.shift(len) + tile);
}
template <typename InT, int L, bool REV, bool VEC>
__device__ __forceinline__ void store_cols4(const Walk<L, REV, VEC>& c, uint32_t off, int it, int p,
                                            int len, f32x4 x, int col, int left, bool f32) {
  if constexpr (VEC) {
    const int v = place4(c, off, it, len);
    if (f32 || sizeof(InT) == 4)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), c.rsrc(len), v, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_rne(x[0], x[1]), pack_rne(x[2], x[3])},
                                            c.rsrc(len), v, 0, 0);
  } else {
    if (p >= len) return;
    char* row = (char*)c.row(p, len);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < left) {
        if (f32 || sizeof(InT) == 4) ((float*)row)[col + r] = x[r];
        else ((uint16_t*)row)[col + r] = (uint16_t)pack_rne(x[r], 0.0f);
      }
  }
}
// The same four columns of an input, as stored (widened when they are used: a value widened at once
// would be waited for at once).
template <typename InT, int L, bool REV, bool VEC>
__device__ __forceinline__ u32x4 load_cols4(const Walk<L, REV, VEC>& c, uint32_t off, int it, int p,
                                            int len, int col, int left) {
  u32x4 x{0, 0, 0, 0};
  if constexpr (VEC) {
    const int v = place4(c, off, it, len);
    if constexpr (sizeof(InT) == 2) {
      const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(c.rsrc(len), v, 0, 0);
      x[0] = u[0];
      x[1] = u[1];
    } else {
      x = __builtin_amdgcn_raw_buffer_load_b128(c.rsrc(len), v, 0, 0);
    }
  } else if (p < len) {
    const InT* row = (const InT*)c.row(p, len);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < left) {
        if constexpr (sizeof(InT) == 2) x[r / 2] |= (uint32_t)row[col + r] << (16 * (r & 1));
        else x[r] = bits(row[col + r]);
      }
  }
  return x;
}
template <typename InT>
__device__ __forceinline__ f32x4 widen4(u32x4 u) {
  if constexpr (sizeof(InT) == 2)
    return f32x4{lo_half(u[0]), hi_half(u[0]), lo_half(u[1]), hi_half(u[1])};
  else
    return __builtin_bit_cast(f32x4, u);
}
// sum of the terms of four consecutive columns in LDS
template <int P>
__device__ __forceinline__ f32x4 lds_cols4(const uint16_t* p, int plane) {
  f32x4 x;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const u32x2 u = *(const u32x2*)(p + i * plane);
    const f32x4 y{lo_half(u[0]), hi_half(u[0]), lo_half(u[1]), hi_half(u[1])};
    x = i ? x + y : y;
  }
  return x;
}

// Workgroups per CU to allow registers for: two, or one where two would spill (a spilled register's
// reload waits for every load in flight before it).  Held to three, the training call at
// B = 16, T = 4096, 16 heads, K = 32, V = 128 takes 1335 us instead of 1188, a prompt of K = V = 64,
// whose registers allow three either way, 234 us in both.
constexpr int sweep_occupancy(int AT, int NT, int mode, int bytes) {  // AT * NT <= 8
  return AT == 8 || (bytes == 4 && mode == kDq && AT * NT >= 4) ? 1 : 2;
}

// KEEP: the state is kept to 24 bits (it may be an output, or goes into the decays' gradient); one that
// only goes into bf16 outputs takes its inputs in two terms, like its readout (234 us for the prompt
// above with its passes; with three terms 247).
template <typename InT, int AT, int NT, int RS, int MODE, bool KEEP, bool VEC>
__global__ void __launch_bounds__(256, sweep_occupancy(AT, NT, MODE, sizeof(InT)))
    m2rnn_ssm_sweep_kernel(const SsmSweepArgs g) {
  using C = Cfg<InT>;
  using S = SweepShared<InT, AT, NT, RS, MODE, VEC>;
  using TA = typename S::TA;
  using TC = typename S::TC;
  constexpr int L = C::L, NI = L / 16, NR = NI >= RS ? NI / RS : 1, P = C::planes, PS = C::score_terms,
                PH = MODE == kY || MODE == kDv ? C::state_terms : 3, CT = KEEP ? 3 : 2;
  __shared__ S sh;

  const int lane = threadIdx.x & 63, m = lane & 15, q4 = lane >> 4;
  // wave: column tiles from 16 NT wc on, and the 16-token rows rg, rg + RS, ... of a chunk's output
  constexpr int CW = 4 / RS;
  const int w = wave_index(), wc = w % CW, rg = w / CW;
  // workgroup id -> (b, segment, head, slab), slabs then heads fastest: the heads that
  // share q and k, and the slabs of a head, run on one XCD and share its L2
  int64_t u = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int slab = (int)(u % g.slabs);
  u /= g.slabs;
  const int n = (int)(u % g.N);
  u /= g.N;
  const int64_t seg = u % g.nseg;
  const int64_t bi = u / g.nseg;
  const int64_t bn = bi * g.N + n;
  const int c0 = slab * (64 * NT / RS);    // first column of this workgroup
  const int dc = g.DC - c0;                // columns left from c0
  constexpr bool REV = S::REV, W_IN = MODE == kY || MODE == kDq, W_OUT = !W_IN;
  constexpr int E = sizeof(InT);

  const int64_t seg0 = seg * g.seglen;
  const int64_t seg1 = seg0 + g.seglen < g.T ? seg0 + g.seglen : g.T;
  const int nch = (int)((seg1 - seg0 + L - 1) / L);

  // the first token of the chunk at hand and of the one being fetched
  int64_t t0 = seg0 + (REV ? (int64_t)(nch - 1) * L : 0), tf = t0;
  auto chunk_len = [&](int64_t t) { return (int)(seg1 - t < L ? seg1 - t : L); };
  // an array of `D` columns of `e` bytes and N / grp heads, from column `col` of the first chunk
  auto walk = [&](const void* p, int grp, int D, int col, int e) {
    const int64_t heads = g.N / grp;
    return Walk<L, REV, VEC>{(const char*)p + (((bi * g.T + t0) * heads + n / grp) * D + col) * e,
                             (decltype(Walk<L, REV, VEC>::stride))(heads * D * e), (D - col) * e};
  };
  const int oE = W_IN && MODE == kY ? E : g.out_f32 ? 4 : E;
  auto ra = walk(g.a, g.a_grp, g.DA, 0, E), rb = walk(g.b, g.b_grp, g.DA, 0, E),
       rc = walk(g.c, g.c_grp, g.DC, c0, E), ro = walk(g.out, 1, g.DC, c0, oE);
  auto re = rc;
  if constexpr (MODE == kDk || MODE == kDq) re = walk(g.e, g.e_grp, g.DC, c0, E);
  const uint32_t oa = TA::offset(ra, g.DA), ob = TA::offset(rb, g.DA), oc = TC::offset(rc, dc),
                 oe = MODE == kDq ? TC::offset(re, dc) : 0;
  // this lane's place in the output and in e: row m of a 16-row tile, four columns of each of its
  // wave's column tiles
  uint32_t oo[NT], ox[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = 16 * (wc * NT + nt) + 4 * q4, row = REV ? L - 1 - m : m;
    oo[nt] = col < dc ? (uint32_t)(row * (int)ro.stride) + (uint32_t)(col * oE) : kOut;
    ox[nt] = col < dc ? (uint32_t)(row * (int)re.stride) + (uint32_t)(col * E) : kOut;
  }
  // the 16-token rows of this wave (fp32's chunks have two: the waves beyond repeat the first ones
  // and write nothing)
  auto row_tile = [&](int k) { return NI < RS ? rg % NI : k * RS + rg; };
  const double* cum = g.cum + bn * g.T + t0;
  const float* dts = g.d + bn * g.T + t0;
  const int64_t tok0 = ((int64_t)slab * g.B * g.N + bn) * g.T;  // of the per-token results

  // scores above the diagonal stay zero: only tiles on and below it are ever written
  for (int i = threadIdx.x; i < (int)(sizeof(sh.p) / 16); i += 256) ((u32x4*)sh.p)[i] = u32x4{0, 0, 0, 0};

  // state: rows 16 at + 4 q4 + r, column 16 ct + m of this workgroup's columns
  f32x4 st[2 * AT][NT];
  {
    const int64_t kv = (int64_t)g.DA * g.DC;
    const float* s0 = g.state0 ? g.state0 + (bn * g.nseg + seg) * kv : nullptr;
    const float* he = nullptr;
    if (g.base)
      he = seg + 1 < g.nseg ? g.hend + (bn * g.nseg + seg + 1) * kv : g.hend_last + bn * kv;
    double dot = 0.0;
#pragma unroll
    for (int at = 0; at < 2 * AT; ++at)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ai = 16 * at + 4 * q4 + r, ci = c0 + 16 * (wc * NT + nt) + m;
          const bool ok = ai < g.DA && ci < g.DC;
          const int64_t o = (int64_t)ai * g.a_stride + (int64_t)ci * g.c_stride;
          const float x = (s0 && ok) ? s0[o] : 0.0f;
          st[at][nt][r] = x;
          if (he && ok && rg == 0) dot += (double)x * (double)he[o];
        }
    if (g.base) {
#pragma unroll
      for (int s = 1; s < 64; s *= 2) dot += __shfl_xor(dot, s);
      double* red = (double*)&sh.red[0][0];
      if (lane == 0) red[w] = dot;
      lds_barrier();
      if (threadIdx.x == 0)
        g.base[((int64_t)slab * g.B * g.N + bn) * g.nseg + seg] =
            (red[0] + red[1]) + (red[2] + red[3]);
      lds_barrier();
    }
  }

  f32x4 skip[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int col = 16 * (wc * NT + nt) + 4 * q4 + r;
      skip[nt][r] = g.skip && col < dc ? g.skip[(int64_t)n * g.DC + c0 + col] : 0.0f;
    }

  TA fa, fb;
  TC fc, fe;
  GateRegs<L, REV> fg;
  u32x4 ev[MODE == kDk ? NR : 1][NT];
  float csum[C::epc];
#pragma unroll
  for (int j = 0; j < C::epc; ++j) csum[j] = 0.0f;
  const bool do_col = MODE == kDq && slab == 0;
  auto fetch = [&]() {  // the chunk at tf, and on to the next
    const int len = chunk_len(tf);
    fa.fetch(ra, oa, len, g.DA);
    fb.fetch(rb, ob, len, g.DA);
    fc.fetch(rc, oc, len, dc);
    if constexpr (MODE == kDq) fe.fetch(re, oe, len, dc);
    if constexpr (MODE == kDk) {
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int cc = 16 * (wc * NT + nt) + 4 * q4, it = row_tile(k);
          ev[k][nt] = load_cols4<InT>(re, ox[nt], it, 16 * it + m, len, cc, dc - cc);
        }
    }
    fg.fetch(cum, dts, len);
    ra.next();
    rb.next();
    rc.next();
    if constexpr (MODE == kDk || MODE == kDq) re.next();
    cum += REV ? -L : L;
    dts += REV ? -L : L;
    tf += REV ? -L : L;
  };
  auto put = [&]() {
    fa.put(sh.a);
    fb.put(sh.b);
    fc.put(sh.c);
    if constexpr (MODE == kDq) {
      fe.put(sh.e);
      if (do_col) TA::dot_cols(fa, fb, csum);
    }
    fg.put(sh.g, W_IN, W_OUT);
  };
  fetch();
  put();
  lds_barrier();

  for (int ch = 0; ch < nch; ++ch) {
    const int len = chunk_len(t0);
    const Gates<L>& G = sh.g;

    // scores: tile (it, jt), jt <= it, of a b^T, decayed and split.  Wave w takes the diagonal tile
    // (w, w) and then tiles below the diagonal, so that a tile's kind is known at compile time and
    // two tiles' products can overlap.
    {
      const int ls = fresh(lane), m = ls & 15, q4 = ls >> 4;
      constexpr int BELOW = NI * (NI - 1) / 2;
#pragma unroll
      for (int rd = 0; rd < 1 + (BELOW + 3) / 4; ++rd) {
        const bool diag = rd == 0;
        const int idx = diag ? w : NI == 4 ? (rd - 1) * 4 + w : w - 2;
        if (idx >= 0 && idx < (diag ? NI : BELOW)) {
          const int it = diag ? idx : idx >= 3 ? 3 : idx >= 1 ? 2 : 1;
          const int jt = diag ? idx : idx - it * (it - 1) / 2;
          f32x4 s{0, 0, 0, 0};
          const uint16_t* ra = sh.a + (16 * it + m) * TA::STRIDE + 8 * q4;
          const uint16_t* rb = sh.b + (16 * jt + m) * TA::STRIDE + 8 * q4;
#pragma unroll
          for (int t = 0; t < AT; ++t) {
            bf16x8 xa[P], xb[P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
              xa[p] = row8(ra + p * TA::PLANE + 32 * t);
              xb[p] = row8(rb + p * TA::PLANE + 32 * t);
            }
            s = mfma_terms(xb, xa, s);
          }
          // lane: token i = 16 it + m, inputs j = 16 jt + 4 q4 + r
          const int i = 16 * it + m, j0 = 16 * jt + 4 * q4;
          f32x4 g4{1, 1, 1, 1};  // input weights not yet in s
          if (diag) {
            const f32x4 ch4 = *(const f32x4*)(G.chi + j0), cl4 = *(const f32x4*)(G.clo + j0);
            g4 = *(const f32x4*)(G.g + j0);
            const float hi = G.chi[i], lo = G.clo[i];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float dec = __builtin_amdgcn_exp2f((hi - ch4[r]) + (lo - cl4[r]));
              s[r] = j0 + r <= i ? s[r] * dec : 0.0f;
            }
          } else {
            const f32x4 e4 = *(const f32x4*)((MODE == kDq ? G.et : G.eg) + j0);
            if constexpr (MODE == kDq) g4 = *(const f32x4*)(G.g + j0);
            const float ri = G.rr[jt][i];
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] *= ri * e4[r];
          }
          if constexpr (MODE == kDq) {
            // the other factor of M: c . e (k . q)
            f32x4 qk{0, 0, 0, 0};
            const uint16_t* re = sh.e + (16 * it + m) * TC::STRIDE + 8 * q4;
            const uint16_t* rc = sh.c + (16 * jt + m) * TC::STRIDE + 8 * q4;
#pragma unroll
            for (int t = 0; t < 2 * NT / RS; ++t) {
              bf16x8 xe[P], xc[P];
#pragma unroll
              for (int p = 0; p < P; ++p) {
                xe[p] = row8(re + p * TC::PLANE + 32 * t);
                xc[p] = row8(rc + p * TC::PLANE + 32 * t);
              }
              qk = mfma_terms(xc, xe, qk);
            }
            f32x4 mm = s * qk, col;
#pragma unroll
            for (int r = 0; r < 4; ++r) col[r] = row16_sum(mm[r]);
            if (m == 0) *(f32x4*)(sh.sums.cs[it] + j0) = col;
            mm *= g4;
            float sum = 0.0f;
            if (diag) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float suf = row_suffix(mm[r]);
                sum += j0 + r < i ? suf : 0.0f;
              }
              sum = rows_sum(sum);
              if (q4 == 0) sh.sums.xd[i] = sum;
            } else {
              sum = rows_sum((mm[0] + mm[1]) + (mm[2] + mm[3]));
              if (q4 == 0) sh.sums.rs[jt][i] = sum;
            }
          }
          if (MODE == kDq || diag) s *= g4;
          uint32_t x0[PS], x1[PS];
          split2<PS>(s[0], s[1], x0);
          split2<PS>(s[2], s[3], x1);
#pragma unroll
          for (int p = 0; p < PS; ++p)
            *(u32x2*)(sh.p[p] + i * S::PSTRIDE + j0) = u32x2{x0[p], x1[p]};
        }
      }
    }

    // readout of the carried state: lane holds out[i = 16 it + m][c = 4 q4 + r]
    f32x4 acc[NR][NT];
    {
      const int ls = fresh(lane), m = ls & 15, q4 = ls >> 4;
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[k][nt] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < AT; ++t) {
        bf16x8 hs[NT][PH];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const f32x4 lo = st[2 * t][nt], hi = st[2 * t + 1][nt];
          const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          split8<PH>(x, hs[nt]);
        }
#pragma unroll
        for (int k = 0; k < NR; ++k) {
          const int row = 16 * row_tile(k) + m;
          bf16x8 xa[P];
#pragma unroll
          for (int p = 0; p < P; ++p)
            xa[p] = row4x2(sh.a + p * TA::PLANE + row * TA::STRIDE + 32 * t + 4 * q4);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[k][nt] = mfma_terms(hs[nt], xa, acc[k][nt]);
        }
      }
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const float R = G.R[16 * row_tile(k) + m];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[k][nt] *= R;
      }
      if constexpr ((MODE == kDk || MODE == kDq)) {
        // e . (the state's part of the output), this wave's columns
#pragma unroll
        for (int k = 0; k < NR; ++k) {
          const int i = 16 * row_tile(k) + m;
          float dot = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int cc = 16 * (wc * NT + nt) + 4 * q4;
            f32x4 y;
            if constexpr (MODE == kDq) y = lds_cols4<P>(sh.e + i * TC::STRIDE + cc, TC::PLANE);
            else y = widen4<InT>(ev[k][nt]);
            const f32x4 x = acc[k][nt];
            dot += (y[0] * x[0] + y[1] * x[1]) + (y[2] * x[2] + y[3] * x[3]);
          }
          dot = rows_sum(dot);
          if (q4 == 0) sh.red[wc][i] = dot;
        }
      }
    }
    lds_barrier();  // the scores are in LDS
    // the next chunk's tiles, here rather than before the scores: their registers are free in the
    // first half, and the second is longer than the loads take
    if (ch + 1 < nch) fetch();

    if constexpr ((MODE == kDk || MODE == kDq)) {
      if (w == 2 && lane < len) {
        const int64_t o = tok0 + t0 + (REV ? len - 1 - lane : lane);
        float sum = sh.red[0][lane];
#pragma unroll
        for (int i = 1; i < CW; ++i) sum += sh.red[i][lane];
        g.rowdot[o] = sum;
      }
    }
    if constexpr (MODE == kDq) {
      if (w == 3) {
        // per token t: all pairs i >= t > j of the chunk, from the tiles' sums; and sum_i M_it / d_t
        const int t = lane & (L - 1), tt = t >> 4;
        float row[NI - 1], rowtot = 0.0f, coltot = 0.0f;
#pragma unroll
        for (int j = 0; j < NI - 1; ++j) {
          row[j] = tt > j ? sh.sums.rs[j][t] : 0.0f;
          rowtot += row[j];
        }
#pragma unroll
        for (int it = NI - 1; it > 0; --it) coltot += it > tt ? sh.sums.cs[it][t] : 0.0f;
        float x = sh.sums.xd[t] + row_suffix(rowtot) + row_prefix_excl(coltot * G.g[t]);
        if constexpr (NI == 4) {  // tiles on both sides of t's
          const float t0s = row16_sum(row[0]), t1s = row16_sum(row[1]);
          const float s20 = lane_value_r(t0s, 32), s30 = lane_value_r(t0s, 48),
                      s31 = lane_value_r(t1s, 48);
          x += tt == 1 ? s20 + s30 : tt == 2 ? s30 + s31 : 0.0f;
        }
        if (lane < len) {
          const int64_t o = tok0 + t0 + (REV ? len - 1 - lane : lane);
          g.pairs[o] = x;
          g.colpairs[o] = coltot + sh.sums.cs[tt][t];
        }
      }
    }

    // the chunk's own inputs, and what they leave in the state
    {
      const int ls = fresh(lane), m = ls & 15, q4 = ls >> 4;
      const float ftot = G.total;
#pragma unroll
      for (int at = 0; at < 2 * AT; ++at)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st[at][nt] *= ftot;
#pragma unroll
      for (int jb = 0; jb < L / 32; ++jb) {
        bf16x8 cw[NT][CT];
        const f32x4 w0 = *(const f32x4*)(G.W + 32 * jb + 8 * q4),
                    w1 = *(const f32x4*)(G.W + 32 * jb + 8 * q4 + 4);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          bf16x8 xc[P];
#pragma unroll
          for (int p = 0; p < P; ++p)
            xc[p] = col8(sh.c + p * TC::PLANE + (32 * jb + 8 * q4) * TC::STRIDE + 16 * (wc * NT + nt),
                         TC::STRIDE, m);
#pragma unroll
          for (int k = 0; k < NR; ++k) {
            const int it = row_tile(k);
            if (it >= 2 * jb) {
              bf16x8 xp[PS];
#pragma unroll
              for (int p = 0; p < PS; ++p)
                xp[p] = row8(sh.p[p] + (16 * it + m) * S::PSTRIDE + 32 * jb + 8 * q4);
              acc[k][nt] = mfma_terms(xc, xp, acc[k][nt]);
            }
          }
          float x[8];
          widen8<P>(xc, x);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= j < 4 ? w0[j & 3] : w1[j & 3];
          split8<CT>(x, cw[nt]);
        }
#pragma unroll
        for (int at = 0; at < 2 * AT; ++at) {
          bf16x8 xb[P];
#pragma unroll
          for (int p = 0; p < P; ++p)
            xb[p] = col8(sh.b + p * TA::PLANE + (32 * jb + 8 * q4) * TA::STRIDE + 16 * at,
                         TA::STRIDE, m);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) st[at][nt] = mfma_terms(xb, cw[nt], st[at][nt]);
        }
      }
    }

    // output
    {
      const int ls = fresh(lane), m = ls & 15, q4 = ls >> 4;
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int it = row_tile(k), i = 16 * it + m;
        if (NI < RS && rg >= NI) break;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int cc = 16 * (wc * NT + nt) + 4 * q4;
          f32x4 x = acc[k][nt];
          if constexpr (W_OUT) x *= G.rho[i];
          if constexpr (MODE == kY || MODE == kDv)
            x += skip[nt] * lds_cols4<P>(sh.c + i * TC::STRIDE + cc, TC::PLANE);
          store_cols4<InT>(ro, oo[nt], it, i, len, x, cc, dc - cc, oE > E);
        }
      }
    }
    ro.next();
    t0 += REV ? -L : L;
    lds_barrier();  // everybody is done with the tiles
    if (ch + 1 < nch) {
      put();
      lds_barrier();
    }
  }

  if (g.stateT && rg == 0) {
    float* sT = g.stateT + bn * (int64_t)g.DA * g.DC;
#pragma unroll
    for (int at = 0; at < 2 * AT; ++at)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ai = 16 * at + 4 * q4 + r, ci = c0 + 16 * (wc * NT + nt) + m;
          if (ai < g.DA && ci < g.DC)
            sT[(int64_t)ai * g.a_stride + (int64_t)ci * g.c_stride] = st[at][nt][r];
        }
  }
  if (do_col) {  // threads with the same columns: 256 / CPR of them, summed in order
    lds_barrier();
    static_assert(sizeof(sh.a) + sizeof(sh.b) >= 256 * C::epc * sizeof(float), "");
    float* red = (float*)&sh;  // over a and b, which nobody reads any more
#pragma unroll
    for (int j = 0; j < C::epc; ++j) red[threadIdx.x * C::epc + j] = csum[j];
    lds_barrier();
    for (int col = threadIdx.x; col < g.DA; col += 256) {
      float sum = 0.0f;
      for (int k = col / C::epc; k < 256; k += TA::CPR) sum += red[k * C::epc + col % C::epc];
      g.colsum[(bn * g.nseg + seg) * g.DA + col] = sum;
    }
  }
}

// The state a segment adds to a zero start: the sweep's state update alone.  Both directions
// walk from the segment's last chunk to its first: with forward decays a chunk's inputs are
// weighted by all that follows (`run`), and the sweep that comes next, walking forward, finds
// the tokens read last in the memory-side cache.  66 us for 294 MB (4.5 TB/s) at the prompt above:
// bound by the loads, two products a chunk against the sweep's five.  One workgroup per CU for wide
// states and fp32 ones, whose registers would spill with two.
template <typename InT, int AT, int NT, int RS, bool REV, bool VEC>
__global__ void __launch_bounds__(256, (AT * NT <= 4 && sizeof(InT) == 2) ? 2 : 1)
    m2rnn_ssm_contrib_kernel(const SsmContribArgs g) {
  using C = Cfg<InT>;
  using TB = Tile<InT, 32 * AT, REV, VEC>;
  using TC = Tile<InT, 64 * NT / RS, REV, VEC>;
  constexpr int L = C::L, P = C::planes, E = sizeof(InT);
  struct Sh {
    alignas(16) uint16_t b[P * TB::PLANE];
    alignas(16) uint16_t c[P * TC::PLANE];
    alignas(16) Gates<L> g;
  };
  __shared__ Sh sh;
  const int lane = threadIdx.x & 63, m = lane & 15, q4 = lane >> 4;
  // wave: column tiles from 16 NT wc on, state rows from 16 HA rg on
  constexpr int CW = 4 / RS, HA = 2 * AT / RS;
  const int w = wave_index(), wc = w % CW, rg = w / CW;
  int64_t u = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int slab = (int)(u % g.slabs);
  u /= g.slabs;
  const int n = (int)(u % g.N);
  u /= g.N;
  const int64_t seg = u % g.nseg;
  const int64_t bi = u / g.nseg;
  const int64_t bn = bi * g.N + n;
  const int c0 = slab * (64 * NT / RS);
  const int64_t seg0 = seg * g.seglen;
  const int64_t seg1 = seg0 + g.seglen < g.T ? seg0 + g.seglen : g.T;
  const int nch = (int)((seg1 - seg0 + L - 1) / L);
  const int dc = g.DC - c0;
  int64_t tf = seg0 + (int64_t)(nch - 1) * L;
  auto walk = [&](const void* p, int grp, int D, int col) {
    const int64_t heads = g.N / grp;
    return Walk<L, REV, VEC>{(const char*)p + (((bi * g.T + tf) * heads + n / grp) * D + col) * E,
                             (decltype(Walk<L, REV, VEC>::stride))(heads * D * E), (D - col) * E};
  };
  auto rb = walk(g.b, g.b_grp, g.DA, 0), rc = walk(g.c, g.c_grp, g.DC, c0);
  const uint32_t ob = TB::offset(rb, g.DA), oc = TC::offset(rc, dc);
  const double* cum = g.cum + bn * g.T + tf;
  const float* dts = g.d + bn * g.T + tf;

  f32x4 st[HA][NT];
#pragma unroll
  for (int at = 0; at < HA; ++at)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) st[at][nt] = f32x4{0, 0, 0, 0};
  float ftot = 1.0f;
  TB fb;
  TC fc;
  GateRegs<L, REV> fg;
  auto fetch = [&]() {
    const int len = (int)(seg1 - tf < L ? seg1 - tf : L);
    fb.fetch(rb, ob, len, g.DA);
    fc.fetch(rc, oc, len, dc);
    fg.fetch(cum, dts, len);
    rb.base -= L * (int64_t)rb.stride;
    rc.base -= L * (int64_t)rc.stride;
    cum -= L;
    dts -= L;
    tf -= L;
  };
  auto put = [&]() {
    fb.put(sh.b);
    fc.put(sh.c);
    fg.put(sh.g, g.w_in, false);
  };
  fetch();
  put();
  lds_barrier();
  for (int ch = 0; ch < nch; ++ch) {
    const Gates<L>& G = sh.g;
    if (ch + 1 < nch) fetch();
    const float f = G.total, run = REV ? 1.0f : ftot;
    ftot *= f;
    if constexpr (REV)
#pragma unroll
      for (int at = 0; at < HA; ++at)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st[at][nt] *= f;
#pragma unroll
    for (int jb = 0; jb < L / 32; ++jb) {
      bf16x8 cw[NT][3];
      f32x4 w0 = *(const f32x4*)(G.W + 32 * jb + 8 * q4),
            w1 = *(const f32x4*)(G.W + 32 * jb + 8 * q4 + 4);
      if constexpr (!REV) {
        w0 *= run;
        w1 *= run;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        bf16x8 xc[P];
#pragma unroll
        for (int p = 0; p < P; ++p)
          xc[p] = col8(sh.c + p * TC::PLANE + (32 * jb + 8 * q4) * TC::STRIDE + 16 * (wc * NT + nt),
                       TC::STRIDE, m);
        float x[8];
        widen8<P>(xc, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= j < 4 ? w0[j & 3] : w1[j & 3];
        split8<3>(x, cw[nt]);
      }
#pragma unroll
      for (int at = 0; at < HA; ++at) {
        bf16x8 xb[P];
#pragma unroll
        for (int p = 0; p < P; ++p)
          xb[p] = col8(sh.b + p * TB::PLANE + (32 * jb + 8 * q4) * TB::STRIDE +
                           16 * (HA * rg + at), TB::STRIDE, m);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st[at][nt] = mfma_terms(xb, cw[nt], st[at][nt]);
      }
    }
    lds_barrier();
    if (ch + 1 < nch) {
      put();
      lds_barrier();
    }
  }
  float* o = g.contrib + (bn * g.nseg + seg) * (int64_t)g.DA * g.DC;
#pragma unroll
  for (int at = 0; at < HA; ++at)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int ai = 16 * (HA * rg + at) + 4 * q4 + r, ci = c0 + 16 * (wc * NT + nt) + m;
        if (ai < g.DA && ci < g.DC) o[(int64_t)ai * g.DC + ci] = st[at][nt][r];
      }
  if (g.fseg && slab == 0 && threadIdx.x == 0) g.fseg[bn * g.nseg + seg] = ftot;
}

}  // namespace ssm
}  // namespace m2rnn
