// Vectors of 1, 4 or 8 consecutive storage elements (float, or bf16 as uint16_t) as fp32
// values: one access of up to 16 bytes, bf16 rounded to nearest even on the way out.
#pragma once

#include <type_traits>

#include "m2rnn_device.h"

namespace m2rnn {
namespace io {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const bf16x2 p{(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

template <int N>
struct Vals {
  float x[N];
};

template <int N>
__device__ __forceinline__ Vals<N> load(const float* p) {
  Vals<N> v;
  if constexpr (N == 1) {
    v.x[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 u = *(const f32x4*)(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.x[i + j] = u[j];
    }
  }
  return v;
}
template <int N>
__device__ __forceinline__ Vals<N> load(const uint16_t* p) {
  Vals<N> v;
  if constexpr (N == 1) {
    v.x[0] = as_float((uint32_t)*p << 16);
  } else {
    uint32_t u[N / 2];
    if constexpr (N == 8) {
      const u32x4 w = *(const u32x4*)p;
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = w[j];
    } else {
      const u32x2 w = *(const u32x2*)p;
      u[0] = w[0];
      u[1] = w[1];
    }
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      v.x[2 * j] = as_float(u[j] << 16);
      v.x[2 * j + 1] = as_float(u[j] & 0xFFFF0000u);
    }
  }
  return v;
}
// The same elements as they are stored, to be widened when they are used: registers of a load that
// stays in flight.
template <typename T, int N>
struct Raw {
  std::conditional_t<N == 1, T, std::conditional_t<N * sizeof(T) == 16, u32x4, u32x2>> r;
  static_assert(N == 1 || N * sizeof(T) == 16 || N * sizeof(T) == 8, "");
  __device__ __forceinline__ void load(const T* p) { r = *(const decltype(r)*)p; }
  __device__ __forceinline__ Vals<N> vals() const {
    Vals<N> v;
    if constexpr (N == 1) {
      if constexpr (sizeof(T) == 2) v.x[0] = as_float((uint32_t)r << 16);
      else v.x[0] = r;
    } else {
      const auto u = r;
#pragma unroll
      for (int j = 0; j < (int)(N * sizeof(T) / 4); ++j) {
        const uint32_t w = u[j];
        if constexpr (sizeof(T) == 2) {
          v.x[2 * j] = as_float(w << 16);
          v.x[2 * j + 1] = as_float(w & 0xFFFF0000u);
        } else {
          v.x[j] = as_float(w);
        }
      }
    }
    return v;
  }
};
template <int N>
__device__ __forceinline__ void store(float* p, const Vals<N>& v) {
  if constexpr (N == 1) {
    *p = v.x[0];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *(f32x4*)(p + i) = f32x4{v.x[i], v.x[i + 1], v.x[i + 2], v.x[i + 3]};
  }
}
template <int N>
__device__ __forceinline__ void store(uint16_t* p, const Vals<N>& v) {
  if constexpr (N == 1) {
    *p = (uint16_t)pack(v.x[0], 0.0f);
  } else if constexpr (N == 4) {
    *(u32x2*)p = u32x2{pack(v.x[0], v.x[1]), pack(v.x[2], v.x[3])};
  } else {
    *(u32x4*)p = u32x4{pack(v.x[0], v.x[1]), pack(v.x[2], v.x[3]), pack(v.x[4], v.x[5]),
                       pack(v.x[6], v.x[7])};
  }
}

// Elements per thread of a 16-byte access.
template <typename IoT>
constexpr int kVec = 16 / (int)sizeof(IoT);

// 1 / (1 + e^-x): the exponential runs to infinity or zero at the ends and its reciprocal to 0 or 1.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

}  // namespace io
}  // namespace m2rnn
