// Shared device helpers of the gated recurrence, the 8-bit checkpoints and the
// residual norm: element types, loads and stores of a few consecutive steps at
// any alignment, and the 8-bit group format.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dssm {

constexpr int kLaneSteps = 8;               // consecutive steps held by one lane
constexpr int kChunk = 64 * kLaneSteps;     // steps of one wave tile, between two kept states
constexpr int kGroup = 64;                  // steps that share a power of two in 8 bits

// Rows of an 8-bit checkpoint: int8 steps padded to 16 bytes, one exponent byte per group.
__host__ __device__ inline int ckpt8_row(int L) { return (L + 15) / 16 * 16; }
__host__ __device__ inline int ckpt8_groups(int L) { return (L + kGroup - 1) / kGroup; }

// N consecutive elements, aligned as one element: the device reads and writes
// them in one instruction at any address.
template <typename T, int N>
struct VecOf {
  typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

// out[0..N) = p[0..N) as float; elements at or past `n` are not read and are 0.
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, int n, float* out) {
  if (n >= N) {
    const typename VecOf<T, N>::type v = *reinterpret_cast<const typename VecOf<T, N>::type*>(p);
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = (float)v[k];
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = k < n ? (float)p[k] : 0.f;
  }
}

// p[0..min(n, N)) = in, rounded to nearest even once.
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, int n, const float* in) {
  if (n >= N) {
    typename VecOf<T, N>::type v;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = (T)in[k];
    *reinterpret_cast<typename VecOf<T, N>::type*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < n) p[k] = (T)in[k];
  }
}

// N consecutive elements as they lie in memory, in 32-bit words.  Words and not
// elements: where a guarded load meets a whole one, elements would each take a
// register of their own.
template <typename T, int N>
struct Packed {
  static constexpr int W = (N * (int)sizeof(T) + 3) / 4;
  uint32_t w[W];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N * sizeof(T) >= 4) {
      const typename VecOf<T, N>::type v = *reinterpret_cast<const typename VecOf<T, N>::type*>(p);
      __builtin_memcpy(w, &v, sizeof(w));
    } else {
      w[0] = bits(p[0]);
    }
  }
  // elements at or past `n` are not read and are `fill`
  __device__ __forceinline__ void load(const T* p, int n, T fill) {
    if (n >= N) {
      load(p);
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) put(k, bits(k < n ? p[k] : fill));
    }
  }
  __device__ __forceinline__ float operator[](int k) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[k]);
    } else {
      const uint16_t h = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
      return (float)__builtin_bit_cast(T, h);
    }
  }
  // rounded to nearest even once
  __device__ __forceinline__ void set(const float* x) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < N; ++k) w[k] = __float_as_uint(x[k]);
    } else {
      static_assert(N % 2 == 0, "16-bit elements are rounded in pairs");
      typedef T two __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        const two v = {(T)x[2 * k], (T)x[2 * k + 1]};
        w[k] = __builtin_bit_cast(uint32_t, v);
      }
    }
  }
  __device__ __forceinline__ void store(T* p, int n) const {
    static_assert(N * sizeof(T) >= 4, "whole words");
    if (n >= N) {
      typename VecOf<T, N>::type v;
      __builtin_memcpy(&v, w, sizeof(w));
      *reinterpret_cast<typename VecOf<T, N>::type*>(p) = v;
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < n) {
          if constexpr (sizeof(T) == 4)
            p[k] = __builtin_bit_cast(T, w[k]);
          else
            p[k] = __builtin_bit_cast(T, (uint16_t)(w[k / 2] >> (16 * (k & 1))));
        }
    }
  }
  // The compiler forgets what it derived from the words before (their values in
  // float32, twice the registers) and derives it again.
  __device__ __forceinline__ void refresh() {
#pragma unroll
    for (int k = 0; k < W; ++k) asm volatile("" : "+v"(w[k]));
  }

 private:
  static __device__ __forceinline__ uint32_t bits(T x) {
    if constexpr (sizeof(T) == 4)
      return __builtin_bit_cast(uint32_t, x);
    else
      return __builtin_bit_cast(uint16_t, x);
  }
  __device__ __forceinline__ void put(int k, uint32_t b) {
    if constexpr (sizeof(T) == 4)
      w[k] = b;
    else
      w[k / 2] |= b << (16 * (k & 1));
  }
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + exp(-x)) and, to full relative precision, 1 minus it.  Where exp(-x)
// is too large for its reciprocal the first is 0 and the second 1; NaN passes.
// The exponent is one rounded product, so both carry (1 + 1.25 |x|) 2^-24 or so
// beside the hardware's 2^-23: 2e-6 of a value of 1e-13 at x = -30, and nothing
// of a step's size (the rest of log2(e) x would cost three more vector
// operations a gate, in kernels whose vector work takes as long as their memory).
__device__ __forceinline__ float sigmoid_pair(float x, float* rest) {
  const float t = exp2_fast(-kLog2e * x);
  const float s = __builtin_amdgcn_rcpf(1.f + t);
  *rest = t > 0x1p126f ? 1.f : t * s;
  return s;
}

// ---------------------------------------------------------------------------
// 8 bits: x ~ q 2^E, |q| <= 127, E the smallest power with max|x| <= 127 2^E,
// not below -126; stored as the byte E + 127.  Scaling by powers of two is
// exact, so the one rounding is that to a whole number (to even).  A group
// that holds Inf or NaN stores 255 and stands for NaN.  Values next to the
// largest of x's type would round to a power of two past it: there q stops at 63.
// ---------------------------------------------------------------------------
constexpr int kExpNan = 255;

// The group's byte from the largest bit pattern of |x| in it (NaN > Inf > finite).
__device__ __forceinline__ int group_byte(uint32_t top) {
  if (top >= 0x7f800000u) return kExpNan;
  // top = m 2^k, m in [1/2, 1): E = k - 7 if m <= 127/128, else k - 6
  const int k = (int)(top >> 23) - 126;
  const int e = k - 7 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return max(e, -126) + 127;
}

__device__ __forceinline__ float pow2f(int n) {  // 2^n, -127 < n < 128
  return __uint_as_float((uint32_t)(n + 127) << 23);
}

// The scale a stored byte stands for.
__device__ __forceinline__ float group_scale(int byte) {
  return byte == kExpNan ? __uint_as_float(0x7fc00000u) : pow2f(byte - 127);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The byte of the one scale whose 64 would be past the largest value of T
// (2^16 for half, 2^128 else).
template <typename T>
constexpr int last_byte() { return 128 - 6 + 127; }
template <>
constexpr int last_byte<_Float16>() { return 16 - 6 + 127; }

// What a gate's logit may reach in 8 bits, 127 / 4: a sigmoid is 0 or 1 to
// 2^-45 there, and a step that is masked by an infinite or the lowest logit
// costs its neighbours no more of their scale.  A step shut by r alone keeps
// sqrt(2 sigmoid(-31.75)) < 2^-22 of its drive.
constexpr float kGateMax = 31.75f;

// Eight steps of one lane, of type T, in 8 bits; the lanes of a group are
// `width` (<= 8) neighbours.  GATE: values past kGateMax (Inf too) count as it.
// Returns the group's byte.
template <typename T, bool GATE>
__device__ __forceinline__ int quantise8(const float* x, int width, uint2* out) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, abs_bits(x[k]));
  for (int o = 1; o < width; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if (GATE && top <= 0x7f800000u) top = min(top, __float_as_uint(kGateMax));
  const int byte = group_byte(top);
  const float inv = byte == kExpNan ? 0.f : pow2f(127 - byte);
  // x inv is exact; added to 3 2^22 it is rounded to a whole number, to even, whose
  // low byte is the float's
  uint32_t q[8];
  if (GATE) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      q[k] = __float_as_uint(__builtin_amdgcn_fmed3f(x[k] * inv, -127.f, 127.f) + 12582912.f);
  } else if (byte == last_byte<T>()) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      q[k] = __float_as_uint(fminf(fmaxf(x[k] * inv, -63.f), 63.f) + 12582912.f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = __float_as_uint(fmaf(x[k], inv, 12582912.f));
  }
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    // bytes 0 of two words side by side, then of two pairs
    const uint32_t lo = __builtin_amdgcn_perm(q[4 * k + 1], q[4 * k], 0x0c0c0400);
    const uint32_t hi = __builtin_amdgcn_perm(q[4 * k + 3], q[4 * k + 2], 0x0c0c0400);
    w[k] = __builtin_amdgcn_perm(hi, lo, 0x05040100);
  }
  *out = make_uint2(w[0], w[1]);
  return byte;
}

__device__ __forceinline__ void dequantise8(uint2 q, int byte, float* x) {
  const float s = group_scale(byte);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t w = k < 4 ? q.x : q.y;
    x[k] = (float)(int)(int8_t)(w >> (8 * (k & 3))) * s;
  }
}

}  // namespace dssm
