// Device helpers of the kernels that take strips of steps with all their
// channels: sums across lanes and waves, and which strip a workgroup takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dssm {

// A value from another lane of its row of 16, by the data-parallel primitives.
template <int CTRL>
__device__ __forceinline__ float row_move(float x) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// v added up over pairs of rows of 16 lanes, and over the wave's halves.
__device__ __forceinline__ float rows_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float halves_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// v summed over the LT lanes of one channel; all of them get the sum.
template <int LT>
__device__ __forceinline__ float lanes_sum(float v) {
  if (LT >= 2) v += row_move<0xb1>(v);    // neighbours swapped
  if (LT >= 4) v += row_move<0x4e>(v);    // pairs swapped
  if (LT >= 8) v += row_move<0x141>(v);   // mirrored in 8 lanes, whose fours agree by now
  if (LT >= 16) v += row_move<0x140>(v);  // mirrored in 16
  if (LT >= 32) v = rows_sum(v);
  if (LT >= 64) v = halves_sum(v);
  return v;
}

// v summed over the lanes of a wave that hold the same steps (every LT-th).
template <int LT>
__device__ __forceinline__ float column_sum(float v) {
  if (LT <= 1) v += row_move<0xb1>(v);
  if (LT <= 2) v += row_move<0x4e>(v);   // the pairs' lanes keep their place
  if (LT <= 4) v += row_move<0x124>(v);  // rotated by 4: with the next, every fourth of 16
  if (LT <= 8) v += row_move<0x128>(v);  // rotated by 8
  if (LT <= 16) v = rows_sum(v);
  if (LT <= 32) v = halves_sum(v);
  return v;
}

// N sets of VE values summed over the workgroup's lanes of the same strip
// column; every thread gets the totals.  buf: [NT / 64][N LT VE] floats.  More
// than four waves are added up by one thread per column, so that not every
// thread reads every wave's sums.
template <int NT, int LT, int VE, int N>
__device__ __forceinline__ void strip_sum(float (*v)[VE], float* buf) {
  constexpr int W = NT / 64, C = N * LT * VE;
#pragma unroll
  for (int m = 0; m < N; ++m)
#pragma unroll
    for (int k = 0; k < VE; ++k) v[m][k] = column_sum<LT>(v[m][k]);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lt = lane % LT;
  __syncthreads();  // the buffer's last readers are done
  if (lane < LT)
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int k = 0; k < VE; ++k) buf[wave * C + (m * LT + lt) * VE + k] = v[m][k];
  __syncthreads();
  if (W > 4) {
    // each column is one thread's: no other reads or writes it before the barrier
    for (int c = threadIdx.x; c < C; c += NT) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += buf[w * C + c];
      buf[c] = s;
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < N; ++m)
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      float s = buf[(m * LT + lt) * VE + k];
      if (W <= 4)
#pragma unroll
        for (int w = 1; w < W; ++w) s += buf[w * C + (m * LT + lt) * VE + k];
      v[m][k] = s;
    }
}

// Steps at or past nv are 0, whatever the parameters: of an infinite one the
// zeros read there would make NaN.  Whole strips (the workgroup's) skip it.
template <int VE>
__device__ __forceinline__ void live_only(float* v, int nv, bool whole) {
  if (whole) return;
#pragma unroll
  for (int k = 0; k < VE; ++k) v[k] = k < nv ? v[k] : 0.f;
}

// Strips to workgroups: each of the 8 dies takes a run of neighbouring strips,
// which share the ends of their 128-byte lines in its cache (workgroups go to
// the dies in turn).  `per` strips to a die; the last dies' numbers run past n.
__device__ __forceinline__ int strip_of_block(int block, int per) {
  return (block & 7) * per + (block >> 3);
}

}  // namespace dssm
