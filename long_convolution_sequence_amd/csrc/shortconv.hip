// The short causal convolution of every channel, its last inputs carried as a
// state, with its gradients:
//
//   pre_t = bias + sum_{k<K} w_k e_{t+k},  y_t = pre_t or silu(pre_t),
//
// e the K - 1 inputs before the row followed by the row itself, so that tap
// K - 1 meets the present step.  With p_t = dy_t act'(pre_t):
//
//   de_i = sum_k w_k p_{i-k},  dw_k = sum p_t e_{t+k},  dbias = sum p_t,
//
// de's first K - 1 being the gradient of the state before the row.
//
// Memory bounds it: an input read and an output written forward, two and one
// backward (rows of 8191 steps, 4 x 1024 of them, 7 taps, float32: 56 us forward, 4.8
// TB/s, 96 backward, 4.2; rows of 4096, 4 x 2048 of them, 4 taps, bf16: 32 and 51, 4.2
// and 3.9).  A lane holds 8 consecutive steps and asks for the 8 before them
// too, which its neighbour has just brought into the cache.
#include <algorithm>
#include <type_traits>

#include "dssm_internal.h"
#include "seq_common.h"

namespace dssm {
namespace {

struct Args {
  const void* u;
  long long su;  // elements between batch rows
  const float *w, *bias;  // bias may be null
  const int* lens;
  int B, H, L, silu;
  long rows;
  const float* x0;  // [rows][K - 1] or null: zero
  float* xT;        // may be null; may be x0
  void* y;
  // backward
  const void* dy;
  const float* dx;  // [rows][K - 1] or null
  void* du;
  long long sdu;
  float* dx0;       // may be null
  float* part;      // [rows][nseg][K + 1]
  int lpr;          // lanes of a row
  int ntile, nseg, seg_tiles;
};

__device__ __forceinline__ int row_len(const Args& p, int b) {
  if (!p.lens) return p.L;
  return min(max(p.lens[b], 0), p.L);
}

// The row's weights and bias.
template <int K>
__device__ __forceinline__ float load_taps(const Args& p, int h, float* w) {
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = p.w[(size_t)h * K + k];
  return p.bias ? p.bias[h] : 0.f;
}

// e[0 .. K + 6]: the K - 1 values before step t (a multiple of 8) and the 8
// steps from it on; steps at or past len are 0.
template <typename T, int K>
__device__ __forceinline__ void load_window(const Args& p, const T* u, long row, int t, int len,
                                            float* e) {
  float v[8];
  if constexpr (K > 1) {
    if (t > 0) {
      load_n<T, 8>(u + t - 8, len - t + 8, v);
#pragma unroll
      for (int k = 0; k < K - 1; ++k) e[k] = v[8 - (K - 1) + k];
    } else {
#pragma unroll
      for (int k = 0; k < K - 1; ++k) e[k] = p.x0 ? p.x0[row * (K - 1) + k] : 0.f;
    }
  }
  load_n<T, 8>(u + t, len - t, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) e[K - 1 + k] = v[k];
}

template <int K>
__device__ __forceinline__ float tap_sum(const float* e, const float* w, float bias) {
  float s = bias;
#pragma unroll
  for (int k = 0; k < K; ++k) s = fmaf(w[k], e[k], s);
  return s;
}

// The 32-bit number of a row (B H <= 2^24): batch row and channel by an unsigned
// division, or one for the whole wave.
template <bool WAVE>
__device__ __forceinline__ void place_row(unsigned row, int H, int* b, int* h) {
  if (WAVE) row = __builtin_amdgcn_readfirstlane(row);
  const unsigned q = row / (unsigned)H;
  *b = (int)q;
  *h = (int)(row - q * (unsigned)H);
}

// A row takes lpr lanes (a power of two, at most the workgroup's 256) and, if
// it has more than 8 lpr steps, several workgroups.  WAVE: 64 lanes at least, so
// that a wave's row, weights and end are scalars (4 taps, 2^25 bf16 elements in
// rows of 2048: 38 us with a 64-bit division per lane, 34 so).
template <typename T, int K, bool WAVE>
__global__ __launch_bounds__(256) void shortconv_fwd_kernel(Args p) {
  const unsigned rb = blockIdx.x / (unsigned)p.ntile;
  const int tile = (int)(blockIdx.x - rb * (unsigned)p.ntile);
  unsigned row = rb * (256u / p.lpr) + threadIdx.x / (unsigned)p.lpr;
  if (WAVE) row = __builtin_amdgcn_readfirstlane(row);
  const int t = (tile * p.lpr + (int)(threadIdx.x & (p.lpr - 1))) * 8;
  if (row >= (unsigned)p.rows || (t >= p.L && t > 0)) return;  // without steps the state passes
  int b, h;
  place_row<WAVE>(row, p.H, &b, &h);
  const int len = row_len(p, b);
  const T* u = static_cast<const T*>(p.u) + (size_t)(b * p.su) + (size_t)h * p.L;
  float w[K], e[K + 7], out[8];
  const float bias = load_taps<K>(p, h, w);
  load_window<T, K>(p, u, row, t, len, e);
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = tap_sum<K>(e + j, w, bias);
  if (p.silu) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      out[j] *= __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * out[j]));
  }
  if (t + 8 > len) {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = t + j < len ? out[j] : 0.f;
  }
  store_n<T, 8>(static_cast<T*>(p.y) + (size_t)row * p.L + t, p.L - t, out);
  // the state after the row: the lane that has read the one before it (which
  // may lie in the same place) writes it
  if (K > 1 && t == 0 && p.xT) {
    float s[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      const int i = len + k;
      s[k] = i < K - 1 ? (p.x0 ? p.x0[(size_t)row * (K - 1) + i] : 0.f) : (float)u[i - (K - 1)];
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) p.xT[(size_t)row * (K - 1) + k] = s[k];
  }
}

// One token: a channel to a thread.
template <typename T, int K>
__global__ __launch_bounds__(256) void shortconv_step_kernel(Args p) {
  const unsigned row = blockIdx.x * 256u + threadIdx.x;
  if (row >= (unsigned)p.rows) return;
  int b, h;
  place_row<false>(row, p.H, &b, &h);
  const bool live = !p.lens || p.lens[b] > 0;
  float w[K], e[K];
  const float bias = load_taps<K>(p, h, w);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) e[k] = p.x0 ? p.x0[(size_t)row * (K - 1) + k] : 0.f;
  e[K - 1] = live ? (float)static_cast<const T*>(p.u)[(size_t)(b * p.su) + h] : 0.f;
  float v = tap_sum<K>(e, w, bias), rest;
  if (p.silu) v *= sigmoid_pair(v, &rest);
  static_cast<T*>(p.y)[row] = (T)(live ? v : 0.f);
  if (p.xT) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) p.xT[(size_t)row * (K - 1) + k] = live ? e[k + 1] : e[k];
  }
}

// A value from the next lane of the wave (the last one gets 0).
__device__ __forceinline__ float next_lane(float x) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x130, 0xf, 0xf, true));
}

// Backward: a lane forms the p of its 8 steps and takes its right neighbour's.
// Rows of up to 512 steps belong to lpr <= 64 lanes; of longer ones a wave
// walks tiles of 63 lanes, the last lane only forming the p that the 63rd
// needs.  The sums over a row's (or segment's) steps stay with the lanes until
// its end: a lane's 8 steps in float32, tiles and lanes in float64.
template <typename T, int K, bool WHOLE>
__global__ __launch_bounds__(256) void shortconv_bwd_kernel(Args p) {
  const int lane = threadIdx.x & 63;
  const unsigned wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  constexpr bool whole = WHOLE;  // a wave to a row or segment
  const unsigned rs = whole ? wave : wave * (64u / p.lpr) + lane / p.lpr;
  unsigned row = whole ? rs / (unsigned)p.nseg : rs;
  const int seg = whole ? (int)(rs - row * (unsigned)p.nseg) : 0;
  const bool in = row < (unsigned)p.rows;
  if (!in) row = (unsigned)p.rows - 1;
  int b, h;
  place_row<whole>(row, p.H, &b, &h);
  const int len = row_len(p, b);
  const int gl = whole ? lane : lane & (p.lpr - 1);
  const bool helper = whole && lane == 63;
  const T* u = static_cast<const T*>(p.u) + (size_t)(b * p.su) + (size_t)h * p.L;
  const T* dy = static_cast<const T*>(p.dy) + (size_t)row * p.L;
  const size_t xs = (size_t)row * (K - 1);
  T* du = static_cast<T*>(p.du) + (size_t)(b * p.sdu) + (size_t)h * p.L;
  float w[K];
  typedef typename std::conditional<WHOLE, double, float>::type Sum;
  Sum total[K + 1];
  const float bias = load_taps<K>(p, h, w);
#pragma unroll
  for (int k = 0; k <= K; ++k) total[k] = 0;
  const int step = whole ? 63 * 8 : 0;
  const int lo = seg * p.seg_tiles, hi = min(p.ntile, lo + p.seg_tiles);
  for (int tile = lo; tile < hi; ++tile) {
    const int t = tile * step + gl * 8;
    float e[K + 7], d[8 + K];
    if (in && t < len) {
      load_window<T, K>(p, u, row, t, len, e);
      load_n<T, 8>(dy + t, len - t, d);
    } else {
#pragma unroll
      for (int k = 0; k < K + 7; ++k) e[k] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.f;
    }
    if (p.silu) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = tap_sum<K>(e + j, w, bias);
        float rest;
        const float s = sigmoid_pair(v, &rest);
        d[j] *= fmaf(v * s, rest, s);
      }
      // behind the row's end, where dy counts as 0, whatever the parameters hold
      if (t + 8 > len) {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = t + j < len ? d[j] : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const float v = next_lane(d[j]);
      d[8 + j] = !whole && gl == p.lpr - 1 ? 0.f : v;
    }
    if (in && !helper) {
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) s = fmaf(w[k], d[j + K - 1 - k], s);
        g[j] = s;
      }
      // the state after the row holds its last inputs
      if (p.dx && t + 8 > len - (K - 1) && t < len) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = t + j + K - 1 - len;
          if (i >= 0 && t + j < len) g[j] += p.dx[xs + i];
        }
      }
      if (t + 8 > len) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = t + j < len ? g[j] : 0.f;
      }
      if (t < p.L) store_n<T, 8>(du + t, p.L - t, g);
      if (t < len) {
        float acc[K + 1];
#pragma unroll
        for (int k = 0; k <= K; ++k) acc[k] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int k = 0; k < K; ++k) acc[k] = fmaf(d[j], e[j + k], acc[k]);
          acc[K] += d[j];
        }
#pragma unroll
        for (int k = 0; k <= K; ++k) total[k] += acc[k];
      }
      if (K > 1 && t == 0 && p.dx0) {
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k <= i; ++k)
            if (i - k < 8) s = fmaf(w[k], d[i - k], s);
          if (p.dx && i >= len) s += p.dx[xs + i - len];
          p.dx0[xs + i] = len > 0 ? s : (p.dx ? p.dx[xs + i] : 0.f);
        }
      }
    }
  }
  const int width = whole ? 64 : p.lpr;
  for (int o = 1; o < width; o <<= 1)
#pragma unroll
    for (int k = 0; k <= K; ++k) total[k] += __shfl_xor(total[k], o);
  if (in && gl == 0) {
#pragma unroll
    for (int k = 0; k <= K; ++k) p.part[(size_t)rs * (K + 1) + k] = (float)total[k];
  }
}

// dw, dbias: the rows' and segments' sums in a fixed order, in float64; a wave
// to a channel.
template <int K>
__global__ __launch_bounds__(256) void shortconv_sum_kernel(const float* part, int B, int H,
                                                            int nseg, float* dw, float* dbias) {
  const int h = (int)(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63;
  if (h >= H) return;
  double acc[K + 1];
#pragma unroll
  for (int k = 0; k <= K; ++k) acc[k] = 0.0;
  const long n = (long)B * nseg;
  for (long i = lane; i < n; i += 64) {
    const long b = i / nseg;
    const float* v = part + ((b * H + h) * nseg + (i - b * nseg)) * (K + 1);
#pragma unroll
    for (int k = 0; k <= K; ++k) acc[k] += (double)v[k];
  }
  for (int o = 1; o < 64; o <<= 1)
#pragma unroll
    for (int k = 0; k <= K; ++k) acc[k] += __shfl_xor(acc[k], o);
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) dw[(size_t)h * K + k] = (float)acc[k];
    if (dbias) dbias[h] = (float)acc[K];
  }
}

int pow2_from(int n, int most) {
  int v = 1;
  while (v < n && v < most) v *= 2;
  return v;
}

struct BwdPlan {
  int lpr, ntile, nseg, seg_tiles;
};

// Rows that are too few to fill the device's wave slots are cut into segments
// of whole tiles (256 rows of 65536 steps, float32: 30 us, whole 149; 1024 of
// 16384: 29 and 45; from 8192 rows on they stay whole).
BwdPlan bwd_plan(long rows, int L) {
  BwdPlan pl;
  const int chunks = (L + 7) / 8;
  pl.lpr = pow2_from(chunks, 64);
  pl.ntile = chunks <= 64 ? 1 : (chunks + 62) / 63;
  const long want = std::max(1L, 8192 / std::max(rows, 1L));
  pl.seg_tiles = (int)std::max(1L, pl.ntile / std::min<long>(want, pl.ntile));
  pl.nseg = (pl.ntile + pl.seg_tiles - 1) / pl.seg_tiles;
  return pl;
}

Args make_args(const ShortconvCall& c) {
  Args a{};
  a.u = c.u;
  a.su = c.stride_b;
  a.w = c.w;
  a.bias = c.bias;
  a.lens = c.lens;
  a.B = c.B;
  a.H = c.H;
  a.L = c.L;
  a.silu = c.silu;
  a.rows = (long)c.B * c.H;
  a.x0 = c.x0;
  a.xT = c.xT;
  a.y = c.y;
  a.dy = c.dy;
  a.dx = c.dx;
  a.du = c.du;
  a.sdu = c.grad_stride_b;
  a.dx0 = c.dx0;
  a.part = static_cast<float*>(c.ws);
  a.ntile = a.nseg = a.seg_tiles = a.lpr = 1;
  return a;
}

enum Pass { kForward, kStep, kBackward };

template <typename T, int K>
hipError_t run(const ShortconvCall& c, Pass pass, hipStream_t st) {
  Args a = make_args(c);
  if (pass == kStep) {
    hipLaunchKernelGGL((shortconv_step_kernel<T, K>), dim3((unsigned)((a.rows + 255) / 256)),
                       dim3(256), 0, st, a);
  } else if (pass == kForward) {
    const int chunks = std::max(1, (c.L + 7) / 8);
    a.lpr = pow2_from(chunks, 256);
    a.ntile = (chunks + a.lpr - 1) / a.lpr;
    const long per = 256 / a.lpr, blocks = (a.rows + per - 1) / per * a.ntile;
    if (!launchable(blocks, 256)) return hipErrorInvalidConfiguration;
    if (a.lpr >= 64)
      hipLaunchKernelGGL((shortconv_fwd_kernel<T, K, true>), dim3((unsigned)blocks), dim3(256), 0,
                         st, a);
    else
      hipLaunchKernelGGL((shortconv_fwd_kernel<T, K, false>), dim3((unsigned)blocks), dim3(256), 0,
                         st, a);
  } else {
    BwdPlan pl = bwd_plan(a.rows, c.L);
    a.lpr = pl.lpr;
    a.ntile = pl.ntile;
    a.nseg = pl.nseg;
    a.seg_tiles = pl.seg_tiles;
    if (a.rows > 0) {
      const long per = pl.ntile > 1 ? 4 : 4 * (64 / pl.lpr);
      const long blocks = (a.rows * pl.nseg + per - 1) / per;
      if (!launchable(blocks, 256)) return hipErrorInvalidConfiguration;
      if (pl.ntile > 1)
        hipLaunchKernelGGL((shortconv_bwd_kernel<T, K, true>), dim3((unsigned)blocks), dim3(256), 0,
                           st, a);
      else
        hipLaunchKernelGGL((shortconv_bwd_kernel<T, K, false>), dim3((unsigned)blocks), dim3(256), 0,
                           st, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((shortconv_sum_kernel<K>), dim3((unsigned)((c.H + 3) / 4)), dim3(256), 0, st,
                       a.part, c.B, c.H, pl.nseg, c.dw, c.dbias);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t run_taps(const ShortconvCall& c, Pass pass, hipStream_t st) {
  switch (c.K) {
    case 1: return run<T, 1>(c, pass, st);
    case 2: return run<T, 2>(c, pass, st);
    case 3: return run<T, 3>(c, pass, st);
    case 4: return run<T, 4>(c, pass, st);
    case 5: return run<T, 5>(c, pass, st);
    case 6: return run<T, 6>(c, pass, st);
    case 7: return run<T, 7>(c, pass, st);
    default: return run<T, 8>(c, pass, st);
  }
}

hipError_t run_type(const ShortconvCall& c, Pass pass, int dtype, hipStream_t st) {
  switch (dtype) {
    case 0: return run_taps<float>(c, pass, st);
    case 1: return run_taps<__bf16>(c, pass, st);
    default: return run_taps<_Float16>(c, pass, st);
  }
}

}  // namespace

size_t shortconv_workspace(int B, int H, int K, int L) {
  const long rows = (long)B * H;
  return align_up((size_t)rows * bwd_plan(rows, L).nseg * (K + 1) * sizeof(float), 256);
}

hipError_t launch_shortconv_forward(const ShortconvCall& c, int dtype, hipStream_t st) {
  return run_type(c, kForward, dtype, st);
}
hipError_t launch_shortconv_step(const ShortconvCall& c, int dtype, hipStream_t st) {
  return run_type(c, kStep, dtype, st);
}
hipError_t launch_shortconv_backward(const ShortconvCall& c, int dtype, hipStream_t st) {
  return run_type(c, kBackward, dtype, st);
}

}  // namespace dssm
