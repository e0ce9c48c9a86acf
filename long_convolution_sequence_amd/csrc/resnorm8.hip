// The residual sum and norm ahead of a product in 8 bits: over the H channels
// of every (b, t),
//
//   o = x + scale norm(y) w_post silu(g)   or   x + y   (or x alone),
//   n = norm(o) w,  s = max_h |n| / M,  q = n / s rounded,
//
// M = 127 (whole numbers) or 448 (e4m3).  q leaves channels fastest, as an 8-bit
// product reads its operand, s one float32 a step.  With d = o - mean and m =
// max |d w|, q = d w M / m and s = m rstd / M: the factor of the norm meets only
// the scale.
//
// Memory bounds it: o's inputs read once, o written, a byte a channel written (2^25
// bf16 elements in rows of 64 to 1024 channels, inputs from memory: x + y 62 to 68 us,
// 3.8 TB/s; with the norm and gate of y 74 to 83, 4 TB/s; inputs that a cache still
// holds, x + y 45).
// A workgroup takes a strip of LT VE steps with all its channels, o held in
// registers as stored; four neighbouring channels to a lane, so that their bytes
// of a step make one word, turned to rows of channels through LDS.
#include <algorithm>
#include <type_traits>

#include "dssm_internal.h"
#include "seq_common.h"
#include "strip.h"

namespace dssm {
namespace {

struct Args {
  const void *x, *y, *g;
  long long sg;
  const float *w_post, *scale, *w;
  const int* lens;
  int B, H, L;
  int ntile, per;
  float eps;
  int e4m3;
  void* o;
  uint8_t* q;
  float *qs, *stats;
};

// Sums and largest bit patterns of VE steps over the workgroup's lanes of the
// same steps; every thread gets both.  buf: [NT / 64 + 1][2 LT VE] words.
template <int LT>
__device__ __forceinline__ uint32_t column_max(uint32_t v) {
  const auto move = [](uint32_t x, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, true);
  };
  if (LT <= 1) v = max(v, move(v, std::integral_constant<int, 0xb1>()));
  if (LT <= 2) v = max(v, move(v, std::integral_constant<int, 0x4e>()));
  if (LT <= 4) v = max(v, move(v, std::integral_constant<int, 0x124>()));
  if (LT <= 8) v = max(v, move(v, std::integral_constant<int, 0x128>()));
  if (LT <= 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
  }
  if (LT <= 32) {
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
  }
  return v;
}

template <int NT, int LT, int VE>
__device__ __forceinline__ void strip_sum_max(float* sum, uint32_t* top, uint32_t* buf) {
  constexpr int W = NT / 64, C = LT * VE;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lt = lane % LT;
#pragma unroll
  for (int k = 0; k < VE; ++k) {
    sum[k] = column_sum<LT>(sum[k]);
    top[k] = column_max<LT>(top[k]);
  }
  __syncthreads();  // the buffer's last readers are done
  if (lane < LT)
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      buf[wave * 2 * C + lt * VE + k] = __float_as_uint(sum[k]);
      buf[wave * 2 * C + C + lt * VE + k] = top[k];
    }
  __syncthreads();
  // each column is one thread's: no other reads or writes it before the barrier
  for (int c = threadIdx.x; c < C; c += NT) {
    float s = 0.f;
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      s += __uint_as_float(buf[w * 2 * C + c]);
      m = max(m, buf[w * 2 * C + C + c]);
    }
    buf[W * 2 * C + c] = __float_as_uint(s);
    buf[W * 2 * C + C + c] = m;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < VE; ++k) {
    sum[k] = __uint_as_float(buf[W * 2 * C + lt * VE + k]);
    top[k] = buf[W * 2 * C + C + lt * VE + k];
  }
}

// A step's scale and what its d w are multiplied by, from the largest |d w|: a
// step that holds Inf or NaN stands for NaN, one below 2^-100 for 0.
__device__ __forceinline__ float step_scale(uint32_t top, float rstd, float most, bool live,
                                            float* mul) {
  const float m = __uint_as_float(top);
  const bool bad = top >= 0x7f800000u, none = !live || m < 0x1p-100f;
  *mul = bad || none ? 0.f : most / m;
  if (none) return 0.f;
  return bad ? __uint_as_float(0x7fc00000u) : m * rstd * (1.f / most);
}

// Four values in [-M, M] as bytes, rounded to nearest even.
__device__ __forceinline__ uint32_t bytes4(const float* v, int e4m3) {
  if (e4m3) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  }
  uint32_t b[4];
#pragma unroll
  // added to 3 2^22 a value is rounded to a whole number, to even, in the low byte
  for (int k = 0; k < 4; ++k) b[k] = __float_as_uint(v[k] + 12582912.f);
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400);
  const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100);
}

// d w in one byte's range; what a bad step's holds is dropped (0 times Inf is NaN).
__device__ __forceinline__ float in_range(float v, float mul, float most) {
  return mul == 0.f ? 0.f : __builtin_amdgcn_fmed3f(v * mul, -most, most);
}

// n bytes of w, at any address.
__device__ __forceinline__ void store_bytes(uint8_t* p, int n, uint2 w) {
  typedef uint32_t two __attribute__((ext_vector_type(2), aligned(1)));
  if (n >= 8) {
    *reinterpret_cast<two*>(p) = two{w.x, w.y};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
  }
}

// FORM: 0 n of x alone, 1 o = x + y, 2 with the norm, scale and gate.  A lane's
// channel j of KH is 4 NR (j / 4) + 4 rs + j % 4.
template <typename T, bool LAYER, int FORM, int NT, int LT, int KH>
__global__ __launch_bounds__(NT) void resnorm8_kernel(Args p) {
  constexpr int VE = 16 / sizeof(T), NR = NT / LT, S = LT * VE, C4 = 4 * NR;
  // a row of C4 bytes and 8 more: the lanes of different steps meet different banks
  constexpr int PITCH = C4 / 4 + 2;
  typedef Packed<T, VE> Vec;
  __shared__ uint32_t buf[(NT / 64 + 1) * 2 * S];
  __shared__ uint32_t turn[S][PITCH];
  const int strip = strip_of_block(blockIdx.x, p.per);
  if (strip >= p.B * p.ntile) return;
  const int b = __builtin_amdgcn_readfirstlane(strip / p.ntile);
  const int lt = threadIdx.x % LT, rs = threadIdx.x / LT;
  const int t0 = (strip - b * p.ntile) * S, t = t0 + lt * VE;
  const int len = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  const int nv = min(max(len - t, 0), VE), ns = min(max(p.L - t, 0), VE);
  const bool whole = t0 + S <= len;
  const float inv_h = 1.f / (float)p.H;
  const size_t base = (size_t)b * p.H * p.L + t0;
  const size_t plane = (size_t)p.B * p.L, at = (size_t)b * p.L + t;
  const auto channel = [&](int j) { return (j / 4) * C4 + rs * 4 + (j & 3); };
  // groups of channels that all lanes have need no check (a scalar's choice)
  const auto has = [&](int j) { return (j / 4 + 1) * C4 <= p.H || channel(j) < p.H; };
  // A lane's place in a strip's first four channels, made opaque: the compiler
  // would keep the address of every channel of every tensor in registers.
  const size_t own = ((size_t)rs * 4 * p.L + lt * VE) * sizeof(T);
  const auto spot = [&](const T* row, int j) {
    size_t o = own;
    asm volatile("" : "+v"(o));
    const char* c = reinterpret_cast<const char*>(row + (size_t)((j / 4) * C4 + (j & 3)) * p.L);
    return const_cast<T*>(reinterpret_cast<const T*>(c + o));
  };
  // channels past the last one, and steps behind the row's end, are 0
  const auto get = [&](Vec& v, const T* row, int j) {
    if (whole && (j / 4 + 1) * C4 <= p.H)
      v.load(spot(row, j));
    else
      v.load(spot(row, j), has(j) ? nv : 0, (T)0.f);
  };
  // with many channels held, no more than four of them in flight
  const auto pause = [&](int j) {
    if (KH > 8 && j % 4 == 0) __builtin_amdgcn_sched_barrier(0);
  };
  // forget what was derived from the held words (their float32 values)
  const auto refresh = [&](Vec* v) {
#pragma unroll
    for (int j = 0; j < KH; ++j) v[j].refresh();
  };
  const T* x = static_cast<const T*>(p.x) + base;
  const T* y = static_cast<const T*>(p.y) + (FORM ? base : 0);
  T* o = static_cast<T*>(p.o) + (FORM ? base : 0);
  Vec a[KH];
  float mean[1][VE], s[1][VE];
  uint32_t top[VE];
  if (FORM == 2) {
    const T* g = static_cast<const T*>(p.g) + (p.g ? (size_t)(b * p.sg) + t0 : 0);
#pragma unroll
    for (int j = 0; j < KH; ++j) get(a[j], y, j);
#pragma unroll
    for (int k = 0; k < VE; ++k) mean[0][k] = s[0][k] = 0.f;
    if (LAYER) {
#pragma unroll
      for (int j = 0; j < KH; ++j)
        if (has(j))
#pragma unroll
          for (int k = 0; k < VE; ++k) mean[0][k] += a[j][k];
      strip_sum<NT, LT, VE, 1>(mean, reinterpret_cast<float*>(buf));
#pragma unroll
      for (int k = 0; k < VE; ++k) mean[0][k] *= inv_h;
    }
#pragma unroll
    for (int j = 0; j < KH; ++j)
      if (!LAYER || has(j))
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float d = a[j][k] - mean[0][k];
          s[0][k] = fmaf(d, d, s[0][k]);
        }
    refresh(a);
    strip_sum<NT, LT, VE, 1>(s, reinterpret_cast<float*>(buf));
    float rstd[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k)
      rstd[k] = k < nv ? __builtin_amdgcn_rsqf(fmaf(s[0][k], inv_h, p.eps)) : 0.f;
    if (p.stats && rs == 0) {
      if (LAYER) store_n<float, VE>(p.stats + at, ns, mean[0]);
      store_n<float, VE>(p.stats + (LAYER ? plane : 0) + at, ns, rstd);
    }
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      pause(j);
      const int h = channel(j);
      const bool in = has(j);
      Vec xv, gv;
      get(xv, x, j);
      if (p.g) get(gv, g, j);
      const float c = in ? p.w_post[h] * p.scale[h] : 0.f;
      float out[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        float silu = 1.f;
        if (p.g) silu = gv[k] * __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * gv[k]));
        out[k] = fmaf((a[j][k] - mean[0][k]) * rstd[k] * c, silu, xv[k]);
      }
      live_only<VE>(out, nv, whole);
      a[j].set(out);
      a[j].refresh();
      if (in) a[j].store(spot(o, j), ns);
    }
  } else if (FORM == 1) {
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      pause(j);
      Vec xv, yv;
      get(xv, x, j);
      get(yv, y, j);
      float out[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) out[k] = xv[k] + yv[k];
      a[j].set(out);
      a[j].refresh();
      if (has(j)) a[j].store(spot(o, j), ns);
    }
  } else {
#pragma unroll
    for (int j = 0; j < KH; ++j) get(a[j], x, j);
  }
  // the norm is of the stream as it is stored
#pragma unroll
  for (int k = 0; k < VE; ++k) {
    mean[0][k] = s[0][k] = 0.f;
    top[k] = 0;
  }
  if (LAYER) {
#pragma unroll
    for (int j = 0; j < KH; ++j)
#pragma unroll
      for (int k = 0; k < VE; ++k) mean[0][k] += a[j][k];
    refresh(a);
    strip_sum<NT, LT, VE, 1>(mean, reinterpret_cast<float*>(buf));
#pragma unroll
    for (int k = 0; k < VE; ++k) mean[0][k] *= inv_h;
  }
#pragma unroll
  for (int j = 0; j < KH; ++j) {
    pause(j);
    if (!has(j)) continue;
    const float w = p.w[channel(j)];
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      const float d = a[j][k] - mean[0][k];
      s[0][k] = fmaf(d, d, s[0][k]);
      top[k] = max(top[k], abs_bits(d * w));
    }
  }
  refresh(a);
  strip_sum_max<NT, LT, VE>(s[0], top, buf);
  const float most = p.e4m3 ? 448.f : 127.f;
  float rstd[VE], unit[VE], mul[VE];
#pragma unroll
  for (int k = 0; k < VE; ++k) {
    rstd[k] = k < nv ? __builtin_amdgcn_rsqf(fmaf(s[0][k], inv_h, p.eps)) : 0.f;
    unit[k] = step_scale(top[k], rstd[k], most, k < nv, &mul[k]);
  }
  if (rs == 0) {
    if (p.stats) {
      if (LAYER) store_n<float, VE>(p.stats + 2 * plane + at, ns, mean[0]);
      store_n<float, VE>(p.stats + (LAYER ? 3 : 1) * plane + at, ns, rstd);
    }
    store_n<float, VE>(p.qs + at, ns, unit);
  }
#pragma unroll
  for (int j4 = 0; j4 < KH / 4; ++j4) {
    const int h0 = j4 * C4;
    if (h0 >= p.H) break;
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = h0 + rs * 4 + i < p.H ? p.w[h0 + rs * 4 + i] : 0.f;
    __syncthreads();  // the last rows are out
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = in_range((a[4 * j4 + i][k] - mean[0][k]) * w[i], mul[k], most);
      turn[lt * VE + k][rs] = bytes4(v, p.e4m3);
    }
    __syncthreads();
    const int count = min(C4, p.H - h0);
    for (int i = threadIdx.x; i < S * (C4 / 8); i += NT) {
      const int row = i / (C4 / 8), c = i % (C4 / 8) * 8;
      if (t0 + row >= p.L || c >= count) continue;
      const uint2 v = *reinterpret_cast<const uint2*>(&turn[row][c / 4]);
      store_bytes(p.q + ((size_t)b * p.L + t0 + row) * p.H + h0 + c, count - c, v);
    }
  }
}

// v summed, top's largest, over a row's NT threads; buf: a word of each per wave.
template <int NT>
__device__ __forceinline__ void row_sum_max(float& v, uint32_t& top, uint32_t (*buf)[NT / 64]) {
  constexpr int W = NT / 64;
  v = column_sum<1>(v);
  top = column_max<1>(top);
  if (W == 1) return;
  if ((threadIdx.x & 63) == 0) {
    buf[0][threadIdx.x >> 6] = __float_as_uint(v);
    buf[1][threadIdx.x >> 6] = top;
  }
  __syncthreads();
  v = 0.f;
  top = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    v += __uint_as_float(buf[0][w]);
    top = max(top, buf[1][w]);
  }
}

// A single step: the channels are the contiguous axis, 8 of them to a thread, a
// row to a workgroup (rows of up to 512 channels to a wave, four to a
// workgroup).  Latency bounds it: everything is asked for before the first sum.
constexpr int token_rows(int NT) { return NT == 64 ? 4 : 1; }
template <typename T, bool LAYER, int FORM, int NT>
__global__ __launch_bounds__(NT * token_rows(NT)) void resnorm8_token_kernel(Args p) {
  __shared__ uint32_t buf[4][2][NT / 64];
  const int b = blockIdx.x * token_rows(NT) + threadIdx.y, h = threadIdx.x * 8;
  if (b >= p.B) return;
  const int m = min(max(p.H - h, 0), 8);
  const bool live = !p.lens || p.lens[b] > 0;
  const int nv = live ? m : 0;
  const size_t at = (size_t)b * p.H + h;
  const float inv_h = 1.f / (float)p.H;
  float x[8], y[8], g[8], wp[8], sc[8], w[8];
  load_n<T, 8>(static_cast<const T*>(p.x) + at, nv, x);
  if (FORM) load_n<T, 8>(static_cast<const T*>(p.y) + at, nv, y);
  if (FORM == 2) {
    if (p.g) load_n<T, 8>(static_cast<const T*>(p.g) + ((size_t)(b * p.sg) + h), nv, g);
    load_n<float, 8>(p.w_post + h, m, wp);
    load_n<float, 8>(p.scale + h, m, sc);
  }
  load_n<float, 8>(p.w + h, m, w);
  uint32_t top = 0;
  // mean (layer norm) and factor of a row; top: of the largest |d w|
  const auto stats = [&](const float* a, int pair, const float* weight, float* mean) {
    float s = 0.f;
    *mean = 0.f;
    if (LAYER) {
#pragma unroll
      for (int k = 0; k < 8; ++k) s += a[k];  // 0 past the row's end
      row_sum_max<NT>(s, top, buf[2 * pair]);
      *mean = s * inv_h;
    }
    s = 0.f;
    top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = k < m ? a[k] - *mean : 0.f;
      s = fmaf(d, d, s);
      if (weight) top = max(top, abs_bits(d * weight[k]));
    }
    row_sum_max<NT>(s, top, buf[2 * pair + 1]);
    return live ? __builtin_amdgcn_rsqf(fmaf(s, inv_h, p.eps)) : 0.f;
  };
  float mean;
  if (FORM) {
    if (FORM == 2) {
      const float rstd = stats(y, 0, nullptr, &mean);
      if (p.stats && threadIdx.x == 0) {
        if (LAYER) p.stats[b] = mean;
        p.stats[(LAYER ? p.B : 0) + b] = rstd;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float silu = 1.f;
        if (p.g) silu = g[k] * __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * g[k]));
        x[k] = fmaf((y[k] - mean) * rstd * (wp[k] * sc[k]), silu, x[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] += y[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < nv ? (float)(T)x[k] : 0.f;
    store_n<T, 8>(static_cast<T*>(p.o) + at, m, x);
  }
  const float rstd = stats(x, 1, w, &mean);
  const float most = p.e4m3 ? 448.f : 127.f;
  float mul;
  const float unit = step_scale(top, rstd, most, live, &mul);
  if (threadIdx.x == 0) {
    if (p.stats) {
      if (LAYER) p.stats[2 * p.B + b] = mean;
      p.stats[(LAYER ? 3 : 1) * p.B + b] = rstd;
    }
    p.qs[b] = unit;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = in_range((x[k] - mean) * w[k], mul, most);
  store_bytes(p.q + at, m, make_uint2(bytes4(x, p.e4m3), bytes4(x + 4, p.e4m3)));
}

template <typename T, bool LAYER, int FORM, int NT, int LT, int KH>
void strips(Args a, hipStream_t st) {
  constexpr int S = LT * (16 / (int)sizeof(T));
  a.ntile = (a.L + S - 1) / S;
  a.per = (a.B * a.ntile + 7) / 8;
  hipLaunchKernelGGL((resnorm8_kernel<T, LAYER, FORM, NT, LT, KH>), dim3((unsigned)a.per * 8),
                     dim3(NT), 0, st, a);
}

template <typename T, bool LAYER, int FORM, int NT>
void token(const Args& a, hipStream_t st) {
  constexpr int R = token_rows(NT);
  hipLaunchKernelGGL((resnorm8_token_kernel<T, LAYER, FORM, NT>), dim3((unsigned)(a.B + R - 1) / R),
                     dim3(NT, R), 0, st, a);
}

// Workgroups as small as hold the channels: those of a compute unit are in different
// parts of their work, so that one's loads run while another sums and rounds.  64
// channels in 64 threads and in 256: 74 us and 181 (2^25 bf16 elements, gate and norm
// of y); 1024 in 512 threads of 8 channels and in 1024 of 4: 84 and 98.  2048 channels
// of 16 bits in 512 threads of 16 and in 1024 of 8: 92 and 97; of 32 bits, 171 and 165.
// (The same inputs every pass, of either side.)  Layer norms of 2049 to 4096 channels of
// 16 bits keep 4 to 26 registers in scratch, beyond that 1 or 2.
template <typename T, bool LAYER, int FORM>
hipError_t run(const Args& a, hipStream_t st) {
  constexpr int kWide = sizeof(T) == 2 ? 512 : 1024;
  if (a.L == 1)
    a.H <= 512    ? token<T, LAYER, FORM, 64>(a, st)
    : a.H <= 2048 ? token<T, LAYER, FORM, 256>(a, st)
                  : token<T, LAYER, FORM, 1024>(a, st);
  else
    a.H <= 64     ? strips<T, LAYER, FORM, 64, 4, 4>(a, st)
    : a.H <= 128  ? strips<T, LAYER, FORM, 128, 4, 4>(a, st)
    : a.H <= 256  ? strips<T, LAYER, FORM, 256, 4, 4>(a, st)
    : a.H <= 512  ? strips<T, LAYER, FORM, 512, 4, 4>(a, st)
    : a.H <= 1024 ? strips<T, LAYER, FORM, 512, 4, 8>(a, st)
    : a.H <= 2048 ? strips<T, LAYER, FORM, kWide, 4, 8192 / kWide>(a, st)
    : a.H <= 4096 ? strips<T, LAYER, FORM, 1024, 4, 16>(a, st)
                  : strips<T, LAYER, FORM, 1024, 2, 16>(a, st);
  return hipGetLastError();
}

template <typename T, bool LAYER>
hipError_t run_form(const Args& a, hipStream_t st) {
  if (!a.y) return run<T, LAYER, 0>(a, st);
  return a.w_post ? run<T, LAYER, 2>(a, st) : run<T, LAYER, 1>(a, st);
}

}  // namespace

hipError_t launch_resnorm8(const ResnormCall& c, int dtype, const Resnorm8Out& out,
                           hipStream_t st) {
  Args a{};
  a.x = c.x;
  a.y = c.y;
  a.g = c.g;
  a.sg = c.stride_g;
  a.w_post = c.w_post;
  a.scale = c.scale;
  a.w = c.w_pre;
  a.lens = c.lens;
  a.B = c.B;
  a.H = c.H;
  a.L = c.L;
  a.eps = c.eps;
  a.e4m3 = out.e4m3;
  a.o = c.o;
  a.q = static_cast<uint8_t*>(out.q);
  a.qs = out.qs;
  a.stats = c.stats;
  switch (dtype) {
    case 0: return c.layer ? run_form<float, true>(a, st) : run_form<float, false>(a, st);
    case 1: return c.layer ? run_form<__bf16, true>(a, st) : run_form<__bf16, false>(a, st);
    default: return c.layer ? run_form<_Float16, true>(a, st) : run_form<_Float16, false>(a, st);
  }
}

}  // namespace dssm
