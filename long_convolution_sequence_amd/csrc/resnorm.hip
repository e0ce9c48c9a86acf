// The residual norm around a layer, over activations [B, H, L] with time
// fastest; every (b, t) column is normalised over its H channels:
//
//   v = norm(y) w_post,  o = x + scale v silu(g),  n = norm(o) w_pre
//   norm(a) = (a - mean) rstd,  rstd = 1 / sqrt(mean((a - mean)^2) + eps)
//   (mean = 0 for the root-mean-square norm)
//
// and its gradients.  With yh, oh the normalised y and o, P = dn w_pre and
// k = scale silu(g) w_post:
//
//   t   = do + rstd_o (P - oh mean(P oh) - mean(P)) = dx
//   dy  = rstd_y (R - yh mean(R yh) - mean(R)),  R = t k
//   dg  = t scale yh w_post silu'(g)
//   dw_pre = sum dn oh,  dscale = sum t yh w_post silu(g),  dw_post = sum t scale silu(g) yh
//   (the mean(P), mean(R) terms only for the layer norm; sums over b, t).
// silu'(g) = s + silu(g) (1 - s), s = sigmoid(g), with 1 - s to full relative
// precision: silu + s - silu s would lose the digits of 1 next to a large g.
//
// Layout: the normalised axis is the strided one.  A workgroup takes a strip
// of LT VE steps (VE consecutive steps to a lane, LT lanes side by side) and
// all H channels, NT / LT channels at a time, so that every row segment it
// touches is one run of LT VE elements; sums over channels are joined across
// lanes by shuffles and across waves through LDS.
#include <algorithm>

#include "dssm_internal.h"
#include "seq_common.h"

namespace dssm {
namespace {

struct Args {
  const void *x, *y, *g;
  long long sg;
  const float *w_post, *scale, *w_pre;
  const int* lens;
  int B, H, L;
  int ntile, per;  // strips of a batch row, strips of a die
  float eps;
  void *o, *n;
  float* stats;
  const void *d_o, *d_n;
  void *dx, *dy, *dg;
  long long sdg;
  float* part;         // [workgroups][2][H]
};

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

// Mean (layer norm) and factor of the columns held in a[KH], per step.
template <bool LAYER, int NT, int LT, int VE, int KH, typename Vec>
__device__ __forceinline__ void column_stats(const Vec* a, int H, int rs, float inv_h, float eps,
                                             int nv, float* buf, float (*mean)[VE],
                                             float (*rstd)[VE]) {
  constexpr int NR = NT / LT;
#pragma unroll
  for (int k = 0; k < VE; ++k) mean[0][k] = 0.f;
  if (LAYER) {
#pragma unroll
    for (int j = 0; j < KH; ++j)
      if (rs + j * NR < H)
#pragma unroll
        for (int k = 0; k < VE; ++k) mean[0][k] += a[j][k];
    strip_sum<NT, LT, VE, 1>(mean, buf);
#pragma unroll
    for (int k = 0; k < VE; ++k) mean[0][k] *= inv_h;
  }
#pragma unroll
  for (int k = 0; k < VE; ++k) rstd[0][k] = 0.f;
#pragma unroll
  for (int j = 0; j < KH; ++j)
    if (rs + j * NR < H)
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const float d = a[j][k] - mean[0][k];
        rstd[0][k] = fmaf(d, d, rstd[0][k]);
      }
  strip_sum<NT, LT, VE, 1>(rstd, buf);
#pragma unroll
  for (int k = 0; k < VE; ++k)
    rstd[0][k] = k < nv ? __builtin_amdgcn_rsqf(fmaf(rstd[0][k], inv_h, eps)) : 0.f;
}

// Where a lane's KH channels lie in a batch row's strip: channel rs + j NR at
// a distance the workgroup shares (in scalar registers) plus the lane's own in
// 32 bits, which a load adds by itself.  Lanes past the last channel take the
// last one's place; they read it again and never count or store it.
template <typename T, int NR, int KH>
struct Rows {
  uint32_t off[KH];
  int H, L;
  __device__ __forceinline__ Rows(int rs, int first, int H_, int L_) : H(H_), L(L_) {
#pragma unroll
    for (int j = 0; j < KH; ++j)
      off[j] = ((uint32_t)(min(rs + j * NR, H - 1) - min(j * NR, H - 1)) * (uint32_t)L +
                (uint32_t)first) * (uint32_t)sizeof(T);
  }
  // strip: the strip's first step in the batch row's first channel
  __device__ __forceinline__ const T* at(const T* strip, int j) const {
    const char* row = reinterpret_cast<const char*>(strip + (size_t)min(j * NR, H - 1) * L);
    return reinterpret_cast<const T*>(row + off[j]);
  }
  __device__ __forceinline__ T* at(T* strip, int j) const {
    return const_cast<T*>(at(const_cast<const T*>(strip), j));
  }
  // A whole strip is read without a guard; of one that ends early `nv` of the
  // lane's steps are live, the others 0.
  template <int VE>
  __device__ __forceinline__ void load(Packed<T, VE>* v, const T* strip, int nv, bool whole) const {
    if (whole) {
#pragma unroll
      for (int j = 0; j < KH; ++j) v[j].load(at(strip, j));
    } else {
#pragma unroll
      for (int j = 0; j < KH; ++j) v[j].load(at(strip, j), nv, (T)0.f);
    }
  }
};

template <typename T, int VE, int KH>
__device__ __forceinline__ void no_rows(Packed<T, VE>* v) {
#pragma unroll
  for (int j = 0; j < KH; ++j)
#pragma unroll
    for (int k = 0; k < Packed<T, VE>::W; ++k) v[j].w[k] = 0;
}

// The whole strip in registers: all inputs are asked for before the first sum
// over channels is formed, so that the sums' barriers wait for memory once.
template <typename T, bool LAYER, int NT, int LT, int VE, int KH>
__global__ __launch_bounds__(NT) void resnorm_fwd_kernel(Args p) {
  typedef Packed<T, VE> Vec;
  constexpr int NR = NT / LT;
  __shared__ float buf[(NT / 64) * LT * VE];
  const int strip = strip_of_block(blockIdx.x, p.per);
  if (strip >= p.B * p.ntile) return;
  const int b = __builtin_amdgcn_readfirstlane(strip / p.ntile);
  const int lt = threadIdx.x % LT, rs = threadIdx.x / LT;
  const int t0 = (strip - b * p.ntile) * (LT * VE), t = t0 + lt * VE;
  const int len = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  const int nv = min(max(len - t, 0), VE), ns = min(max(p.L - t, 0), VE);
  const bool whole = t0 + LT * VE <= len;
  const float inv_h = 1.f / (float)p.H;
  const size_t base = (size_t)b * p.H * p.L + t0;
  const size_t plane = (size_t)p.B * p.L;
  const size_t at = (size_t)b * p.L + t;
  const Rows<T, NR, KH> rows(rs, lt * VE, p.H, p.L);
  const T* x = static_cast<const T*>(p.x) + base;
  Vec a[KH];
  float mean[1][VE], rstd[1][VE];
  if (p.y) {
    Vec xv[KH], gv[KH];
    const T* g = static_cast<const T*>(p.g) + (p.g ? (size_t)(b * p.sg) + t0 : 0);
    rows.load(a, static_cast<const T*>(p.y) + base, nv, whole);
    if (p.g) rows.load(gv, g, nv, whole);
    rows.load(xv, x, nv, whole);
    column_stats<LAYER, NT, LT, VE, KH>(a, p.H, rs, inv_h, p.eps, nv, buf, mean, rstd);
#pragma unroll
    for (int j = 0; j < KH; ++j) a[j].refresh();
    if (p.stats && rs == 0) {
      if (LAYER) store_n<float, VE>(p.stats + at, ns, mean[0]);
      store_n<float, VE>(p.stats + (LAYER ? plane : 0) + at, ns, rstd[0]);
    }
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      const int h = rs + j * NR;
      const bool in = h < p.H;
      const float c = in ? p.w_post[h] * p.scale[h] : 0.f;
      float out[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        float silu = 1.f;
        if (p.g)
          silu = gv[j][k] * __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * gv[j][k]));
        const float v = (a[j][k] - mean[0][k]) * rstd[0][k];
        out[k] = fmaf(v * c, silu, xv[j][k]);
      }
      live_only<VE>(out, nv, whole);
      a[j].set(out);
      if (in) a[j].store(rows.at(static_cast<T*>(p.o) + base, j), ns);
    }
  } else {
    rows.load(a, x, nv, whole);
  }
  if (!p.n) return;
  // the norm before the next block is of the stream as it is stored
  column_stats<LAYER, NT, LT, VE, KH>(a, p.H, rs, inv_h, p.eps, nv, buf, mean, rstd);
  if (p.stats && rs == 0) {
    if (LAYER) store_n<float, VE>(p.stats + 2 * plane + at, ns, mean[0]);
    store_n<float, VE>(p.stats + (LAYER ? 3 : 1) * plane + at, ns, rstd[0]);
  }
#pragma unroll
  for (int j = 0; j < KH; ++j) {
    const int h = rs + j * NR;
    if (h >= p.H) continue;
    const float w = p.w_pre[h];
    float out[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) out[k] = (a[j][k] - mean[0][k]) * rstd[0][k] * w;
    live_only<VE>(out, nv, whole);
    store_n<T, VE>(rows.at(static_cast<T*>(p.n) + base, j), ns, out);
  }
}

// v summed over a row's NT threads, in the same order everywhere; buf: one
// float per wave, of this sum alone (so one barrier does).
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  constexpr int W = NT / 64;
  v = column_sum<1>(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  return lanes_sum<W>(buf[threadIdx.x & (W - 1)]);
}

// Mean (layer norm) and factor of a row held 8 channels to a thread, m of them.
template <bool LAYER, int NT>
__device__ __forceinline__ void row_stats(const float* a, int m, float inv_h, float eps,
                                          float (*buf)[NT / 64], float* mean, float* rstd) {
  *mean = 0.f;
  if (LAYER) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += a[k];  // 0 past the row's end
    *mean = row_sum<NT>(s, buf[0]) * inv_h;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float d = k < m ? a[k] - *mean : 0.f;
    s = fmaf(d, d, s);
  }
  *rstd = __builtin_amdgcn_rsqf(fmaf(row_sum<NT>(s, buf[1]), inv_h, eps));
}

// A single step: the channels are the contiguous axis, 8 of them to a thread.
// A row to a workgroup of NT threads; rows of up to 512 channels to a wave each
// (NT = 64), four to a workgroup.  What bounds it is latency: everything the
// row needs, parameters too, is asked for before the first sum (a graph of 50
// calls, bf16, us a call: 64 rows of 4096 channels 3.6, 1 row of 1024 2.8, with
// the parameters asked for after the sums and channels side by side 6.8, 3.5).
constexpr int token_rows(int NT) { return NT == 64 ? 4 : 1; }
template <typename T, bool LAYER, int NT>
__global__ __launch_bounds__(NT * token_rows(NT)) void resnorm_token_kernel(Args p) {
  __shared__ float buf[4][NT / 64];
  const int b = blockIdx.x * token_rows(NT) + threadIdx.y, h = threadIdx.x * 8;
  if (b >= p.B) return;
  const int m = min(max(p.H - h, 0), 8);
  const bool live = !p.lens || p.lens[b] > 0;
  const int nv = live ? m : 0;
  const size_t at = (size_t)b * p.H + h;
  const float inv_h = 1.f / (float)p.H;
  float x[8], y[8], g[8], wp[8], sc[8], wn[8];
  load_n<T, 8>(static_cast<const T*>(p.x) + at, nv, x);
  if (p.y) {
    load_n<T, 8>(static_cast<const T*>(p.y) + at, nv, y);
    if (p.g) load_n<T, 8>(static_cast<const T*>(p.g) + ((size_t)(b * p.sg) + h), nv, g);
    load_n<float, 8>(p.w_post + h, m, wp);
    load_n<float, 8>(p.scale + h, m, sc);
  }
  if (p.n) load_n<float, 8>(p.w_pre + h, m, wn);
  float mean, rstd;
  if (p.y) {
    row_stats<LAYER, NT>(y, m, inv_h, p.eps, buf, &mean, &rstd);
    if (!live) rstd = 0.f;
    if (p.stats && threadIdx.x == 0) {
      if (LAYER) p.stats[b] = mean;
      p.stats[(LAYER ? p.B : 0) + b] = rstd;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float silu = 1.f;
      if (p.g) silu = g[k] * __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * g[k]));
      x[k] = fmaf((y[k] - mean) * rstd * (wp[k] * sc[k]), silu, x[k]);
      x[k] = k < nv ? (float)(T)x[k] : 0.f;  // the second norm is of the stream as it is stored
    }
    store_n<T, 8>(static_cast<T*>(p.o) + at, m, x);
  }
  if (!p.n) return;
  row_stats<LAYER, NT>(x, m, inv_h, p.eps, buf + 2, &mean, &rstd);
  if (!live) rstd = 0.f;
  if (p.stats && threadIdx.x == 0) {
    if (LAYER) p.stats[2 * p.B + b] = mean;
    p.stats[(LAYER ? 3 : 1) * p.B + b] = rstd;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = live ? (x[k] - mean) * rstd * wn[k] : 0.f;
  store_n<T, 8>(static_cast<T*>(p.n) + at, m, x);
}

// One strip of a workgroup that loops over its channels.
template <typename T, int NT, int LT, int VE>
struct WideStrip {
  typedef Packed<T, VE> Vec;
  static constexpr int NR = NT / LT;
  int b, t0, t, nv, ns, H, L, lt, rs;
  bool whole;
  size_t base, at, plane;
  __device__ __forceinline__ WideStrip(const Args& p, int strip) {
    b = __builtin_amdgcn_readfirstlane(strip / p.ntile);
    lt = threadIdx.x % LT;
    rs = threadIdx.x / LT;
    t0 = (strip - b * p.ntile) * (LT * VE);
    t = t0 + lt * VE;
    H = p.H;
    L = p.L;
    const int len = p.lens ? min(max(p.lens[b], 0), L) : L;
    nv = min(max(len - t, 0), VE);
    ns = min(max(L - t, 0), VE);
    whole = t0 + LT * VE <= len;
    base = (size_t)b * H * L + t0;
    plane = (size_t)p.B * L;
    at = (size_t)b * L + t;
  }
  // the lane's steps of channel rs + j NR (past the end, the last one's place)
  __device__ __forceinline__ const T* spot(const T* strip, int j) const {
    const int first = min(j * NR, H - 1);
    const uint32_t off = ((uint32_t)(min(rs + j * NR, H - 1) - first) * (uint32_t)L +
                          (uint32_t)(lt * VE)) * (uint32_t)sizeof(T);
    return reinterpret_cast<const T*>(reinterpret_cast<const char*>(strip + (size_t)first * L) +
                                      off);
  }
  __device__ __forceinline__ T* spot(T* strip, int j) const {
    return const_cast<T*>(spot(const_cast<const T*>(strip), j));
  }
  __device__ __forceinline__ void get(Vec& v, const T* strip, int j) const {
    if (whole)
      v.load(spot(strip, j));
    else
      v.load(spot(strip, j), nv, (T)0.f);
  }
  // nothing where there is no such tensor
  __device__ __forceinline__ void get_any(Vec& v, const T* strip, int j) const {
    if (strip)
      get(v, strip, j);
    else
#pragma unroll
      for (int k = 0; k < Vec::W; ++k) v.w[k] = 0;
  }
};

// The forward pass for more channels than the registers hold: y is read once
// for its sums and, still in a cache, again; o is read back for its own.  Loops
// over the channels, U of them in flight; a few registers per lane, so that
// a compute unit holds more waves, and longer segments of each row (bf16, 2^25
// elements, 1024 channels: 81 us against 87 with the strip in registers; 2048
// channels: 90 against 106).
template <typename T, bool LAYER, int NT, int LT, int VE, int U>
__global__ __launch_bounds__(NT) void resnorm_fwd_wide_kernel(Args p) {
  typedef Packed<T, VE> Vec;
  constexpr int NR = NT / LT;
  __shared__ float buf[(NT / 64) * LT * VE];
  const int strip = strip_of_block(blockIdx.x, p.per);
  if (strip >= p.B * p.ntile) return;
  const WideStrip<T, NT, LT, VE> at(p, strip);
  const int rs = at.rs, H = at.H, nv = at.nv, ns = at.ns;
  const float inv_h = 1.f / (float)H;
  const int nj = (H + NR - 1) / NR;
  const T* x = static_cast<const T*>(p.x) + at.base;
  T* o = static_cast<T*>(p.o) + at.base;
  // A lane's channels one by one: their sum of squares, or for the layer norm
  // their mean and the squares' sum about it, whatever the first ones were
  // (Welford's update); the lanes' are then joined about the column's mean.
  float mean[VE], rstd[VE], s[1][VE], m[1][VE];
  float count = 0.f;
  const auto clear = [&]() {
    count = 0.f;
#pragma unroll
    for (int k = 0; k < VE; ++k) s[0][k] = m[0][k] = 0.f;
  };
  const auto take = [&](bool in, const Vec& v) {
    if (!in) return;
    if (LAYER) {
      count += 1.f;
      const float inv = __builtin_amdgcn_rcpf(count);
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const float d = v[k] - m[0][k];
        m[0][k] = fmaf(d, inv, m[0][k]);
        s[0][k] = fmaf(d, v[k] - m[0][k], s[0][k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k) s[0][k] = fmaf(v[k], v[k], s[0][k]);
    }
  };
  const auto finish = [&]() {
#pragma unroll
    for (int k = 0; k < VE; ++k) mean[k] = 0.f;
    if (LAYER) {
      float t[1][VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) t[0][k] = count * m[0][k];
      strip_sum<NT, LT, VE, 1>(t, buf);
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        mean[k] = t[0][k] * inv_h;
        const float d = m[0][k] - mean[k];
        s[0][k] = fmaf(count * d, d, s[0][k]);
      }
    }
    strip_sum<NT, LT, VE, 1>(s, buf);
#pragma unroll
    for (int k = 0; k < VE; ++k)
      rstd[k] = k < nv ? __builtin_amdgcn_rsqf(fmaf(s[0][k], inv_h, p.eps)) : 0.f;
  };
  clear();
  const T* first = p.y ? static_cast<const T*>(p.y) + at.base : x;
  for (int j0 = 0; j0 < nj; j0 += U) {
    Vec v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at.get(v[u], first, j0 + u);
#pragma unroll
    for (int u = 0; u < U; ++u) take(rs + (j0 + u) * NR < H, v[u]);
  }
  finish();
  const T* stream = first;
  if (p.y) {
    if (p.stats && rs == 0) {
      if (LAYER) store_n<float, VE>(p.stats + at.at, ns, mean);
      store_n<float, VE>(p.stats + (LAYER ? at.plane : 0) + at.at, ns, rstd);
    }
    const T* g = static_cast<const T*>(p.g) + (p.g ? (size_t)(at.b * p.sg) + at.t0 : 0);
    clear();
    for (int j0 = 0; j0 < nj; j0 += U) {
      Vec yv[U], xv[U], gv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        at.get(yv[u], first, j0 + u);
        at.get(xv[u], x, j0 + u);
        if (p.g) at.get(gv[u], g, j0 + u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = rs + (j0 + u) * NR;
        const bool in = h < H;
        const float c = in ? p.w_post[h] * p.scale[h] : 0.f;
        float out[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          float silu = 1.f;
          if (p.g) silu = gv[u][k] * __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * gv[u][k]));
          const float v = (yv[u][k] - mean[k]) * rstd[k];
          out[k] = fmaf(v * c, silu, xv[u][k]);
        }
        live_only<VE>(out, nv, at.whole);
        Vec ov;
        ov.set(out);
        if (in) ov.store(at.spot(o, j0 + u), ns);
        take(in, ov);
      }
    }
    if (!p.n) return;
    finish();
    stream = o;
  }
  if (p.stats && rs == 0) {
    if (LAYER) store_n<float, VE>(p.stats + 2 * at.plane + at.at, ns, mean);
    store_n<float, VE>(p.stats + (LAYER ? 3 : 1) * at.plane + at.at, ns, rstd);
  }
  T* n = static_cast<T*>(p.n) + at.base;
  for (int j0 = 0; j0 < nj; j0 += U) {
    Vec v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at.get(v[u], stream, j0 + u);  // a lane's own stores
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = rs + (j0 + u) * NR;
      if (h >= H) continue;
      const float c = p.w_pre[h];
      float out[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) out[k] = (v[u][k] - mean[k]) * rstd[k] * c;
      live_only<VE>(out, nv, at.whole);
      store_n<T, VE>(at.spot(n, j0 + u), ns, out);
    }
  }
}

// Strips of one workgroup, one after another.  All five inputs of a strip are
// held in registers, so memory is read once; the sums over b, t stay in the
// registers of the channel's lanes until the end, in float32 (a workgroup's
// share: 4 strips for 2^25 elements of 256 channels; from there in float64).
// With oh = o ro - mo ro and so on, the factors that a column shares are formed
// once per strip.
template <typename T, bool LAYER, int NT, int LT, int VE, int KH>
__global__ __launch_bounds__(NT) void resnorm_bwd_kernel(Args p) {
  typedef Packed<T, VE> Vec;
  constexpr int NR = NT / LT, N = LAYER ? 2 : 1;
  __shared__ float buf[(NT / 64) * N * LT * VE];
  const int lt = threadIdx.x % LT, rs = threadIdx.x / LT;
  const int H = p.H;
  const float inv_h = 1.f / (float)H;
  const size_t plane = (size_t)p.B * p.L;
  const Rows<T, NR, KH> rows(rs, lt * VE, H, p.L);
  float a_v[KH], a_n[KH];  // sums of t yh silu(g) and of dn oh
#pragma unroll
  for (int j = 0; j < KH; ++j) a_v[j] = a_n[j] = 0.f;
  const int total = p.B * p.ntile;
  for (int block = blockIdx.x; block < 8 * p.per; block += gridDim.x) {
    const int strip = strip_of_block(block, p.per);
    if (strip >= total) continue;
    const int b = __builtin_amdgcn_readfirstlane(strip / p.ntile);
    const int t0 = (strip - b * p.ntile) * (LT * VE), t = t0 + lt * VE;
    const int len = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
    const int nv = min(max(len - t, 0), VE), ns = min(max(p.L - t, 0), VE);
    const bool whole = t0 + LT * VE <= len;
    const size_t base = (size_t)b * H * p.L + t0;
    const size_t at = (size_t)b * p.L + t;
    Vec ov[KH], nn[KH], dv[KH], yv[KH], gv[KH];
    const auto load = [&](Vec* v, const void* q, size_t off) {
      if (q)
        rows.load(v, static_cast<const T*>(q) + off, nv, whole);
      else
        no_rows<T, VE, KH>(v);
    };
    load(ov, p.d_n ? p.x : nullptr, base);
    load(nn, p.d_n, base);
    // factor and (layer norm) -mean factor of o and of y; past the end 0
    float ro[VE], mo[VE], ry[VE], my[VE];
    load_n<float, VE>(p.stats + (LAYER ? 3 : 1) * plane + at, p.d_n ? nv : 0, ro);
    load_n<float, VE>(p.stats + 2 * plane + at, LAYER && p.d_n ? nv : 0, mo);
    load(dv, p.d_o, base);
    load(yv, p.y, base);
    load(gv, p.g, (size_t)(b * p.sg) + t0);
    load_n<float, VE>(p.stats + (LAYER ? plane : 0) + at, p.y ? nv : 0, ry);
    load_n<float, VE>(p.stats + at, LAYER && p.y ? nv : 0, my);
    float s[N][VE];
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int k = 0; k < VE; ++k) s[m][k] = 0.f;
    if (p.d_n) {
#pragma unroll
      for (int k = 0; k < VE; ++k) mo[k] *= -ro[k];
#pragma unroll
      for (int j = 0; j < KH; ++j) {
        const int h = rs + j * NR;
        const float w = h < H ? p.w_pre[h] : 0.f;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float oh = LAYER ? fmaf(ov[j][k], ro[k], mo[k]) : ov[j][k] * ro[k];
          const float m = nn[j][k] * oh;
          a_n[j] += m;
          s[0][k] = fmaf(w, m, s[0][k]);
          if (LAYER) s[N - 1][k] = fmaf(w, nn[j][k], s[N - 1][k]);
        }
      }
      strip_sum<NT, LT, VE, N>(s, buf);
    }
    // t = do + ro w dn - c1 oh - c0
    float c1[VE], c0[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      c1[k] = -ro[k] * s[0][k] * inv_h;
      c0[k] = -ro[k] * s[N - 1][k] * inv_h;
      if (LAYER) my[k] *= -ry[k];
    }
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      ov[j].refresh();
      nn[j].refresh();
    }
    float R[KH][VE], r[N][VE];
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int k = 0; k < VE; ++k) r[m][k] = 0.f;
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      const int h = rs + j * NR;
      const bool in = h < H;
      const float w = in && p.d_n ? p.w_pre[h] : 0.f;
      float tv[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const float oh = LAYER ? fmaf(ov[j][k], ro[k], mo[k]) : ov[j][k] * ro[k];
        tv[k] = fmaf(nn[j][k], w * ro[k], dv[j][k]);
        tv[k] = fmaf(c1[k], oh, tv[k]);
        if (LAYER) tv[k] += c0[k];
      }
      live_only<VE>(tv, nv, whole);
      if (in) store_n<T, VE>(rows.at(static_cast<T*>(p.dx) + base, j), ns, tv);
      if (!p.y) continue;
      const float c = in ? p.w_post[h] * p.scale[h] : 0.f;
      float dgv[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        float silu = 1.f, dsilu = 0.f;
        if (p.g) {
          const float gk = gv[j][k];
          float rest;
          const float sg = sigmoid_pair(gk, &rest);
          silu = gk * sg;
          dsilu = fmaf(silu, rest, sg);
        }
        const float yh = LAYER ? fmaf(yv[j][k], ry[k], my[k]) : yv[j][k] * ry[k];
        const float ty = tv[k] * yh;
        const float v = ty * silu;
        a_v[j] += v;
        r[0][k] = fmaf(c, v, r[0][k]);
        R[j][k] = tv[k] * silu * c;
        if (LAYER) r[N - 1][k] += R[j][k];
        dgv[k] = ty * dsilu * c;
      }
      live_only<VE>(dgv, nv, whole);
      if (in && p.dg)
        store_n<T, VE>(rows.at(static_cast<T*>(p.dg) + (size_t)(b * p.sdg) + t0, j), ns, dgv);
    }
    if (!p.y) continue;
#pragma unroll
    for (int j = 0; j < KH; ++j) yv[j].refresh();
    strip_sum<NT, LT, VE, N>(r, buf);
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      c1[k] = -ry[k] * r[0][k] * inv_h;
      c0[k] = -ry[k] * r[N - 1][k] * inv_h;
    }
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      const int h = rs + j * NR;
      if (h >= H) continue;
      float out[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const float yh = LAYER ? fmaf(yv[j][k], ry[k], my[k]) : yv[j][k] * ry[k];
        out[k] = fmaf(c1[k], yh, R[j][k] * ry[k]);
        if (LAYER) out[k] += c0[k];
      }
      live_only<VE>(out, nv, whole);
      store_n<T, VE>(rows.at(static_cast<T*>(p.dy) + base, j), ns, out);
    }
  }
  float* part = p.part + (size_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int j = 0; j < KH; ++j) {
    const int h = rs + j * NR;
    const float v = lanes_sum<LT>(a_v[j]), n = lanes_sum<LT>(a_n[j]);
    if (lt == 0 && h < H) {
      part[h] = v;
      part[H + h] = n;
    }
  }
}

// The backward pass for more channels than the registers hold.  The second
// norm's sums need t, which needs the first norm's; but t is a combination of
// do, dn, oh and 1 whose weights a column shares, so one reading of the inputs
// gives sums from which both norms' follow (with k = scale silu(g) w_post):
//   sum R yh = sum do k yh + ro (sum P k yh - mean(P oh) sum oh k yh - mean(P) sum k yh)
//   sum R    = sum do k    + ro (sum P k    - mean(P oh) sum oh k    - mean(P) sum k)
// and a second reading, still in a cache, writes the gradients.
template <typename T, bool LAYER, int NT, int LT, int VE, int U>
__global__ __launch_bounds__(NT) void resnorm_bwd_wide_kernel(Args p) {
  typedef Packed<T, VE> Vec;
  constexpr int NR = NT / LT, N = LAYER ? 10 : 4;
  __shared__ float buf[(NT / 64) * N * LT * VE];
  extern __shared__ float sums[];  // [2][H]: t yh silu(g), dn oh; a channel is always the same lanes'
  const int H = p.H;
  const float inv_h = 1.f / (float)H;
  const int nj = (H + NR - 1) / NR;
  for (int h = threadIdx.x / LT; h < H; h += NR)
    if (threadIdx.x % LT == 0) sums[h] = sums[H + h] = 0.f;
  const int total = p.B * p.ntile;
  for (int block = blockIdx.x; block < 8 * p.per; block += gridDim.x) {
    const int strip = strip_of_block(block, p.per);
    if (strip >= total) continue;
    const WideStrip<T, NT, LT, VE> at(p, strip);
    const int ns = at.ns;
    const auto input = [&](const void* q, size_t off) {
      return q ? static_cast<const T*>(q) + off : nullptr;
    };
    const T* o = input(p.d_n ? p.x : nullptr, at.base);
    const T* dn = input(p.d_n, at.base);
    const T* dout = input(p.d_o, at.base);
    const T* y = input(p.y, at.base);
    const T* g = input(p.g, (size_t)(at.b * p.sg) + at.t0);
    // factor and (layer norm) -mean factor of o and of y; past the end 0
    float ro[VE], mo[VE], ry[VE], my[VE];
    load_n<float, VE>(p.stats + (LAYER ? 3 : 1) * at.plane + at.at, dn ? at.nv : 0, ro);
    load_n<float, VE>(p.stats + 2 * at.plane + at.at, LAYER && dn ? at.nv : 0, mo);
    load_n<float, VE>(p.stats + (LAYER ? at.plane : 0) + at.at, y ? at.nv : 0, ry);
    load_n<float, VE>(p.stats + at.at, LAYER && y ? at.nv : 0, my);
    float s[N][VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      mo[k] *= -ro[k];
      my[k] *= -ry[k];
    }
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int k = 0; k < VE; ++k) s[m][k] = 0.f;
    for (int j0 = 0; j0 < nj; j0 += U) {
      Vec ov[U], nn[U], dv[U], yv[U], gv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        at.get_any(ov[u], o, j0 + u);
        at.get_any(nn[u], dn, j0 + u);
        at.get_any(dv[u], dout, j0 + u);
        at.get_any(yv[u], y, j0 + u);
        at.get_any(gv[u], g, j0 + u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = at.rs + (j0 + u) * NR;
        const bool in = h < H;
        const float w = in && dn ? p.w_pre[h] : 0.f;
        const float c = in && y ? p.w_post[h] * p.scale[h] : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float oh = LAYER ? fmaf(ov[u][k], ro[k], mo[k]) : ov[u][k] * ro[k];
          const float m = nn[u][k] * oh;
          sum += m;
          s[0][k] = fmaf(w, m, s[0][k]);
          const float P = nn[u][k] * w;
          float q = c;
          if (g) q *= gv[u][k] * __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * gv[u][k]));
          const float yh = LAYER ? fmaf(yv[u][k], ry[k], my[k]) : yv[u][k] * ry[k];
          const float e = q * yh;
          s[1][k] = fmaf(dv[u][k], e, s[1][k]);
          s[2][k] = fmaf(P, e, s[2][k]);
          s[3][k] = fmaf(oh, e, s[3][k]);
          if (LAYER) {
            s[N - 6][k] += P;
            s[N - 5][k] += e;
            s[N - 4][k] = fmaf(dv[u][k], q, s[N - 4][k]);
            s[N - 3][k] = fmaf(P, q, s[N - 3][k]);
            s[N - 2][k] = fmaf(oh, q, s[N - 2][k]);
            s[N - 1][k] += q;
          }
        }
        sum = lanes_sum<LT>(sum);
        if (at.lt == 0 && in) sums[H + h] += sum;
      }
    }
    strip_sum<NT, LT, VE, N>(s, buf);
    float c1[VE], c0[VE], d1[VE], d0[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      const float a = s[0][k] * inv_h, b = LAYER ? s[N - 6][k] * inv_h : 0.f;
      c1[k] = -ro[k] * a;
      c0[k] = -ro[k] * b;
      float r1 = fmaf(-a, s[3][k], s[2][k]), r0 = 0.f;
      if (LAYER) {
        r1 = fmaf(-b, s[N - 5][k], r1);
        r0 = fmaf(-a, s[N - 2][k], s[N - 3][k]);
        r0 = fmaf(-b, s[N - 1][k], r0);
        r0 = fmaf(ro[k], r0, s[N - 4][k]);
      }
      r1 = fmaf(ro[k], r1, s[1][k]);
      d1[k] = -ry[k] * r1 * inv_h;
      d0[k] = -ry[k] * r0 * inv_h;
    }
    T* dx = static_cast<T*>(p.dx) + at.base;
    T* dy = static_cast<T*>(p.dy) + at.base;
    T* dg = static_cast<T*>(p.dg) + (size_t)(at.b * p.sdg) + at.t0;
    for (int j0 = 0; j0 < nj; j0 += U) {
      Vec ov[U], nn[U], dv[U], yv[U], gv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        at.get_any(ov[u], o, j0 + u);
        at.get_any(nn[u], dn, j0 + u);
        at.get_any(dv[u], dout, j0 + u);
        at.get_any(yv[u], y, j0 + u);
        at.get_any(gv[u], g, j0 + u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = at.rs + (j0 + u) * NR;
        const bool in = h < H;
        const float w = in && dn ? p.w_pre[h] : 0.f;
        const float c = in && y ? p.w_post[h] * p.scale[h] : 0.f;
        float tv[VE], dgv[VE], dyv[VE], sum = 0.f;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float oh = LAYER ? fmaf(ov[u][k], ro[k], mo[k]) : ov[u][k] * ro[k];
          float tk = fmaf(nn[u][k], w * ro[k], dv[u][k]);
          tk = fmaf(c1[k], oh, tk);
          if (LAYER) tk += c0[k];
          if (!at.whole) tk = k < at.nv ? tk : 0.f;  // the parameters' sums take it too
          float silu = 1.f, dsilu = 0.f;
          if (g) {
            const float gk = gv[u][k];
            float rest;
            const float sg = sigmoid_pair(gk, &rest);
            silu = gk * sg;
            dsilu = fmaf(silu, rest, sg);
          }
          const float yh = LAYER ? fmaf(yv[u][k], ry[k], my[k]) : yv[u][k] * ry[k];
          const float ty = tk * yh;
          sum = fmaf(ty, silu, sum);
          dgv[k] = ty * dsilu * c;
          dyv[k] = fmaf(d1[k], yh, tk * silu * c * ry[k]);
          if (LAYER) dyv[k] += d0[k];
          tv[k] = tk;
        }
        live_only<VE>(dyv, at.nv, at.whole);
        live_only<VE>(dgv, at.nv, at.whole);
        if (in) {
          store_n<T, VE>(at.spot(dx, j0 + u), ns, tv);
          if (y) store_n<T, VE>(at.spot(dy, j0 + u), ns, dyv);
          if (g) store_n<T, VE>(at.spot(dg, j0 + u), ns, dgv);
        }
        sum = lanes_sum<LT>(sum);
        if (at.lt == 0 && in) sums[h] += sum;
      }
    }
  }
  float* part = p.part + (size_t)blockIdx.x * 2 * H;
  for (int h = threadIdx.x / LT; h < H; h += NR)
    if (threadIdx.x % LT == 0) {
      part[h] = sums[h];
      part[H + h] = sums[H + h];
    }
}

// The workgroups' sums, in order and in float64: 16 channels by 64 slices of
// the workgroups to a block.  With V = sum t yh silu(g): dw_post = scale V,
// dscale = w_post V.
__global__ __launch_bounds__(1024) void resnorm_sum_kernel(const float* __restrict__ part, int G,
                                                           int H, const float* w_post,
                                                           const float* scale, float* dw_post,
                                                           float* dscale, float* dw_pre) {
  __shared__ double s[64][17];
  const int c = threadIdx.x & 15, z = threadIdx.x >> 4;
  const int k = blockIdx.x * 16 + c;
  double v = 0.0;
  if (k < 2 * H) {
#pragma unroll 4
    for (int w = z; w < G; w += 64) v += (double)part[(size_t)w * 2 * H + k];
  }
  s[z][c] = v;
  __syncthreads();
  if (threadIdx.x < 256) {  // 16 slices' sums at a time, then these
    v = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) v += s[z * 4 + j][c];
  }
  __syncthreads();
  if (threadIdx.x < 256) s[z][c] = v;
  __syncthreads();
  if (z == 0 && k < 2 * H) {
    v = 0.0;
#pragma unroll
    for (int j = 0; j < 16; ++j) v += s[j][c];
    if (k >= H) {
      if (dw_pre) dw_pre[k - H] = (float)v;
    } else {
      // nothing to add up is 0, whatever the parameter
      if (dw_post) dw_post[k] = (float)(v != 0.0 ? v * (double)scale[k] : 0.0);
      if (dscale) dscale[k] = (float)(v != 0.0 ? v * (double)w_post[k] : 0.0);
    }
  }
}

constexpr int kMaxGroups = 512;  // workgroups of the backward pass

// How a call is laid out: lanes to a row segment and steps to a lane, held in
// registers (threads, channels to a lane) or looped over.
//
// Held, the strip's channels set the segments' length, which memory wants long
// (backward, bf16, 2^25 elements: 136-145 us with 256 or 128 bytes for up to
// 256 channels, 170 with 64, 200 with 32); looped, it is free, at the price of
// reading inputs again from a cache.  Forward: held up to 512 channels (83 us
// against 88 at 512; 87 against 81 at 1024).  Backward: held up to 1024 (200
// against 209 there; 255 against 213 at 2048, 600 against 266 at 4096).
// Up to 128 channels and where channels are looped over, strips are as wide as
// the registers allow and as leaves one for every compute unit (32 channels,
// forward / backward: 79 / 178 us with 256 and 512 bytes, 115 / 275 with 128
// and 256).  A single step has a kernel of its own forward; backward its
// channels lie side by side.
struct Form {
  int nt, lt, ve, kh;  // kh 0: looped
};

int strips(const Form& f, int L) { return (L + f.lt * f.ve - 1) / (f.lt * f.ve); }

// f, or narrower until there is a strip for every compute unit.
Form spread(Form f, int B, int L, int least) {
  while (f.lt > least && (long)B * strips(f, L) < 256) f.lt /= 2;
  return f;
}

Form fwd_form(int B, int H, int L, int dtype) {
  if (L == 1) return {H <= 512 ? 64 : H <= 1024 ? 128 : H <= 4096 ? 512 : 1024, 1, 1, 8};
  const int ve = dtype == 0 ? 4 : 8;
  if (H > 512) return spread({1024, 16, ve, 0}, B, L, 2);
  if (H > 128) return {H <= 256 ? 512 : 1024, 8, ve, 4};
  return spread({256, H <= 16 ? 64 : H <= 32 ? 32 : H <= 64 ? 16 : 8, ve, 4}, B, L, 8);
}

Form bwd_form(int B, int H, int L, int dtype) {
  if (L == 1) return H <= 1024 ? Form{256, 1, 1, 4} : Form{1024, 1, 1, 8};
  const int ve = dtype == 0 ? 4 : 8;
  if (H > 1024) return spread({1024, 16, 4, 0}, B, L, 4);
  if (H > 128) return {512, H <= 256 ? 8 : H <= 512 ? 4 : 2, ve, 4};
  return spread({512, H <= 32 ? 64 : H <= 64 ? 32 : 16, ve, 4}, B, L, 16);
}

int groups_of(int B, int H, int L, int dtype) {
  const long n = (long)B * strips(bwd_form(B, H, L, dtype), L);
  return (int)std::min<long>((n + 7) / 8 * 8, kMaxGroups);
}

template <typename T, bool LAYER, int NT, int LT, int VE, int KH>
void fwd_held(const Args& a, hipStream_t st) {
  hipLaunchKernelGGL((resnorm_fwd_kernel<T, LAYER, NT, LT, VE, KH>), dim3(8u * a.per), dim3(NT), 0,
                     st, a);
}

template <typename T, bool LAYER, int NT>
void fwd_token(const Args& a, hipStream_t st) {
  constexpr int R = token_rows(NT);
  hipLaunchKernelGGL((resnorm_token_kernel<T, LAYER, NT>), dim3((unsigned)(a.B + R - 1) / R),
                     dim3(NT, R), 0, st, a);
}

template <typename T, bool LAYER, int LT>
void fwd_wide(const Args& a, hipStream_t st) {
  hipLaunchKernelGGL((resnorm_fwd_wide_kernel<T, LAYER, 1024, LT, 16 / (int)sizeof(T), 4>),
                     dim3(8u * a.per), dim3(1024), 0, st, a);
}

template <typename T, bool LAYER>
void fwd_run(const Args& a, const Form& f, hipStream_t st) {
  constexpr int VE = 16 / sizeof(T);
  if (a.L == 1)
    f.nt == 64    ? fwd_token<T, LAYER, 64>(a, st)
    : f.nt == 128 ? fwd_token<T, LAYER, 128>(a, st)
    : f.nt == 512 ? fwd_token<T, LAYER, 512>(a, st)
                  : fwd_token<T, LAYER, 1024>(a, st);
  else if (f.kh)
    f.lt == 64    ? fwd_held<T, LAYER, 256, 64, VE, 4>(a, st)
    : f.lt == 32  ? fwd_held<T, LAYER, 256, 32, VE, 4>(a, st)
    : f.lt == 16  ? fwd_held<T, LAYER, 256, 16, VE, 4>(a, st)
    : f.nt == 256 ? fwd_held<T, LAYER, 256, 8, VE, 4>(a, st)
    : f.nt == 512 ? fwd_held<T, LAYER, 512, 8, VE, 4>(a, st)
                  : fwd_held<T, LAYER, 1024, 8, VE, 4>(a, st);
  else
    f.lt == 16  ? fwd_wide<T, LAYER, 16>(a, st)
    : f.lt == 8 ? fwd_wide<T, LAYER, 8>(a, st)
    : f.lt == 4 ? fwd_wide<T, LAYER, 4>(a, st)
                : fwd_wide<T, LAYER, 2>(a, st);
}

template <typename T, bool LAYER, int NT, int LT, int VE, int KH>
void bwd_held(const Args& a, int groups, hipStream_t st) {
  hipLaunchKernelGGL((resnorm_bwd_kernel<T, LAYER, NT, LT, VE, KH>), dim3((unsigned)groups),
                     dim3(NT), 0, st, a);
}

template <typename T, bool LAYER, int LT>
void bwd_wide(const Args& a, int groups, hipStream_t st) {
  hipLaunchKernelGGL((resnorm_bwd_wide_kernel<T, LAYER, 1024, LT, 4, 2>), dim3((unsigned)groups),
                     dim3(1024), 2 * a.H * sizeof(float), st, a);
}

template <typename T, bool LAYER>
void bwd_run(const Args& a, const Form& f, int groups, hipStream_t st) {
  constexpr int VE = 16 / sizeof(T);
  if (a.L == 1)
    f.nt == 256 ? bwd_held<T, LAYER, 256, 1, 1, 4>(a, groups, st)
                : bwd_held<T, LAYER, 1024, 1, 1, 8>(a, groups, st);
  else if (f.kh)
    f.lt == 64   ? bwd_held<T, LAYER, 512, 64, VE, 4>(a, groups, st)
    : f.lt == 32 ? bwd_held<T, LAYER, 512, 32, VE, 4>(a, groups, st)
    : f.lt == 16 ? bwd_held<T, LAYER, 512, 16, VE, 4>(a, groups, st)
    : f.lt == 8 ? bwd_held<T, LAYER, 512, 8, VE, 4>(a, groups, st)
    : f.lt == 4 ? bwd_held<T, LAYER, 512, 4, VE, 4>(a, groups, st)
                : bwd_held<T, LAYER, 512, 2, VE, 4>(a, groups, st);
  else
    f.lt == 16  ? bwd_wide<T, LAYER, 16>(a, groups, st)
    : f.lt == 8 ? bwd_wide<T, LAYER, 8>(a, groups, st)
                : bwd_wide<T, LAYER, 4>(a, groups, st);
}

template <typename T, bool LAYER>
hipError_t run(const ResnormCall& c, int dtype, bool backward, hipStream_t st) {
  const Form f = backward ? bwd_form(c.B, c.H, c.L, dtype) : fwd_form(c.B, c.H, c.L, dtype);
  Args a{};
  a.x = c.x;
  a.y = c.y;
  a.g = c.g;
  a.sg = c.stride_g;
  a.w_post = c.w_post;
  a.scale = c.scale;
  a.w_pre = c.w_pre;
  a.lens = c.lens;
  a.B = c.B;
  a.H = c.H;
  a.L = c.L;
  a.ntile = strips(f, c.L);
  a.per = (c.B * a.ntile + 7) / 8;
  a.eps = c.eps;
  a.o = c.o;
  a.n = c.n;
  a.stats = c.stats;
  a.d_o = c.d_o;
  a.d_n = c.d_n;
  a.dx = c.dx;
  a.dy = c.dy;
  a.dg = c.dg;
  a.sdg = c.stride_dg;
  a.part = static_cast<float*>(c.ws);
  if (!backward) {
    fwd_run<T, LAYER>(a, f, st);
    return hipGetLastError();
  }
  const int groups = groups_of(c.B, c.H, c.L, dtype);
  bwd_run<T, LAYER>(a, f, groups, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(resnorm_sum_kernel, dim3((unsigned)((2 * c.H + 15) / 16)), dim3(1024), 0, st,
                     a.part, groups, c.H, c.w_post, c.scale, c.dw_post, c.dscale, c.dw_pre);
  return hipGetLastError();
}

template <typename T>
hipError_t run_norm(const ResnormCall& c, int dtype, bool backward, hipStream_t st) {
  return c.layer ? run<T, true>(c, dtype, backward, st) : run<T, false>(c, dtype, backward, st);
}

hipError_t run_type(const ResnormCall& c, int dtype, bool backward, hipStream_t st) {
  switch (dtype) {
    case 0: return run_norm<float>(c, dtype, backward, st);
    case 1: return run_norm<__bf16>(c, dtype, backward, st);
    default: return run_norm<_Float16>(c, dtype, backward, st);
  }
}

}  // namespace

size_t resnorm_workspace(int B, int H, int L, int dtype) {
  return align_up((size_t)groups_of(B, H, L, dtype) * 2 * H * sizeof(float), 256);
}

hipError_t launch_resnorm_forward(const ResnormCall& c, int dtype, hipStream_t st) {
  return run_type(c, dtype, false, st);
}

// B = 0 or L = 0: no strips, so the sums are zero.
hipError_t launch_resnorm_backward(const ResnormCall& c, int dtype, hipStream_t st) {
  if (c.B == 0 || c.L == 0) {
    hipLaunchKernelGGL(resnorm_sum_kernel, dim3((unsigned)((2 * c.H + 15) / 16)), dim3(1024), 0, st,
                       static_cast<const float*>(nullptr), 0, c.H, c.w_post, c.scale, c.dw_post,
                       c.dscale, c.dw_pre);
    return hipGetLastError();
  }
  return run_type(c, dtype, true, st);
}

}  // namespace dssm
