// The gated linear recurrence: per channel h a real mode of the DLR bank whose
// decay and drive are set by two gates at every step,
//
//   q = sigmoid(r_t), s = sigmoid(i_t), z = log_re^2 q,
//   a_t = exp(-z),  b_t = sqrt(1 - a_t^2) s u_t,  h_t = a_t h_{t-1} + b_t,  y_t = h_t
//
// and its gradients.  With G_t = dy_t + a_{t+1} G_{t+1} (the state's gradient
// entering from the right):
//
//   du = G beta s,  di = G beta u s (1 - s),  beta = sqrt(1 - a^2),
//   dz = G s u a^2 / beta - a G h_{t-1},  dr = dz log_re^2 q (1 - q),
//   dlog_re = 2 log_re sum_{b,t} dz q,  dx0 = a_0 G_0.
//
// Layout.  A lane holds 8 consecutive steps, a wave a tile of 512; a wave's
// lanes are joined by a scan of pairs (S, V): S the sum of z log2(e) over the
// steps (so the decay over them is exp2(-S), one rounding however many steps),
// V the state they leave from zero.  Keeping the exponents' sum instead of the
// decays' product matters for slow channels: 10^4 remembered steps would add
// up 10^4 roundings next to 1.
#include <algorithm>

#include "dssm_internal.h"
#include "seq_common.h"

namespace dssm {
namespace {

constexpr float kTiny = 1.17549435e-38f;  // below it 1 - a^2 counts as 0 (no drive, no gradient)

struct Gate {
  float a, q, s, w;  // decay, sigmoid(r), sigmoid(i), 1 - a^2
  float nq, ns;      // 1 - q, 1 - s
};

// kappa = log_re^2 log2(e).  1 - a^2 loses its digits where a is close to 1:
// there it is the series of 1 - exp(-x), x = 2 z, up to the term that 24 bits see.
__device__ __forceinline__ Gate gate(float r, float i, float kappa, float* e) {
  Gate g;
  g.q = sigmoid_pair(r, &g.nq);
  g.s = sigmoid_pair(i, &g.ns);
  *e = kappa * g.q;
  g.a = exp2_fast(-*e);
  const float x = *e * (2.f / kLog2e);
  const float far = fmaf(-g.a, g.a, 1.f);
  // x (1 - x/2 (1 - x/3 (1 - x/4 (1 - x/5 (1 - x/6 (1 - x/7))))))
  float p = fmaf(x, -1.f / 7.f, 1.f);
  p = fmaf(x * p, -1.f / 6.f, 1.f);
  p = fmaf(x * p, -1.f / 5.f, 1.f);
  p = fmaf(x * p, -1.f / 4.f, 1.f);
  p = fmaf(x * p, -1.f / 3.f, 1.f);
  p = fmaf(x * p, -1.f / 2.f, 1.f);
  g.w = x < 0.5f ? x * p : far;
  if (!(g.w >= kTiny)) g.w = g.w != g.w ? g.w : 0.f;
  return g;
}

// Inclusive scan over groups of n lanes (n a power of two), in time order or
// (REV) against it: (S1, V1) then (S2, V2) = (S1 + S2, exp2(-S2) V1 + V2).
template <bool REV>
__device__ __forceinline__ void pair_scan(float& S, float& V, int gl, int n) {
  for (int o = 1; o < n; o <<= 1) {
    const float Sp = REV ? __shfl_down(S, o) : __shfl_up(S, o);
    const float Vp = REV ? __shfl_down(V, o) : __shfl_up(V, o);
    if (REV ? gl + o < n : gl >= o) {
      V = fmaf(exp2_fast(-S), Vp, V);
      S += Sp;
    }
  }
}

// The neighbour's inclusive pair (nothing before the first lane).
template <bool REV>
__device__ __forceinline__ void pair_shift(float& S, float& V, int gl, int n) {
  const float Sp = REV ? __shfl_down(S, 1) : __shfl_up(S, 1);
  const float Vp = REV ? __shfl_down(V, 1) : __shfl_up(V, 1);
  const bool first = REV ? gl == n - 1 : gl == 0;
  S = first ? 0.f : Sp;
  V = first ? 0.f : Vp;
}

// What enters segment `seg` of a split row: the pairs of the segments before
// it (REV: after it) applied to `start`.  Every lane of the wave gets it.
template <bool REV>
__device__ float join_segments(const float2* agg, int nseg, int seg, float start) {
  const int lane = threadIdx.x & 63;
  const int count = REV ? nseg - 1 - seg : seg;
  float c = start;
  for (int base = 0; base < count; base += 64) {
    // lane order = order of application
    const int j = base + lane;
    float2 t = make_float2(0.f, 0.f);
    if (j < count) t = agg[REV ? nseg - 1 - j : j];
    float S = t.x, V = t.y;
    pair_scan<false>(S, V, lane, 64);
    c = fmaf(exp2_fast(-__shfl(S, 63)), c, __shfl(V, 63));
  }
  return c;
}

struct Args {
  const void *u, *r, *i;
  long long sb;  // elements between batch rows of u, r, i
  const float* log_re;
  const int* lens;
  long rows;
  int H, L;
  const float* x0;  // forward: state before step 0; may be null (zero)
  float* xT;        // forward: state after the last step; may be null
  void* y;
  float* bounds;    // [rows][nch] state entering each chunk
  int8_t* q8[3];    // u, r, i in 8 bits, and their exponents
  uint8_t* e8[3];
  // backward
  const void* dy;
  const float* dx;  // gradient of the state after the last step; may be null
  void *du, *dr, *di;
  long long sdb;
  float* dx0;       // may be null
  double* part;     // [rows][nseg] sum of dz q
  // a row's tiles in nseg segments of seg_tiles (a tile: WPR chunks)
  int nseg, seg_tiles;
  float2* agg;      // [rows][nseg] pairs of the segments
  int lpr;          // lanes per row (64 unless rows are short)
};

__device__ __forceinline__ int row_len(const Args& p, long row) {
  if (!p.lens) return p.L;
  return min(max(p.lens[row / p.H], 0), p.L);
}

__device__ __forceinline__ int clamp8(int n) { return min(max(n, 0), 8); }

// u, r, i of a lane's 8 steps from step t (nv of them live), from the inputs
// or (Q8) their 8-bit form; dead steps are 0.
template <typename T, bool Q8>
__device__ __forceinline__ void load_one(const Args& p, const void* x, int which, long row, int t,
                                         int nv, float* out) {
  if (Q8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = 0.f;
    if (nv > 0) {
      const uint2 q = *reinterpret_cast<const uint2*>(p.q8[which] + (size_t)row * ckpt8_row(p.L) + t);
      const int byte = p.e8[which][(size_t)row * ckpt8_groups(p.L) + t / kGroup];
      dequantise8(q, byte, out);
#pragma unroll
      for (int k = 0; k < 8; ++k) out[k] = k < nv ? out[k] : 0.f;
    }
  } else {
    const long b = row / p.H;
    const T* base = static_cast<const T*>(x) + b * p.sb + (row - b * p.H) * p.L;
    load_n<T, 8>(base + t, nv, out);
  }
}

// Which row, segment and lanes a thread works on.  WPR waves share a row; with
// WPR == 1 a workgroup of 4 waves holds 4 rows, or 4 (64 / lpr) short ones.
template <int WPR>
struct Place {
  long row;
  int seg, gl, n, wave, lane;
  bool live;
  __device__ Place(const Args& p) {
    lane = threadIdx.x & 63;
    wave = threadIdx.x >> 6;
    seg = 0;
    n = 64;
    if (WPR == 1) {
      n = p.lpr;
      gl = lane & (n - 1);
      row = ((long)blockIdx.x * 4 + wave) * (64 / n) + lane / n;
    } else {
      gl = lane;
      row = blockIdx.x / p.nseg;
      seg = blockIdx.x % p.nseg;
    }
    live = row < p.rows;
    if (!live) row = p.rows - 1;
  }
};

template <int WPR>
constexpr int threads_of() { return WPR == 1 ? 256 : 64 * WPR; }

// The carries of a tile's WPR waves: every wave leaves its pair, then takes
// what enters it and what leaves the tile.  One barrier: the buffers alternate.
template <int WPR, bool REV>
__device__ __forceinline__ float tile_carry(float2 (*tot)[WPR], int flip, int wave, int lane,
                                            float S, float V, float& carry) {
  if (WPR == 1) {
    const float in = carry;
    carry = fmaf(exp2_fast(-S), carry, V);
    return in;
  }
  if (lane == 0) tot[flip][wave] = make_float2(S, V);
  __syncthreads();
  float in = carry, c = carry;
#pragma unroll
  for (int k = 0; k < WPR; ++k) {
    const int w = REV ? WPR - 1 - k : k;
    if (w == wave) in = c;
    const float2 t = tot[flip][w];
    c = fmaf(exp2_fast(-t.x), c, t.y);
  }
  carry = c;
  return in;
}

// Forward over a row (or one segment of it).  AGG: only the segment's pair.
// CK: 0 nothing kept, 1 the state entering every chunk, 2 also u, r, i in 8 bits.
template <typename T, int WPR, int CK, bool AGG>
__global__ __launch_bounds__(threads_of<WPR>()) void gated_fwd_kernel(Args p) {
  __shared__ float2 tot[2][WPR];
  const Place<WPR> at(p);
  const int len = row_len(p, at.row);
  const float lr = p.log_re[at.row % p.H];
  const float kappa = lr * lr * kLog2e;
  const int tile = kChunk * WPR;
  const int ntile = (p.L + tile - 1) / tile;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  float carry = (p.x0 && !AGG) ? p.x0[at.row] : 0.f;
  if (WPR > 1 && !AGG && p.nseg > 1)
    carry = join_segments<false>(p.agg + at.row * p.nseg, p.nseg, at.seg, carry);
  float Sseg = 0.f;
  for (int k = t_lo; k < t_hi; ++k) {
    const int t = k * tile + (WPR > 1 ? at.wave * kChunk : 0) + at.gl * 8;
    const int nv = at.live ? clamp8(len - t) : 0;
    const int ns = at.live ? clamp8(p.L - t) : 0;
    float u[8], r[8], i[8], a[8], b[8];
    load_one<T, false>(p, p.u, 0, at.row, t, nv, u);
    load_one<T, false>(p, p.r, 1, at.row, t, nv, r);
    load_one<T, false>(p, p.i, 2, at.row, t, nv, i);
    float S = 0.f, V = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float e;
      const Gate g = gate(r[j], i[j], kappa, &e);
      const bool in = j < nv;
      a[j] = in ? g.a : 1.f;
      b[j] = in ? __builtin_amdgcn_sqrtf(g.w) * (g.s * u[j]) : 0.f;
      S += in ? e : 0.f;
      V = fmaf(a[j], V, b[j]);
    }
    pair_scan<false>(S, V, at.gl, at.n);
    const float St = __shfl(S, 63), Vt = __shfl(V, 63);  // used where a wave is one row's
    pair_shift<false>(S, V, at.gl, at.n);
    Sseg += St;
    const float in = tile_carry<WPR, false>(tot, (k - t_lo) & 1, at.wave, at.lane, St, Vt, carry);
    if (AGG) {
      // the segment's exponent sum: every wave's part
      if (WPR > 1) {
#pragma unroll
        for (int w = 0; w < WPR; ++w)
          if (w != at.wave) Sseg += tot[(k - t_lo) & 1][w].x;
      }
      continue;
    }
    if (CK >= 1 && at.live && at.gl == 0 && t < p.L)
      p.bounds[(size_t)at.row * ((p.L + kChunk - 1) / kChunk) + t / kChunk] = in;
    if (CK == 2) {
      const float* x[3] = {u, r, i};
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        uint2 q;
        const int byte = quantise8<T>(x[m], min(8, at.n), &q);
        if (ns > 0) {
          *reinterpret_cast<uint2*>(p.q8[m] + (size_t)at.row * ckpt8_row(p.L) + t) = q;
          if ((t & (kGroup - 1)) == 0)
            p.e8[m][(size_t)at.row * ckpt8_groups(p.L) + t / kGroup] = (uint8_t)byte;
        }
      }
    }
    float h = fmaf(exp2_fast(-S), in, V);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h = fmaf(a[j], h, b[j]);
      y[j] = j < nv ? h : 0.f;
    }
    store_n<T, 8>(static_cast<T*>(p.y) + (size_t)at.row * p.L + t, ns, y);
    if (WPR == 1 && at.n < 64) {  // short rows: the last lane's state is the row's
      carry = __shfl(h, at.lane | (at.n - 1));
    }
  }
  if (!at.live) return;
  if (AGG) {
    if (threadIdx.x == 0) p.agg[at.row * p.nseg + at.seg] = make_float2(Sseg, carry);
  } else if (p.xT && at.gl == 0 && (WPR == 1 || (threadIdx.x == 0 && at.seg == p.nseg - 1))) {
    p.xT[at.row] = carry;
  }
}

// The pair of a segment against time: S as before, V the gradient that leaves
// it to the left from zero.  Reads r and dy only.
template <typename T, int WPR, bool Q8>
__global__ __launch_bounds__(threads_of<WPR>()) void gated_bwd_agg_kernel(Args p) {
  __shared__ float2 tot[2][WPR];
  const Place<WPR> at(p);
  const int len = row_len(p, at.row);
  const float lr = p.log_re[at.row % p.H];
  const float kappa = lr * lr * kLog2e;
  const int tile = kChunk * WPR;
  const int ntile = (p.L + tile - 1) / tile;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  float carry = 0.f, Sseg = 0.f;
  for (int k = t_hi - 1; k >= t_lo; --k) {
    const int t = k * tile + at.wave * kChunk + at.gl * 8;
    const int nv = clamp8(len - t);
    float r[8], dy[8];
    load_one<T, Q8>(p, p.r, 1, at.row, t, nv, r);
    load_n<T, 8>(static_cast<const T*>(p.dy) + (size_t)at.row * p.L + t, nv, dy);
    float S = 0.f, V = 0.f;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      float nq;
      const float e = j < nv ? kappa * sigmoid_pair(r[j], &nq) : 0.f;
      V = exp2_fast(-e) * (dy[j] + V);
      S += e;
    }
    pair_scan<true>(S, V, at.gl, 64);
    const int flip = (t_hi - 1 - k) & 1;
    const float St = __shfl(S, 0), Vt = __shfl(V, 0);
    tile_carry<WPR, true>(tot, flip, at.wave, at.lane, St, Vt, carry);
#pragma unroll
    for (int w = 0; w < WPR; ++w) Sseg += tot[flip][w].x;
  }
  if (threadIdx.x == 0) p.agg[at.row * p.nseg + at.seg] = make_float2(Sseg, carry);
}

// Backward over a row (or one segment of it), tiles from the last to the
// first.  Each wave's tile is one chunk, whose entering state the checkpoint
// holds: the states need no walk of their own.
template <typename T, int WPR, bool Q8>
__global__ __launch_bounds__(threads_of<WPR>()) void gated_bwd_kernel(Args p) {
  __shared__ float2 tot[2][WPR];
  __shared__ double red[threads_of<WPR>() / 64];
  const Place<WPR> at(p);
  const int len = row_len(p, at.row);
  const float lr = p.log_re[at.row % p.H];
  const float lr2 = lr * lr;
  const float kappa = lr2 * kLog2e;
  const long b = at.row / p.H;
  const size_t gbase = (size_t)(b * p.sdb + (at.row - b * p.H) * p.L);
  const int tile = kChunk * WPR;
  const int ntile = (p.L + tile - 1) / tile;
  const int nch = (p.L + kChunk - 1) / kChunk;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  float carry = p.dx ? p.dx[at.row] : 0.f;
  if (WPR > 1 && p.nseg > 1)
    carry = join_segments<true>(p.agg + at.row * p.nseg, p.nseg, at.seg, carry);
  double acc = 0.0;
  for (int k = t_hi - 1; k >= t_lo; --k) {
    const int t = k * tile + (WPR > 1 ? at.wave * kChunk : 0) + at.gl * 8;
    const int nv = at.live ? clamp8(len - t) : 0;
    const int ns = at.live ? clamp8(p.L - t) : 0;
    float u[8], r[8], i[8], dy[8], a[8], e[8], hp[8];
    load_one<T, Q8>(p, p.u, 0, at.row, t, nv, u);
    load_one<T, Q8>(p, p.r, 1, at.row, t, nv, r);
    load_one<T, Q8>(p, p.i, 2, at.row, t, nv, i);
    load_n<T, 8>(static_cast<const T*>(p.dy) + (size_t)at.row * p.L + t, nv, dy);
    const int ch = min(t / kChunk, nch - 1);
    const float bound = p.bounds[(size_t)at.row * nch + ch];
    // the states before each step, from the chunk's entering state
    float S = 0.f, V = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Gate g = gate(r[j], i[j], kappa, &e[j]);
      if (j >= nv) e[j] = 0.f;
      a[j] = j < nv ? g.a : 1.f;
      hp[j] = j < nv ? __builtin_amdgcn_sqrtf(g.w) * (g.s * u[j]) : 0.f;  // b_j for now
      S += e[j];
      V = fmaf(a[j], V, hp[j]);
    }
    const float Sl = S;
    pair_scan<false>(S, V, at.gl, at.n);
    pair_shift<false>(S, V, at.gl, at.n);
    float h = fmaf(exp2_fast(-S), bound, V);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float bj = hp[j];
      hp[j] = h;
      h = fmaf(a[j], h, bj);
    }
    // the gradients entering each lane from the right
    S = Sl;
    V = 0.f;
#pragma unroll
    for (int j = 7; j >= 0; --j) V = a[j] * (dy[j] + V);
    pair_scan<true>(S, V, at.gl, at.n);
    const float St = __shfl(S, 0), Vt = __shfl(V, 0);  // used where a wave is one row's
    pair_shift<true>(S, V, at.gl, at.n);
    const float in =
        tile_carry<WPR, true>(tot, (t_hi - 1 - k) & 1, at.wave, at.lane, St, Vt, carry);
    float c = fmaf(exp2_fast(-S), in, V);
    float sum = 0.f;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      float ej;
      const Gate g = gate(r[j], i[j], kappa, &ej);
      const float G = dy[j] + c;
      const float rs = g.w > 0.f ? __builtin_amdgcn_rsqf(g.w) : (g.w != g.w ? g.w : 0.f);
      const float beta = g.w * rs;
      const float db = G * g.s;  // gradient of beta u
      const float aG = a[j] * G;
      const float dz = fmaf(db * u[j], g.a * g.a * rs, -aG * hp[j]);
      c = aG;
      const float bu = db * beta;
      const float di_ = bu * u[j] * g.ns;
      const float dzq = dz * g.q;
      sum += j < nv ? dzq : 0.f;
      u[j] = j < nv ? bu : 0.f;
      i[j] = j < nv ? di_ : 0.f;
      r[j] = j < nv ? dzq * g.nq * lr2 : 0.f;
    }
    acc += (double)sum;
    store_n<T, 8>(static_cast<T*>(p.du) + gbase + t, ns, u);
    store_n<T, 8>(static_cast<T*>(p.dr) + gbase + t, ns, r);
    store_n<T, 8>(static_cast<T*>(p.di) + gbase + t, ns, i);
    if (WPR == 1 && at.n < 64) carry = __shfl(c, at.lane & ~(at.n - 1));
  }
  if (p.dx0 && at.live && at.gl == 0 && (WPR == 1 || (threadIdx.x == 0 && at.seg == 0)))
    p.dx0[at.row] = carry;
  for (int o = 1; o < at.n; o <<= 1) acc += __shfl_xor(acc, o);
  if (WPR == 1) {
    if (at.live && at.gl == 0) p.part[at.row] = acc;
  } else {
    if (at.lane == 0) red[at.wave] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int w = 0; w < WPR; ++w) s += red[w];
      p.part[at.row * p.nseg + at.seg] = s;
    }
  }
}

// dlog_re[h] = 2 log_re[h] sum over the batch (and segments); a wave per channel,
// always in the same order.
__global__ __launch_bounds__(256) void gated_dlog_kernel(const double* __restrict__ part,
                                                         const float* __restrict__ log_re, int B,
                                                         int H, int nseg, float* dlog_re) {
  const int h = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (h >= H) return;
  double s = 0.0;
  const long n = (long)B * nseg;
  for (long j = threadIdx.x & 63; j < n; j += 64) {
    const long b = j / nseg;
    s += part[(b * H + h) * nseg + (j - b * nseg)];
  }
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) dlog_re[h] = (float)(2.0 * (double)log_re[h] * s);
}

// One token for every (b, h).
template <typename T>
__global__ __launch_bounds__(256) void gated_step_kernel(const T* __restrict__ u,
                                                         const T* __restrict__ r,
                                                         const T* __restrict__ i, long long sb,
                                                         const float* __restrict__ log_re,
                                                         const int* __restrict__ lens, long n,
                                                         int H, const float* x0, float* x,
                                                         T* __restrict__ y) {
  const long k = (long)blockIdx.x * 256 + threadIdx.x;
  if (k >= n) return;
  const long b = k / H;
  const long h = k - b * H;
  const float xv = x0 ? x0[k] : 0.f;
  if (lens && lens[b] <= 0) {  // an idle stream: no input is read
    y[k] = (T)0.f;
    if (x) x[k] = xv;
    return;
  }
  const float lr = log_re[h];
  float e;
  const long at = b * sb + h;
  const Gate g = gate((float)r[at], (float)i[at], lr * lr * kLog2e, &e);
  const float v = fmaf(g.a, xv, __builtin_amdgcn_sqrtf(g.w) * (g.s * (float)u[at]));
  if (x) x[k] = v;
  y[k] = (T)v;
}

// Waves per row, lanes per row and segments per row.
struct Plan {
  int wpr, lpr, nseg, seg_tiles;
};

Plan plan_of(long rows, int L) {
  Plan p{1, 64, 1, 1};
  if (L <= kChunk) {  // one wave tile holds the row; short rows share a wave
    p.lpr = 1;
    while (p.lpr < 64 && p.lpr * 8 < L) p.lpr *= 2;
    return p;
  }
  if (rows >= 8192) {
    p.seg_tiles = (L + kChunk - 1) / kChunk;
    return p;
  }
  p.wpr = 4;
  const int ntile = (L + 4 * kChunk - 1) / (4 * kChunk);
  // few rows: segments of whole tiles, about 1024 workgroups in all
  long nseg = rows >= 512 ? 1 : std::min<long>(ntile, (1024 + rows - 1) / rows);
  p.seg_tiles = (int)((ntile + nseg - 1) / nseg);
  p.nseg = (ntile + p.seg_tiles - 1) / p.seg_tiles;
  return p;
}

Args make_args(const GatedCall& c, const Plan& pl) {
  Args a{};
  a.u = c.u;
  a.r = c.r;
  a.i = c.i;
  a.sb = c.stride_b;
  a.log_re = c.log_re;
  a.lens = c.lens;
  a.rows = (long)c.B * c.H;
  a.H = c.H;
  a.L = c.L;
  a.x0 = c.x0;
  a.xT = c.xT;
  a.y = c.y;
  if (c.ckpt) {
    const GatedCkpt k = gated_ckpt_layout(a.rows, c.L, c.kind);
    char* base = static_cast<char*>(c.ckpt);
    a.bounds = reinterpret_cast<float*>(base);
    for (int m = 0; m < 3 && c.kind == 2; ++m) {
      a.q8[m] = reinterpret_cast<int8_t*>(base + k.q8[m]);
      a.e8[m] = reinterpret_cast<uint8_t*>(base + k.q8[m] + ckpt8_exp_offset(a.rows, c.L));
    }
  }
  a.dy = c.dy;
  a.dx = c.dx;
  a.du = c.du;
  a.dr = c.dr;
  a.di = c.di;
  a.sdb = c.grad_stride_b;
  a.dx0 = c.dx0;
  a.nseg = pl.nseg;
  a.seg_tiles = pl.seg_tiles;
  a.lpr = pl.lpr;
  a.agg = static_cast<float2*>(c.ws);
  a.part = reinterpret_cast<double*>(static_cast<char*>(c.ws) +
                                     align_up((size_t)a.rows * pl.nseg * sizeof(float2), 256));
  return a;
}

unsigned grid_of(const Plan& p, long rows) {
  if (p.wpr > 1) return (unsigned)(rows * p.nseg);
  const long per = 4L * (64 / p.lpr);
  return (unsigned)((rows + per - 1) / per);
}

template <typename T, int WPR>
hipError_t fwd_launch(const Args& a, const Plan& pl, int kind, hipStream_t st) {
  const dim3 grid(grid_of(pl, a.rows)), block(threads_of<WPR>());
  if (pl.nseg > 1)
    hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 0, true>), grid, block, 0, st, a);
  switch (kind) {
    case 0: hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 0, false>), grid, block, 0, st, a); break;
    case 1: hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 1, false>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 2, false>), grid, block, 0, st, a); break;
  }
  return hipGetLastError();
}

template <typename T, int WPR, bool Q8>
hipError_t bwd_launch(const Args& a, const Plan& pl, hipStream_t st) {
  const dim3 grid(grid_of(pl, a.rows)), block(threads_of<WPR>());
  if (pl.nseg > 1) hipLaunchKernelGGL((gated_bwd_agg_kernel<T, WPR, Q8>), grid, block, 0, st, a);
  hipLaunchKernelGGL((gated_bwd_kernel<T, WPR, Q8>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t gated_run(const GatedCall& c, bool backward, hipStream_t st) {
  const long rows = (long)c.B * c.H;
  const Plan pl = plan_of(rows, c.L);
  const Args a = make_args(c, pl);
  if (!backward) {
    return pl.wpr == 1 ? fwd_launch<T, 1>(a, pl, c.kind, st) : fwd_launch<T, 4>(a, pl, c.kind, st);
  }
  hipError_t e;
  if (c.kind == 2)
    e = pl.wpr == 1 ? bwd_launch<T, 1, true>(a, pl, st) : bwd_launch<T, 4, true>(a, pl, st);
  else
    e = pl.wpr == 1 ? bwd_launch<T, 1, false>(a, pl, st) : bwd_launch<T, 4, false>(a, pl, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gated_dlog_kernel, dim3((unsigned)((c.H + 3) / 4)), dim3(256), 0, st, a.part,
                     c.log_re, c.B, c.H, pl.nseg, c.dlog_re);
  return hipGetLastError();
}

template <typename T>
hipError_t step_run(const GatedCall& c, hipStream_t st) {
  const long n = (long)c.B * c.H;
  hipLaunchKernelGGL((gated_step_kernel<T>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st,
                     static_cast<const T*>(c.u), static_cast<const T*>(c.r),
                     static_cast<const T*>(c.i), c.stride_b, c.log_re, c.lens, n, c.H, c.x0, c.xT,
                     static_cast<T*>(c.y));
  return hipGetLastError();
}

}  // namespace

size_t ckpt8_exp_offset(long rows, int L) { return align_up((size_t)rows * ckpt8_row(L), 256); }

size_t ckpt8_bytes(long rows, int L) {
  return ckpt8_exp_offset(rows, L) + align_up((size_t)rows * ckpt8_groups(L), 256);
}

GatedCkpt gated_ckpt_layout(long rows, int L, int kind) {
  GatedCkpt k;
  size_t off = align_up((size_t)rows * ((L + kChunk - 1) / kChunk) * sizeof(float), 256);
  for (int m = 0; m < 3 && kind == 2; ++m) {
    k.q8[m] = off;
    off += ckpt8_bytes(rows, L);
  }
  k.total = off;
  return k;
}

size_t gated_workspace(int B, int H, int L) {
  const long rows = (long)B * H;
  const Plan pl = plan_of(rows, L);
  return align_up((size_t)rows * pl.nseg * sizeof(float2), 256) +
         align_up((size_t)rows * pl.nseg * sizeof(double), 256);
}

hipError_t launch_gated_forward(const GatedCall& c, int dtype, hipStream_t st) {
  switch (dtype) {
    case 0: return gated_run<float>(c, false, st);
    case 1: return gated_run<__bf16>(c, false, st);
    default: return gated_run<_Float16>(c, false, st);
  }
}

hipError_t launch_gated_backward(const GatedCall& c, int dtype, hipStream_t st) {
  if ((long)c.B * c.H == 0) {  // no rows: the parameter's gradient is zero
    hipLaunchKernelGGL(gated_dlog_kernel, dim3((unsigned)((c.H + 3) / 4)), dim3(256), 0, st,
                       static_cast<const double*>(nullptr), c.log_re, 0, c.H, 1, c.dlog_re);
    return hipGetLastError();
  }
  switch (dtype) {
    case 0: return gated_run<float>(c, true, st);
    case 1: return gated_run<__bf16>(c, true, st);
    default: return gated_run<_Float16>(c, true, st);
  }
}

hipError_t launch_gated_step(const GatedCall& c, int dtype, hipStream_t st) {
  switch (dtype) {
    case 0: return step_run<float>(c, st);
    case 1: return step_run<__bf16>(c, st);
    default: return step_run<_Float16>(c, st);
  }
}

}  // namespace dssm
