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

constexpr float kTiny = 1.17549435e-38f;

// 1 - exp2(-2 e) for small e: the series of 1 - exp(-x), x = 2 ln(2) e.
// Where exp2(-e) is close to 1, 1 - a^2 would lose its digits.  The border
// weighs the series' length against them: eight terms up to x = 1/2 (the ninth
// is 2^-27 of the first; above, 1 - a^2 keeps 2^-23).  The same for every type
// of activations: states and parameter gradients are float32 in all of them, and
// a token's kernel takes up the state a sequence's left (five terms up to 1/4
// would put the drive off by 12 half steps; a training step of 2^26 bf16
// elements takes 305 us with either, kept in 8 bits 325 against 322).
__device__ __forceinline__ float one_minus_sq(float e, float a) {
  constexpr double c = 2.0 * 0.69314718055994530942;
  const float far = fmaf(-a, a, 1.f);
  float p = (float)(-c * c * c * c * c * c * c * c / 40320.0);
  p = fmaf(p, e, (float)(c * c * c * c * c * c * c / 5040.0));
  p = fmaf(p, e, (float)(-c * c * c * c * c * c / 720.0));
  p = fmaf(p, e, (float)(c * c * c * c * c / 120.0));
  p = fmaf(p, e, (float)(-c * c * c * c / 24.0));
  p = fmaf(p, e, (float)(c * c * c / 6.0));
  p = fmaf(p, e, (float)(-c * c / 2.0));
  p = fmaf(p, e, (float)c);
  return e < (float)(0.5 / c) ? p * e : far;
}

// A value from another lane, by the data-parallel primitives of the vector
// unit; lanes the pattern does not reach get 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL,
                                                               ROWS, 0xf, CTRL < 0x140));
}
constexpr int kRowShl = 0x100, kRowShr = 0x110, kWaveShl = 0x130, kWaveShr = 0x138,
              kBcast15 = 0x142, kBcast31 = 0x143;

__device__ __forceinline__ float lane_of(float x, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ void pair_step(float& S, float& V) {
  const float Sp = dpp<CTRL, ROWS>(S), Vp = dpp<CTRL, ROWS>(V);
  V = fmaf(exp2_fast(-S), Vp, V);
  S += Sp;
}

// Inclusive scan over a wave, in time order or (REV) against it: (S1, V1)
// then (S2, V2) = (S1 + S2, exp2(-S2) V1 + V2).  Lanes without a neighbour
// join (0, 0), which changes nothing.
template <bool REV>
__device__ __forceinline__ void wave_scan(float& S, float& V) {
  if (!REV) {
    pair_step<kRowShr + 1, 0xf>(S, V);
    pair_step<kRowShr + 2, 0xf>(S, V);
    pair_step<kRowShr + 4, 0xf>(S, V);
    pair_step<kRowShr + 8, 0xf>(S, V);
    pair_step<kBcast15, 0xa>(S, V);  // rows 1 and 3 join the row before
    pair_step<kBcast31, 0xc>(S, V);  // rows 2 and 3 join the first half
  } else {
    pair_step<kRowShl + 1, 0xf>(S, V);
    pair_step<kRowShl + 2, 0xf>(S, V);
    pair_step<kRowShl + 4, 0xf>(S, V);
    pair_step<kRowShl + 8, 0xf>(S, V);
    const int lane = threadIdx.x & 63;
    {  // rows 0 and 2 join the row after
      const bool in = !(lane & 16);
      const float S1 = lane_of(S, 16), V1 = lane_of(V, 16);
      const float S3 = lane_of(S, 48), V3 = lane_of(V, 48);
      const float Sp = in ? (lane & 32 ? S3 : S1) : 0.f, Vp = in ? (lane & 32 ? V3 : V1) : 0.f;
      V = fmaf(exp2_fast(-S), Vp, V);
      S += Sp;
    }
    {  // the first half joins the second
      const float Sh = lane_of(S, 32), Vh = lane_of(V, 32);
      const float Sp = lane < 32 ? Sh : 0.f, Vp = lane < 32 ? Vh : 0.f;
      V = fmaf(exp2_fast(-S), Vp, V);
      S += Sp;
    }
  }
}

// The same over groups of n lanes (n a power of two), for short rows.
template <bool REV>
__device__ __forceinline__ void group_scan(float& S, float& V, int gl, int n) {
  for (int o = 1; o < n; o <<= 1) {
    const float Sp = REV ? __shfl_down(S, o) : __shfl_up(S, o);
    const float Vp = REV ? __shfl_down(V, o) : __shfl_up(V, o);
    if (REV ? gl + o < n : gl >= o) {
      V = fmaf(exp2_fast(-S), Vp, V);
      S += Sp;
    }
  }
}

// The neighbour's inclusive pair ((0, 0) at the first lane).
template <bool REV, bool SHORT>
__device__ __forceinline__ void pair_shift(float& S, float& V, int gl, int n) {
  S = dpp<REV ? kWaveShl : kWaveShr, 0xf>(S);
  V = dpp<REV ? kWaveShl : kWaveShr, 0xf>(V);
  if (SHORT && (REV ? gl == n - 1 : gl == 0)) S = V = 0.f;
}

// Scans a tile and leaves each lane what enters it; St, Vt: the whole tile's
// pair (for rows of whole waves).
template <bool REV, bool SHORT>
__device__ __forceinline__ void tile_scan(float& S, float& V, int gl, int n, float* St,
                                          float* Vt) {
  if (SHORT)
    group_scan<REV>(S, V, gl, n);
  else
    wave_scan<REV>(S, V);
  *St = lane_of(S, REV ? 0 : 63);
  *Vt = lane_of(V, REV ? 0 : 63);
  pair_shift<REV, SHORT>(S, V, gl, n);
}

// What enters segment `seg` of a split row: the pairs of the segments before
// it (REV: after it) applied to `start`, four neighbours to a lane and all
// asked for at once.  Every lane of the wave gets it.
constexpr int kJoin = 256;  // segments of a row at most (64 lanes, four each)
template <bool REV>
__device__ float join_segments(const float2* agg, int nseg, int seg, float start) {
  const int lane = threadIdx.x & 63;
  const int count = REV ? nseg - 1 - seg : seg;
  // lane order = order of application
  float2 t[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = 4 * lane + k;
    t[k] = make_float2(0.f, 0.f);
    if (j < count) t[k] = agg[REV ? nseg - 1 - j : j];
  }
  float S = 0.f, V = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    V = fmaf(exp2_fast(-t[k].x), V, t[k].y);
    S += t[k].x;
  }
  wave_scan<false>(S, V);
  return fmaf(exp2_fast(-lane_of(S, 63)), start, lane_of(V, 63));
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

__device__ __forceinline__ int row_len(const Args& p, long b) {
  if (!p.lens) return p.L;
  return min(max(p.lens[b], 0), p.L);
}

__device__ __forceinline__ int clamp8(int n) { return min(max(n, 0), 8); }

// Eight steps of one lane as they lie in memory, so that the next tile's can be
// on their way while this one is worked on.  Steps that are not live hold
// `fill`: for the recurrence gate -inf, which shuts it (a = 1, no drive, no
// gradient), for the others 0.
template <typename T>
struct Raw {
  Packed<T, 8> v;
  __device__ __forceinline__ void fetch(const T* p, int nv, T fill) { v.load(p, nv, fill); }
  __device__ __forceinline__ void get(float* out, int, float) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = v[k];
  }
};

// The same of a row in 8 bits.
struct Raw8 {
  uint2 q;
  int byte;
  __device__ __forceinline__ void fetch(const int8_t* q8, const uint8_t* e8, int t, int nv) {
    q = make_uint2(0, 0);
    byte = 1;
    if (nv > 0) {
      q = *reinterpret_cast<const uint2*>(q8 + t);
      byte = e8[t / kGroup];
    }
  }
  __device__ __forceinline__ void get(float* out, int nv, float fill) const {
    dequantise8(q, byte, out);
    if (nv < 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) out[k] = k < nv ? out[k] : fill;
    }
  }
};

template <typename T>
__device__ __forceinline__ T shut() { return (T)(-__builtin_inff()); }

// u, r and i of a row, from the inputs or (Q8) their 8-bit form.
template <typename T, bool Q8>
struct Source {
  const T *u, *r, *i;
  __device__ Source(const Args& p, long row, long b) {
    const size_t at = (size_t)(b * p.sb + (row - b * p.H) * p.L);
    u = static_cast<const T*>(p.u) + at;
    r = static_cast<const T*>(p.r) + at;
    i = static_cast<const T*>(p.i) + at;
  }
  struct Tile {
    Raw<T> u, r, i;
  };
  __device__ __forceinline__ void fetch_r(Tile& x, int t, int nv) const {
    x.r.fetch(r + t, nv, shut<T>());
  }
  __device__ __forceinline__ void fetch(Tile& x, int t, int nv) const {
    x.u.fetch(u + t, nv, (T)0.f);
    x.r.fetch(r + t, nv, shut<T>());
    x.i.fetch(i + t, nv, (T)0.f);
  }
};

template <typename T>
struct Source<T, true> {
  const int8_t* q[3];
  const uint8_t* e[3];
  __device__ Source(const Args& p, long row, long) {
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      q[m] = p.q8[m] + (size_t)row * ckpt8_row(p.L);
      e[m] = p.e8[m] + (size_t)row * ckpt8_groups(p.L);
    }
  }
  struct Tile {
    Raw8 u, r, i;
  };
  __device__ __forceinline__ void fetch_r(Tile& x, int t, int nv) const {
    x.r.fetch(q[1], e[1], t, nv);
  }
  __device__ __forceinline__ void fetch(Tile& x, int t, int nv) const {
    x.u.fetch(q[0], e[0], t, nv);
    x.r.fetch(q[1], e[1], t, nv);
    x.i.fetch(q[2], e[2], t, nv);
  }
};

// Which row, segment and lanes a thread works on.  WPR waves share a row; with
// WPR == 1 a workgroup of 4 waves holds 4 rows, or (SHORT: rows of at most
// 256 steps) 4 (64 / n) of them, n lanes each.
template <int WPR, bool SHORT>
struct Place {
  long row, b;
  int seg, gl, n, wave, lane, t0;
  bool live;
  __device__ Place(const Args& p) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    seg = 0;
    n = SHORT ? p.lpr : 64;
    gl = SHORT ? lane & (n - 1) : lane;
    if (WPR == 1) {
      row = (long)blockIdx.x * 4 + wave;
      if (SHORT) row = row * (64 / n) + lane / n;
    } else {
      row = blockIdx.x / p.nseg;
      seg = blockIdx.x - (int)row * p.nseg;
    }
    live = row < p.rows;
    if (!live) row = p.rows - 1;
    b = row / p.H;
    t0 = (WPR > 1 ? wave * kChunk : 0) + gl * 8;
  }
};

template <int WPR>
constexpr int threads_of() { return WPR == 1 ? 256 : 64 * WPR; }

// The carries of a tile's WPR waves: every wave leaves its pair, then takes
// what enters it and what leaves the tile.  One barrier: the buffers alternate.
template <int WPR, bool REV>
__device__ __forceinline__ float tile_carry(float2 (*tot)[WPR], int flip, int wave, int lane,
                                            float S, float V, float& carry, float* Ssum) {
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
    if (Ssum) *Ssum += t.x;
  }
  carry = c;
  return in;
}

// log_re^2, finite with its product by log2(e) unless NaN: a shut gate's zero
// times either has to be 0.
__device__ __forceinline__ float square_of(float log_re) {
  const float s = log_re * log_re;
  return s > 0x1p126f ? 0x1p126f : s;
}

// Forward over a row (or one segment of it).  AGG: only the segment's pair.
// CK: 0 nothing kept, 1 the state entering every chunk, 2 also u, r, i in 8 bits.
template <typename T, int WPR, int CK, bool SHORT, bool AGG>
__global__ __launch_bounds__(threads_of<WPR>()) void gated_fwd_kernel(Args p) {
  __shared__ float2 tot[2][WPR];
  const Place<WPR, SHORT> at(p);
  const int len = at.live ? row_len(p, at.b) : 0;
  const int end = at.live ? p.L : 0;
  const float lr = p.log_re[at.row - at.b * p.H];
  const float kappa = square_of(lr) * kLog2e;
  constexpr int tile = kChunk * WPR;
  const int ntile = (p.L + tile - 1) / tile;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  if (AGG && at.seg == p.nseg - 1) {
    // Nobody joins the last segment: its place keeps the state before the row,
    // which every segment starts from and the last one may overwrite (xT = x0).
    if (threadIdx.x == 0)
      p.agg[at.row * p.nseg + at.seg] = make_float2(0.f, p.x0 ? p.x0[at.row] : 0.f);
    return;
  }
  const Source<T, false> src(p, at.row, at.b);
  typename Source<T, false>::Tile next;
  if (t_lo < t_hi) src.fetch(next, t_lo * tile + at.t0, clamp8(len - t_lo * tile - at.t0));
  float carry = 0.f;
  if (WPR > 1 && !AGG && p.nseg > 1) {
    const float2* agg = p.agg + at.row * p.nseg;
    carry = join_segments<false>(agg, p.nseg, at.seg, agg[p.nseg - 1].y);
  } else if (!AGG && p.x0) {
    carry = p.x0[at.row];
  }
  const float start = carry;
  float Sseg = 0.f;
  for (int k = t_lo; k < t_hi; ++k) {
    const int t = k * tile + at.t0;
    const int nv = clamp8(len - t);
    if (!SHORT && k * tile >= len) {  // behind the row's end: the state stays, outputs are 0
      if (AGG) break;
      const int ns = clamp8(end - t);
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      store_n<T, 8>(static_cast<T*>(p.y) + (size_t)at.row * p.L + t, ns, zero);
      if (CK >= 1 && at.gl == 0 && t < end)
        p.bounds[(size_t)at.row * ((p.L + kChunk - 1) / kChunk) + t / kChunk] = carry;
      if (CK == 2 && ns > 0) {
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          *reinterpret_cast<uint2*>(p.q8[m] + (size_t)at.row * ckpt8_row(p.L) + t) =
              make_uint2(0, 0);
          if ((t & (kGroup - 1)) == 0)
            p.e8[m][(size_t)at.row * ckpt8_groups(p.L) + t / kGroup] = (uint8_t)group_byte(0);
        }
      }
      continue;
    }
    const typename Source<T, false>::Tile now = next;
    if (k + 1 < t_hi) src.fetch(next, t + tile, clamp8(len - t - tile));
    float u[8], r[8], i[8], a[8], b[8];
    now.u.get(u, nv, 0.f);
    now.r.get(r, nv, 0.f);
    now.i.get(i, nv, 0.f);
    float S = 0.f, V = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float rest;
      const float e = kappa * sigmoid_pair(r[j], &rest);
      const float s = sigmoid_pair(i[j], &rest);
      a[j] = exp2_fast(-e);
      b[j] = __builtin_amdgcn_sqrtf(one_minus_sq(e, a[j])) * (s * u[j]);
      S += e;
      V = fmaf(a[j], V, b[j]);
    }
    float St, Vt;
    tile_scan<false, SHORT>(S, V, at.gl, at.n, &St, &Vt);
    const float in = tile_carry<WPR, false>(tot, (k - t_lo) & 1, at.wave, at.lane, St, Vt, carry,
                                            AGG ? &Sseg : nullptr);
    if (AGG) continue;
    const int ns = clamp8(end - t);
    if (CK >= 1 && at.gl == 0 && t < end)
      p.bounds[(size_t)at.row * ((p.L + kChunk - 1) / kChunk) + t / kChunk] = in;
    if (CK == 2) {
      if (nv < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = j < nv ? r[j] : 0.f;
      }
      const float* x[3] = {u, r, i};
      const int width = SHORT ? min(8, at.n) : 8;
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        uint2 q;
        const int byte = m == 0 ? quantise8<T, false>(x[m], width, &q)
                                : quantise8<T, true>(x[m], width, &q);
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
      y[j] = h;
    }
    if (nv < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = j < nv ? y[j] : 0.f;
    }
    store_n<T, 8>(static_cast<T*>(p.y) + (size_t)at.row * p.L + t, ns, y);
    if (SHORT) {  // the last lane's state is the row's; an empty row keeps its own
      const float last = __shfl(h, at.lane | (at.n - 1));
      carry = len > 0 ? last : start;
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
  const Place<WPR, false> at(p);
  const int len = row_len(p, at.b);
  const float lr = p.log_re[at.row - at.b * p.H];
  const float kappa = square_of(lr) * kLog2e;
  constexpr int tile = kChunk * WPR;
  const int ntile = (p.L + tile - 1) / tile;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  if (at.seg == 0) return;  // nobody joins the first segment
  const Source<T, Q8> src(p, at.row, at.b);
  const T* dyp = static_cast<const T*>(p.dy) + (size_t)at.row * p.L;
  float carry = 0.f, Sseg = 0.f;
  for (int k = t_hi - 1; k >= t_lo; --k) {
    if (k * tile >= len) continue;
    const int t = k * tile + at.t0;
    const int nv = clamp8(len - t);
    typename Source<T, Q8>::Tile now;
    Raw<T> g;
    src.fetch_r(now, t, nv);
    g.fetch(dyp + t, nv, (T)0.f);
    float r[8], dy[8];
    now.r.get(r, nv, -__builtin_inff());
    g.get(dy, nv, 0.f);
    float S = 0.f, V = 0.f;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      float rest;
      const float e = kappa * sigmoid_pair(r[j], &rest);
      V = exp2_fast(-e) * (dy[j] + V);
      S += e;
    }
    float St, Vt;
    tile_scan<true, false>(S, V, at.gl, 64, &St, &Vt);
    tile_carry<WPR, true>(tot, (t_hi - 1 - k) & 1, at.wave, at.lane, St, Vt, carry, &Sseg);
  }
  if (threadIdx.x == 0) p.agg[at.row * p.nseg + at.seg] = make_float2(Sseg, carry);
}

// Backward over a row (or one segment of it), tiles from the last to the
// first.  Each wave's tile is one chunk, whose entering state the checkpoint
// holds: the states need no walk of their own.
template <typename T, int WPR, bool SHORT, bool Q8>
__global__ __launch_bounds__(threads_of<WPR>()) void gated_bwd_kernel(Args p) {
  __shared__ float2 tot[2][WPR];
  __shared__ double red[threads_of<WPR>() / 64];
  const Place<WPR, SHORT> at(p);
  const int len = at.live ? row_len(p, at.b) : 0;
  const int end = at.live ? p.L : 0;
  const float lr = p.log_re[at.row - at.b * p.H];
  const float lr2 = square_of(lr);
  const float kappa = lr2 * kLog2e;
  const size_t gbase = (size_t)(at.b * p.sdb + (at.row - at.b * p.H) * p.L);
  constexpr int tile = kChunk * WPR;
  const int ntile = (p.L + tile - 1) / tile;
  const int nch = (p.L + kChunk - 1) / kChunk;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  const Source<T, Q8> src(p, at.row, at.b);
  const T* dyp = static_cast<const T*>(p.dy) + (size_t)at.row * p.L;
  const float* bounds = p.bounds + (size_t)at.row * nch;
  typename Source<T, Q8>::Tile next;
  Raw<T> next_g;
  float next_x = 0.f;
  auto fetch = [&](int k) {
    const int t = k * tile + at.t0;
    src.fetch(next, t, clamp8(len - t));
    next_g.fetch(dyp + t, clamp8(len - t), (T)0.f);
    next_x = bounds[min(t / kChunk, nch - 1)];
  };
  if (t_lo < t_hi) fetch(t_hi - 1);
  float carry = p.dx ? p.dx[at.row] : 0.f;
  if (WPR > 1 && p.nseg > 1)
    carry = join_segments<true>(p.agg + at.row * p.nseg, p.nseg, at.seg, carry);
  const float start = carry;
  double acc = 0.0;
  for (int k = t_hi - 1; k >= t_lo; --k) {
    const int t = k * tile + at.t0;
    const int nv = clamp8(len - t);
    const typename Source<T, Q8>::Tile now = next;
    const Raw<T> g = next_g;
    const float bound = next_x;
    if (k > t_lo) fetch(k - 1);
    if (!SHORT && k * tile >= len) {  // behind the row's end: nothing enters from there
      const int ns = clamp8(end - t);
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      store_n<T, 8>(static_cast<T*>(p.du) + gbase + t, ns, zero);
      store_n<T, 8>(static_cast<T*>(p.dr) + gbase + t, ns, zero);
      store_n<T, 8>(static_cast<T*>(p.di) + gbase + t, ns, zero);
      continue;
    }
    float u[8], r[8], i[8], dy[8];
    now.u.get(u, nv, 0.f);
    now.r.get(r, nv, -__builtin_inff());
    now.i.get(i, nv, 0.f);
    g.get(dy, nv, 0.f);
    float a[8], q[8], qn[8], b[8], bn[8], c2[8], hp[8];
    // the states before each step, from the chunk's entering state
    float S = 0.f, V = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float sn;
      q[j] = sigmoid_pair(r[j], &qn[j]);
      const float s = sigmoid_pair(i[j], &sn);
      const float e = kappa * q[j];
      a[j] = exp2_fast(-e);
      const float w = one_minus_sq(e, a[j]);
      const float rs = __builtin_amdgcn_rsqf(w < kTiny ? kTiny : w);  // 1 / beta
      const float B = w * rs * s;  // du = G B
      b[j] = B;
      bn[j] = sn;
      c2[j] = a[j] * rs;  // a / beta
      S += e;
      V = fmaf(a[j], V, B * u[j]);
    }
    const float Sl = S;
    float St, Vt;
    tile_scan<false, SHORT>(S, V, at.gl, at.n, &St, &Vt);
    float h = fmaf(exp2_fast(-S), bound, V);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hp[j] = h;
      h = fmaf(a[j], h, b[j] * u[j]);
    }
    // the gradients entering each lane from the right
    S = Sl;
    V = 0.f;
#pragma unroll
    for (int j = 7; j >= 0; --j) V = a[j] * (dy[j] + V);
    tile_scan<true, SHORT>(S, V, at.gl, at.n, &St, &Vt);
    const float in = tile_carry<WPR, true>(tot, (t_hi - 1 - k) & 1, at.wave, at.lane, St, Vt,
                                           carry, nullptr);
    float c = fmaf(exp2_fast(-S), in, V);
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      const float G = dy[j] + c;
      c = a[j] * G;
      const float du = G * b[j];
      const float gb = du * u[j];
      const float dz = fmaf(gb * c2[j], c2[j], -c * hp[j]);
      u[j] = du;
      i[j] = gb * bn[j];
      r[j] = dz * q[j];
    }
    if (nv < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = j < nv ? u[j] : 0.f;
        r[j] = j < nv ? r[j] : 0.f;
        i[j] = j < nv ? i[j] : 0.f;
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum += r[j];
      r[j] *= qn[j] * lr2;
    }
    if (nv < 8) {  // with a parameter that is NaN too
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = j < nv ? r[j] : 0.f;
    }
    acc += (double)sum;
    const int ns = clamp8(end - t);
    store_n<T, 8>(static_cast<T*>(p.du) + gbase + t, ns, u);
    store_n<T, 8>(static_cast<T*>(p.dr) + gbase + t, ns, r);
    store_n<T, 8>(static_cast<T*>(p.di) + gbase + t, ns, i);
    if (SHORT) {
      const float first = __shfl(c, at.lane & ~(at.n - 1));
      carry = len > 0 ? first : start;
    }
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
  // nothing to add up is 0, whatever the parameter
  if ((threadIdx.x & 63) == 0)
    dlog_re[h] = (float)(s != 0.0 ? 2.0 * (double)log_re[h] * s : 0.0);
}

// One token for every (b, h); V neighbouring channels to a thread.
template <typename T, int V>
__global__ __launch_bounds__(256) void gated_step_kernel(const T* __restrict__ u,
                                                         const T* __restrict__ r,
                                                         const T* __restrict__ i, long long sb,
                                                         const float* __restrict__ log_re,
                                                         const int* __restrict__ lens, unsigned n,
                                                         unsigned per, int H, const float* x0,
                                                         float* x, T* __restrict__ y) {
  const unsigned k = blockIdx.x * 256 + threadIdx.x;
  if (k >= n) return;
  const unsigned b = k / per;
  const int h = (int)(k - b * per) * V;
  const size_t row = (size_t)b * H + h;
  const int m = min(V, H - h);
  float xv[V], uv[V], rv[V], iv[V], lr[V], yv[V];
  // an idle stream's inputs are not read
  const int live = lens && lens[b] <= 0 ? 0 : m;
  load_n<float, V>(x0 ? x0 + row : log_re + h, x0 ? m : 0, xv);
  load_n<T, V>(u + b * sb + h, live, uv);
  load_n<T, V>(r + b * sb + h, live, rv);
  load_n<T, V>(i + b * sb + h, live, iv);
  load_n<float, V>(log_re + h, live, lr);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float rest;
    const float e = square_of(lr[j]) * kLog2e * sigmoid_pair(rv[j], &rest);
    const float s = sigmoid_pair(iv[j], &rest);
    const float a = exp2_fast(-e);
    const float v =
        fmaf(a, xv[j], __builtin_amdgcn_sqrtf(one_minus_sq(e, a)) * (s * uv[j]));
    xv[j] = live ? v : xv[j];
    yv[j] = live ? v : 0.f;
  }
  if (x) store_n<float, V>(x + row, m, xv);
  store_n<T, V>(y + row, m, yv);
}

// Waves per row, lanes per row and segments per row.
struct Plan {
  int wpr, lpr, nseg, seg_tiles;
};

// A row of up to 512 steps is one wave tile; shorter ones share a wave.
//
// Longer rows are walked by four waves, or by one each when there are enough
// of them: the waves then meet no barrier and all rows are under way at once
// (bf16, 2^26 elements, forward / backward: 8192 rows 109 / 190 us against 107 /
// 215 with four waves; 2048 rows 111 / 192 against 112 / 195; 1024 rows 141 /
// 244 against 113 / 200).
//
// Few rows leave compute units idle: they are cut into segments, about 2048
// workgroups in all and no more to a row than a wave joins at once, at the price
// of reading the inputs (backward: the recurrence gate and dy) twice (bf16, 2^25 elements, forward / backward: 64
// rows 90 / 109 us against 274 / 403 unsplit, with 1024 workgroups 92 / 114;
// 256 rows 91 / 111 against 76 / 121; 512 rows 88 / 108 against 55 / 103).
Plan plan_of(long rows, int L, bool backward) {
  Plan p{1, 64, 1, 1};
  if (L <= kChunk) {
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
  const long nseg = rows >= (backward ? 512 : 256)
                        ? 1
                        : std::min<long>(std::min(ntile, kJoin), (2048 + rows - 1) / rows);
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

template <typename T, int WPR, bool SHORT>
hipError_t fwd_launch(const Args& a, const Plan& pl, int kind, hipStream_t st) {
  const dim3 grid(grid_of(pl, a.rows)), block(threads_of<WPR>());
  if constexpr (WPR > 1) {
    if (pl.nseg > 1)
      hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 0, false, true>), grid, block, 0, st, a);
  }
  switch (kind) {
    case 0: hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 0, SHORT, false>), grid, block, 0, st, a); break;
    case 1: hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 1, SHORT, false>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((gated_fwd_kernel<T, WPR, 2, SHORT, false>), grid, block, 0, st, a); break;
  }
  return hipGetLastError();
}

template <typename T, int WPR, bool SHORT, bool Q8>
hipError_t bwd_launch(const Args& a, const Plan& pl, hipStream_t st) {
  const dim3 grid(grid_of(pl, a.rows)), block(threads_of<WPR>());
  if constexpr (WPR > 1) {
    if (pl.nseg > 1) hipLaunchKernelGGL((gated_bwd_agg_kernel<T, WPR, Q8>), grid, block, 0, st, a);
  }
  hipLaunchKernelGGL((gated_bwd_kernel<T, WPR, SHORT, Q8>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <typename T, bool Q8>
hipError_t bwd_plan(const Args& a, const Plan& pl, hipStream_t st) {
  if (pl.wpr > 1) return bwd_launch<T, 4, false, Q8>(a, pl, st);
  return pl.lpr < 64 ? bwd_launch<T, 1, true, Q8>(a, pl, st)
                     : bwd_launch<T, 1, false, Q8>(a, pl, st);
}

template <typename T>
hipError_t gated_run(const GatedCall& c, bool backward, hipStream_t st) {
  const long rows = (long)c.B * c.H;
  const Plan pl = plan_of(rows, c.L, backward);
  const Args a = make_args(c, pl);
  if (!backward) {
    if (pl.wpr > 1) return fwd_launch<T, 4, false>(a, pl, c.kind, st);
    return pl.lpr < 64 ? fwd_launch<T, 1, true>(a, pl, c.kind, st)
                       : fwd_launch<T, 1, false>(a, pl, c.kind, st);
  }
  const hipError_t e = c.kind == 2 ? bwd_plan<T, true>(a, pl, st) : bwd_plan<T, false>(a, pl, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gated_dlog_kernel, dim3((unsigned)((c.H + 3) / 4)), dim3(256), 0, st, a.part,
                     c.log_re, c.B, c.H, pl.nseg, c.dlog_re);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t step_launch(const GatedCall& c, hipStream_t st) {
  const unsigned per = (unsigned)(c.H + V - 1) / V;
  const unsigned n = (unsigned)c.B * per;
  hipLaunchKernelGGL((gated_step_kernel<T, V>), dim3((n + 255) / 256), dim3(256), 0, st,
                     static_cast<const T*>(c.u), static_cast<const T*>(c.r),
                     static_cast<const T*>(c.i), c.stride_b, c.log_re, c.lens, n, per, c.H, c.x0,
                     c.xT, static_cast<T*>(c.y));
  return hipGetLastError();
}

// Up to 2^17 channels a thread each fills the device sooner; more are
// bound by memory and take four to a thread.
template <typename T>
hipError_t step_run(const GatedCall& c, hipStream_t st) {
  return (long)c.B * c.H <= (1L << 17) ? step_launch<T, 1>(c, st) : step_launch<T, 4>(c, st);
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
  // the backward pass is split at least as often as the forward pass
  const Plan pl = plan_of(rows, L, true);
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
