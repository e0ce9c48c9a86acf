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
  int B, H, L, ntile;  // strips per batch row
  float eps;
  void *o, *n;
  float* stats;
  const void *d_o, *d_n;
  void *dx, *dy, *dg;
  long long sdg;
  float* part;         // [workgroups][3][H]
};

// v summed over the LT lanes of one channel.
template <int LT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < LT; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// v[0..VE) summed over the workgroup's lanes of the same strip column; every
// thread gets the totals.  buf: [NT / 64][LT VE] floats.  Two barriers.
template <int NT, int LT, int VE>
__device__ __forceinline__ void strip_sum(float* v, float* buf) {
#pragma unroll
  for (int o = LT; o < 64; o <<= 1)
#pragma unroll
    for (int k = 0; k < VE; ++k) v[k] += __shfl_xor(v[k], o);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lt = lane % LT;
  __syncthreads();  // the buffer's last readers are done
  if (lane < LT)
#pragma unroll
    for (int k = 0; k < VE; ++k) buf[wave * (LT * VE) + lt * VE + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < VE; ++k) v[k] = 0.f;
  for (int w = 0; w < NT / 64; ++w)
#pragma unroll
    for (int k = 0; k < VE; ++k) v[k] += buf[w * (LT * VE) + lt * VE + k];
}

// Mean (layer norm) and factor of the columns held in h[KH], per step.
template <typename T, bool LAYER, int NT, int LT, int VE, int KH, typename Vec>
__device__ __forceinline__ void column_stats(const Vec* a, int H, int rs, float inv_h, float eps,
                                             int nv, float* buf, float* mean, float* rstd) {
  constexpr int NR = NT / LT;
#pragma unroll
  for (int k = 0; k < VE; ++k) mean[k] = 0.f;
  if (LAYER) {
#pragma unroll
    for (int j = 0; j < KH; ++j)
#pragma unroll
      for (int k = 0; k < VE; ++k) mean[k] += (float)a[j][k];
    strip_sum<NT, LT, VE>(mean, buf);
#pragma unroll
    for (int k = 0; k < VE; ++k) mean[k] *= inv_h;
  }
#pragma unroll
  for (int k = 0; k < VE; ++k) rstd[k] = 0.f;
#pragma unroll
  for (int j = 0; j < KH; ++j)
    if (rs + j * NR < H)  // channels past H hold 0, which is off the mean
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const float d = (float)a[j][k] - mean[k];
        rstd[k] = fmaf(d, d, rstd[k]);
      }
  strip_sum<NT, LT, VE>(rstd, buf);
#pragma unroll
  for (int k = 0; k < VE; ++k)
    rstd[k] = k < nv ? __builtin_amdgcn_rsqf(fmaf(rstd[k], inv_h, eps)) : 0.f;
}

template <typename T, int VE>
__device__ __forceinline__ typename VecOf<T, VE>::type load_vec(const T* p, int n) {
  typename VecOf<T, VE>::type v;
  if (n >= VE) {
    v = *reinterpret_cast<const typename VecOf<T, VE>::type*>(p);
  } else {
#pragma unroll
    for (int k = 0; k < VE; ++k) v[k] = k < n ? p[k] : (T)0.f;
  }
  return v;
}

template <typename T, int VE>
__device__ __forceinline__ void store_vec(T* p, int n, typename VecOf<T, VE>::type v) {
  if (n >= VE) {
    *reinterpret_cast<typename VecOf<T, VE>::type*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < VE; ++k)
      if (k < n) p[k] = v[k];
  }
}

template <typename T, bool LAYER, int NT, int LT, int VE, int KH>
__global__ __launch_bounds__(NT) void resnorm_fwd_kernel(Args p) {
  typedef typename VecOf<T, VE>::type Vec;
  constexpr int NR = NT / LT;
  __shared__ float buf[(NT / 64) * LT * VE];
  const int b = blockIdx.x / p.ntile;
  const int lt = threadIdx.x % LT, rs = threadIdx.x / LT;
  const int t = (blockIdx.x - b * p.ntile) * (LT * VE) + lt * VE;
  const int len = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  const int nv = min(max(len - t, 0), VE), ns = min(max(p.L - t, 0), VE);
  const float inv_h = 1.f / (float)p.H;
  const size_t base = (size_t)b * p.H * p.L + t;
  const T* x = static_cast<const T*>(p.x) + base;
  const size_t plane = (size_t)p.B * p.L;
  const size_t at = (size_t)b * p.L + t;
  Vec a[KH];
  float mean[VE], rstd[VE];
  if (p.y) {
    const T* y = static_cast<const T*>(p.y) + base;
    const T* g = static_cast<const T*>(p.g) + (p.g ? (size_t)(b * p.sg) + t : 0);
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      const int h = rs + j * NR;
      a[j] = load_vec<T, VE>(y + (size_t)h * p.L, h < p.H ? nv : 0);
    }
    column_stats<T, LAYER, NT, LT, VE, KH>(a, p.H, rs, inv_h, p.eps, nv, buf, mean, rstd);
    if (p.stats && rs == 0) {
      if (LAYER) store_n<float, VE>(p.stats + at, ns, mean);
      store_n<float, VE>(p.stats + (LAYER ? plane : 0) + at, ns, rstd);
    }
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      const int h = rs + j * NR;
      const bool in = h < p.H;
      const Vec xv = load_vec<T, VE>(x + (size_t)h * p.L, in ? nv : 0);
      float c = in ? p.w_post[h] * p.scale[h] : 0.f;
      float gv[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) gv[k] = 1.f;
      if (p.g) {
        const Vec gr = load_vec<T, VE>(g + (size_t)h * p.L, in ? nv : 0);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          float rest;
          gv[k] = (float)gr[k] * sigmoid_pair((float)gr[k], &rest);
        }
      }
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const float v = ((float)a[j][k] - mean[k]) * rstd[k];
        a[j][k] = (T)(k < nv ? fmaf(v * c, gv[k], (float)xv[k]) : 0.f);
      }
      if (in) store_vec<T, VE>(static_cast<T*>(p.o) + base + (size_t)h * p.L, ns, a[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < KH; ++j) {
      const int h = rs + j * NR;
      a[j] = load_vec<T, VE>(x + (size_t)h * p.L, h < p.H ? nv : 0);
    }
  }
  if (!p.n) return;
  // the norm before the next block is of the stream as it is stored
  column_stats<T, LAYER, NT, LT, VE, KH>(a, p.H, rs, inv_h, p.eps, nv, buf, mean, rstd);
  if (p.stats && rs == 0) {
    if (LAYER) store_n<float, VE>(p.stats + 2 * plane + at, ns, mean);
    store_n<float, VE>(p.stats + (LAYER ? 3 : 1) * plane + at, ns, rstd);
  }
#pragma unroll
  for (int j = 0; j < KH; ++j) {
    const int h = rs + j * NR;
    if (h >= p.H) continue;
    const float w = p.w_pre[h];
    Vec out;
#pragma unroll
    for (int k = 0; k < VE; ++k)
      out[k] = (T)(k < nv ? ((float)a[j][k] - mean[k]) * rstd[k] * w : 0.f);
    store_vec<T, VE>(static_cast<T*>(p.n) + base + (size_t)h * p.L, ns, out);
  }
}

// Strips w, w + gridDim.x, ... of one workgroup.  Its sums over b, t stay in
// LDS until the end: a channel is always the same LT lanes'.
template <typename T, bool LAYER, int NT, int LT, int VE>
__global__ __launch_bounds__(NT) void resnorm_bwd_kernel(Args p) {
  constexpr int NR = NT / LT;
  __shared__ float buf[(NT / 64) * LT * VE];
  __shared__ float sums[3 * kResnormMaxH / LT];  // [3][H]
  const int lt = threadIdx.x % LT, rs = threadIdx.x / LT;
  const int H = p.H;
  const float inv_h = 1.f / (float)H;
  const size_t plane = (size_t)p.B * p.L;
  for (int h = rs; h < H; h += NR)
    if (lt == 0) sums[h] = sums[H + h] = sums[2 * H + h] = 0.f;
  const int total = p.B * p.ntile;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const int b = tile / p.ntile;
    const int t = (tile - b * p.ntile) * (LT * VE) + lt * VE;
    const int len = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
    const int nv = min(max(len - t, 0), VE), ns = min(max(p.L - t, 0), VE);
    const size_t base = (size_t)b * H * p.L + t;
    const size_t at = (size_t)b * p.L + t;
    const T* o = static_cast<const T*>(p.x) + base;
    const T* dn = p.d_n ? static_cast<const T*>(p.d_n) + base : nullptr;
    const T* dout = p.d_o ? static_cast<const T*>(p.d_o) + base : nullptr;
    float mo[VE], ro[VE], s1[VE], s0[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) mo[k] = ro[k] = s1[k] = s0[k] = 0.f;
    if (dn) {
      if (LAYER) load_n<float, VE>(p.stats + 2 * plane + at, nv, mo);
      load_n<float, VE>(p.stats + (LAYER ? 3 : 1) * plane + at, nv, ro);
      for (int h = rs; h < H; h += NR) {
        const float w = p.w_pre[h];
        float ov[VE], dv[VE], sum = 0.f;
        load_n<T, VE>(o + (size_t)h * p.L, nv, ov);
        load_n<T, VE>(dn + (size_t)h * p.L, nv, dv);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float oh = (ov[k] - mo[k]) * ro[k];
          const float P = dv[k] * w;
          s1[k] = fmaf(P, oh, s1[k]);
          if (LAYER) s0[k] += P;
          sum = fmaf(dv[k], oh, sum);  // past the end dv is 0
        }
        sum = lanes_sum<LT>(sum);
        if (lt == 0) sums[2 * H + h] += sum;
      }
      strip_sum<NT, LT, VE>(s1, buf);
      if (LAYER) strip_sum<NT, LT, VE>(s0, buf);
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        s1[k] *= inv_h;
        s0[k] *= inv_h;
      }
    }
    // t of one channel's steps
    auto stream = [&](int h, float* tv) {
#pragma unroll
      for (int k = 0; k < VE; ++k) tv[k] = 0.f;
      if (dout) load_n<T, VE>(dout + (size_t)h * p.L, nv, tv);
      if (dn) {
        const float w = p.w_pre[h];
        float ov[VE], dv[VE];
        load_n<T, VE>(o + (size_t)h * p.L, nv, ov);
        load_n<T, VE>(dn + (size_t)h * p.L, nv, dv);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float oh = (ov[k] - mo[k]) * ro[k];
          float q = fmaf(dv[k], w, -oh * s1[k]);
          if (LAYER) q -= s0[k];
          tv[k] = fmaf(ro[k], q, tv[k]);
        }
      }
    };
    if (!p.y) {
      for (int h = rs; h < H; h += NR) {
        float tv[VE];
        stream(h, tv);
        store_n<T, VE>(static_cast<T*>(p.dx) + base + (size_t)h * p.L, ns, tv);
      }
      continue;
    }
    const T* y = static_cast<const T*>(p.y) + base;
    const T* g = static_cast<const T*>(p.g) + (p.g ? (size_t)(b * p.sg) + t : 0);
    float my[VE], ry[VE], r1[VE], r0[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) my[k] = r1[k] = r0[k] = 0.f;
    if (LAYER) load_n<float, VE>(p.stats + at, nv, my);
    load_n<float, VE>(p.stats + (LAYER ? plane : 0) + at, nv, ry);
    for (int h = rs; h < H; h += NR) {
      const float wp = p.w_post[h], sc = p.scale[h];
      float tv[VE], yv[VE], gv[VE], dgv[VE];
      stream(h, tv);
      load_n<T, VE>(y + (size_t)h * p.L, nv, yv);
      if (p.g) load_n<T, VE>(g + (size_t)h * p.L, nv, gv);
      float sv = 0.f;
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        float rest, silu = 1.f, dsilu = 0.f;
        if (p.g) {
          const float s = sigmoid_pair(gv[k], &rest);
          silu = gv[k] * s;
          dsilu = s * fmaf(gv[k], rest, 1.f);
        }
        const float yh = (yv[k] - my[k]) * ry[k];  // past the end the factor is 0
        const float ty = tv[k] * yh;
        sv = fmaf(ty, silu, sv);
        dgv[k] = ty * (wp * sc) * dsilu;
        const float R = tv[k] * (sc * wp) * silu;
        r1[k] = fmaf(R, yh, r1[k]);
        if (LAYER) r0[k] += R;
      }
      store_n<T, VE>(static_cast<T*>(p.dx) + base + (size_t)h * p.L, ns, tv);
      if (p.dg)
        store_n<T, VE>(static_cast<T*>(p.dg) + (size_t)(b * p.sdg) + t + (size_t)h * p.L, ns, dgv);
      sv = lanes_sum<LT>(sv);
      if (lt == 0) {
        sums[h] = fmaf(sv, sc, sums[h]);
        sums[H + h] = fmaf(sv, wp, sums[H + h]);
      }
    }
    strip_sum<NT, LT, VE>(r1, buf);
    if (LAYER) strip_sum<NT, LT, VE>(r0, buf);
    for (int h = rs; h < H; h += NR) {
      const float c = p.w_post[h] * p.scale[h];
      float tv[VE], yv[VE], gv[VE], out[VE];
      stream(h, tv);
      load_n<T, VE>(y + (size_t)h * p.L, nv, yv);
      if (p.g) load_n<T, VE>(g + (size_t)h * p.L, nv, gv);
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        float rest;
        const float silu = p.g ? gv[k] * sigmoid_pair(gv[k], &rest) : 1.f;
        const float yh = (yv[k] - my[k]) * ry[k];
        float q = fmaf(tv[k] * c, silu, -yh * (r1[k] * inv_h));
        if (LAYER) q -= r0[k] * inv_h;
        out[k] = ry[k] * q;
      }
      store_n<T, VE>(static_cast<T*>(p.dy) + base + (size_t)h * p.L, ns, out);
    }
  }
  float* part = p.part + (size_t)blockIdx.x * 3 * H;
  for (int h = rs; h < H; h += NR)
    if (lt == 0) {
      part[h] = sums[h];
      part[H + h] = sums[H + h];
      part[2 * H + h] = sums[2 * H + h];
    }
}

// The workgroups' sums, in order and in float64: 16 channels by 16 slices of
// the workgroups to a block.
__global__ __launch_bounds__(256) void resnorm_sum_kernel(const float* __restrict__ part, int G,
                                                          int n, int H, float* dw_post,
                                                          float* dscale, float* dw_pre) {
  __shared__ double s[16][17];
  const int c = threadIdx.x & 15, z = threadIdx.x >> 4;
  const int k = blockIdx.x * 16 + c;
  double v = 0.0;
  if (k < n)
    for (int w = z; w < G; w += 16) v += (double)part[(size_t)w * n + k];
  s[z][c] = v;
  __syncthreads();
  if (z == 0 && k < n) {
    double t = 0.0;
#pragma unroll
    for (int j = 0; j < 16; ++j) t += s[j][c];
    float* out = k < H ? dw_post : k < 2 * H ? dscale : dw_pre;
    if (out) out[k % H] = (float)t;
  }
}

constexpr int kMaxGroups = 512;  // workgroups of the backward pass

// Steps to a lane, lanes to a row segment: 128 bytes of each row at a time
// while the forward pass holds the strip's H channels in registers, shorter
// segments for more channels; a single step takes its channels side by side.
struct Strip {
  int lt, ve;
};

Strip strip_of(int H, int L, int dtype) {
  if (L == 1) return {1, 1};
  const int ve = dtype == 0 ? 4 : 8;
  return {H <= 1024 ? 8 : H <= 2048 ? 4 : H <= 4096 ? 2 : 1, ve};
}

int strips(const Strip& s, int L) { return (L + s.lt * s.ve - 1) / (s.lt * s.ve); }

int groups_of(int B, int H, int L, int dtype) {
  return (int)std::min<long>((long)B * strips(strip_of(H, L, dtype), L), kMaxGroups);
}

template <typename T, bool LAYER, int NT, int LT, int VE, int KH>
void fwd_start(const Args& a, hipStream_t st) {
  hipLaunchKernelGGL((resnorm_fwd_kernel<T, LAYER, NT, LT, VE, KH>),
                     dim3((unsigned)(a.B * a.ntile)), dim3(NT), 0, st, a);
}

template <typename T, bool LAYER, int LT, int VE>
void bwd_start(const Args& a, int groups, hipStream_t st) {
  hipLaunchKernelGGL((resnorm_bwd_kernel<T, LAYER, 512, LT, VE>), dim3((unsigned)groups),
                     dim3(512), 0, st, a);
}

template <typename T, bool LAYER>
hipError_t run(const ResnormCall& c, int dtype, bool backward, hipStream_t st) {
  constexpr int VE = 16 / sizeof(T);
  const Strip s = strip_of(c.H, c.L, dtype);
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
  a.ntile = strips(s, c.L);
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
    if (s.ve == 1)
      c.H <= 2048 ? fwd_start<T, LAYER, 256, 1, 1, 8>(a, st)
                  : fwd_start<T, LAYER, 1024, 1, 1, 8>(a, st);
    else if (s.lt == 8)
      c.H <= 128   ? fwd_start<T, LAYER, 256, 8, VE, 4>(a, st)
      : c.H <= 512 ? fwd_start<T, LAYER, 512, 8, VE, 8>(a, st)
                   : fwd_start<T, LAYER, 1024, 8, VE, 8>(a, st);
    else
      s.lt == 4   ? fwd_start<T, LAYER, 1024, 4, VE, 8>(a, st)
      : s.lt == 2 ? fwd_start<T, LAYER, 1024, 2, VE, 8>(a, st)
                  : fwd_start<T, LAYER, 1024, 1, VE, 8>(a, st);
    return hipGetLastError();
  }
  const int groups = groups_of(c.B, c.H, c.L, dtype);
  if (s.ve == 1) bwd_start<T, LAYER, 1, 1>(a, groups, st);
  else if (s.lt == 8) bwd_start<T, LAYER, 8, VE>(a, groups, st);
  else if (s.lt == 4) bwd_start<T, LAYER, 4, VE>(a, groups, st);
  else if (s.lt == 2) bwd_start<T, LAYER, 2, VE>(a, groups, st);
  else bwd_start<T, LAYER, 1, VE>(a, groups, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int n = 3 * c.H;
  hipLaunchKernelGGL(resnorm_sum_kernel, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, st, a.part,
                     groups, n, c.H, c.dw_post, c.dscale, c.dw_pre);
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
  return align_up((size_t)groups_of(B, H, L, dtype) * 3 * H * sizeof(float), 256);
}

hipError_t launch_resnorm_forward(const ResnormCall& c, int dtype, hipStream_t st) {
  return run_type(c, dtype, false, st);
}

// B = 0 or L = 0: no strips, so the sums are zero.
hipError_t launch_resnorm_backward(const ResnormCall& c, int dtype, hipStream_t st) {
  if (c.B == 0 || c.L == 0) {
    const int n = 3 * c.H;
    hipLaunchKernelGGL(resnorm_sum_kernel, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, st,
                       static_cast<const float*>(nullptr), 0, n, c.H, c.dw_post, c.dscale,
                       c.dw_pre);
    return hipGetLastError();
  }
  return run_type(c, dtype, true, st);
}

}  // namespace dssm
