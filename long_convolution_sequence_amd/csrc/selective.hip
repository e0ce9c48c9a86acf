// The selective scan: per channel h a bank of N real modes (as the DLR's, with
// no phase) whose step size, drive and read-out come with every step,
//
//   dt_t = softplus(delta_t + dt_bias[h]),  a_t = exp(-log_re[h,n]^2 dt_t),
//   x_t = a_t x_{t-1} + dt_t B_t[g,n] u_t,  y_t = (sum_n C_t[g,n] x_t + D[h] u_t) silu(z_t),
//
// g the group of the channel, and its gradients.  With p_t = dy_t silu(z_t) and
// G_t = C_t p_t + a_{t+1} G_{t+1} (the state's gradient), w_t = G_t a_t x_{t-1}:
//
//   q = sum_n G B,  du = dt q + D p,  d(dt) = u q - sum_n log_re^2 w,
//   ddelta = d(dt) sigmoid(delta + dt_bias),  dB = sum_h G dt u,  dC = sum_h p x,
//   dlog_re = -2 log_re sum_{b,t} w dt,  dD = sum p u,  ddt_bias = sum ddelta,
//   dz = dy (sum_n C x + D u) silu'(z),  dx0 = a_0 G_0.
//
// Layout.  A row (b, h) takes 16 lanes, ST consecutive steps each; a wave four
// rows.  16 lanes are what the data-parallel primitives shift and rotate
// within, so that joining the lanes of a mode costs about one vector operation
// per step where a lane holds 16 steps; the modes are walked one by one, a
// lane's decays and drives of a mode in registers.  B and C are the same for
// all rows of a group: the workgroup's tile of them lies in LDS as float32.
//
// What bounds it is the vector unit: a product for the exponent, the
// exponential (its own rate a quarter), the drive, two passes of the
// recurrence (one to join the lanes, one from the joined state) and the
// read-out, about 6 operations and an exponential per mode and step.
#include <algorithm>
#include <type_traits>

#include "dssm_internal.h"
#include "seq_common.h"
#include "strip.h"

namespace dssm {
namespace {

constexpr int kSeg = 16;  // lanes of a row
constexpr int kKeep = 128; // steps between two kept states
constexpr int kModes = 8; // modes whose B and C are in LDS at once
constexpr int kPair = 2;  // modes a wave walks side by side
constexpr int kRowShl = 0x100, kRowRor = 0x120;

struct Args {
  const void *u, *delta, *z, *Bm, *Cm;
  long long su, sd, sz, sB, sC;  // elements between batch rows
  const float *log_re, *D, *dt_bias;
  const int* lens;
  int B, H, G, N, L, HG;  // HG = H / G
  const float* x0;
  float* xT;
  void* y;
  float* bounds;          // [rows][chunks][N] state entering each chunk
  int nchunk;
  // a row's tiles in nseg segments of seg_tiles
  int nrb, nseg, seg_tiles;
  float* agg;             // [rows][nseg][N]: ends of the segments, then what enters them
  float* aggS;            // [rows][nseg]: sum of dt
  // backward
  const void* dy;
  const float* dx;
  void *du, *ddelta, *dz, *dB, *dC;
  long long sdu, sdd, sdz, sdB, sdC;
  float *dlog_re, *dD, *ddt_bias, *dx0;
  float* part_bc;         // [nrb][B][G][2][N][nchunk kKeep]
  float* part_n;          // [rows][nseg][N]
  float* part_h;          // [rows][nseg][2]
};

// Inclusive scan over a row's 16 lanes, in time order or (REV) against it, of
// x -> P x + V, and what each lane's neighbour leaves (0 at the first lane).  A
// lane without a neighbour joins 0; its P, 0 from there on, meets no further
// neighbour.  In assembly, as the compiler moves a lane's value first and adds
// it in an instruction of its own.  A lane's value is read two wait states after
// it is written at the earliest.
#define DSSM_ROW(dir, n) "row_sh" dir ":" n " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"
#define DSSM_SCAN1(dir)                                                   \
  "s_nop 1\n\t"                                                          \
  "v_fmac_f32_dpp %0, %0, %1 " DSSM_ROW(dir, "1")                         \
  "v_mul_f32_dpp %1, %1, %1 " DSSM_ROW(dir, "1") "s_nop 0\n\t"           \
  "v_fmac_f32_dpp %0, %0, %1 " DSSM_ROW(dir, "2")                         \
  "v_mul_f32_dpp %1, %1, %1 " DSSM_ROW(dir, "2") "s_nop 0\n\t"           \
  "v_fmac_f32_dpp %0, %0, %1 " DSSM_ROW(dir, "4")                         \
  "v_mul_f32_dpp %1, %1, %1 " DSSM_ROW(dir, "4") "s_nop 0\n\t"           \
  "v_fmac_f32_dpp %0, %0, %1 " DSSM_ROW(dir, "8") "s_nop 1\n\t"          \
  "v_mov_b32_dpp %2, %0 " DSSM_ROW(dir, "1")
#define DSSM_SCAN2(dir)                                                   \
  "s_nop 1\n\t"                                                          \
  "v_fmac_f32_dpp %0, %0, %2 " DSSM_ROW(dir, "1")                         \
  "v_fmac_f32_dpp %1, %1, %3 " DSSM_ROW(dir, "1")                         \
  "v_mul_f32_dpp %2, %2, %2 " DSSM_ROW(dir, "1")                          \
  "v_mul_f32_dpp %3, %3, %3 " DSSM_ROW(dir, "1")                          \
  "v_fmac_f32_dpp %0, %0, %2 " DSSM_ROW(dir, "2")                         \
  "v_fmac_f32_dpp %1, %1, %3 " DSSM_ROW(dir, "2")                         \
  "v_mul_f32_dpp %2, %2, %2 " DSSM_ROW(dir, "2")                          \
  "v_mul_f32_dpp %3, %3, %3 " DSSM_ROW(dir, "2")                          \
  "v_fmac_f32_dpp %0, %0, %2 " DSSM_ROW(dir, "4")                         \
  "v_fmac_f32_dpp %1, %1, %3 " DSSM_ROW(dir, "4")                         \
  "v_mul_f32_dpp %2, %2, %2 " DSSM_ROW(dir, "4")                          \
  "v_mul_f32_dpp %3, %3, %3 " DSSM_ROW(dir, "4")                          \
  "v_fmac_f32_dpp %0, %0, %2 " DSSM_ROW(dir, "8")                         \
  "v_fmac_f32_dpp %1, %1, %3 " DSSM_ROW(dir, "8") "s_nop 0\n\t"          \
  "v_mov_b32_dpp %4, %0 " DSSM_ROW(dir, "1")                              \
  "v_mov_b32_dpp %5, %1 " DSSM_ROW(dir, "1")

template <bool REV>
__device__ __forceinline__ void row_scan(float (&P)[1], float (&V)[1], float (&in)[1]) {
  if (REV)
    asm(DSSM_SCAN1("l") : "+v"(V[0]), "+v"(P[0]), "=&v"(in[0]));
  else
    asm(DSSM_SCAN1("r") : "+v"(V[0]), "+v"(P[0]), "=&v"(in[0]));
}
template <bool REV>
__device__ __forceinline__ void row_scan(float (&P)[2], float (&V)[2], float (&in)[2]) {
  if (REV)
    asm(DSSM_SCAN2("l")
        : "+v"(V[0]), "+v"(V[1]), "+v"(P[0]), "+v"(P[1]), "=&v"(in[0]), "=&v"(in[1]));
  else
    asm(DSSM_SCAN2("r")
        : "+v"(V[0]), "+v"(V[1]), "+v"(P[0]), "+v"(P[1]), "=&v"(in[0]), "=&v"(in[1]));
}

// x summed over a row's 16 lanes; all of them get the sum.
__device__ __forceinline__ float row_total(float x) {
  x += row_move<kRowRor + 8>(x);
  x += row_move<kRowRor + 4>(x);
  x += row_move<kRowRor + 2>(x);
  x += row_move<kRowRor + 1>(x);
  return x;
}

// log(1 + exp(v)), NaN passing: max(v, 0) + log1p(t), t = exp(-|v|), log1p(t) / t
// on [0, 1] the polynomial of least relative error (3e-8; 2e-7 with its
// roundings).  Steps of 1e-3 and less are what the map is used with: log2(1 + t)
// would keep ten bits of them, and this takes half the operations of the series
// of t / (2 + t).
__device__ __forceinline__ float softplus(float v) {
  const float t = exp2_fast(-kLog2e * fabsf(v));
  float r = 0.005232690833508968f;
  r = fmaf(r, t, -0.029505228623747826f);
  r = fmaf(r, t, 0.07822594791650772f);
  r = fmaf(r, t, -0.13663245737552643f);
  r = fmaf(r, t, 0.19106008112430573f);
  r = fmaf(r, t, -0.2484298199415207f);
  r = fmaf(r, t, 0.3331909775733948f);
  r = fmaf(r, t, -0.4999949336051941f);
  r = fmaf(r, t, 0.9999999403953552f);
  return fmaf(r, t, fmaxf(v, 0.f));
}

// log_re^2, finite with its product by log2(e) unless NaN: a step of length
// zero has to decay nothing.
__device__ __forceinline__ float square_of(float log_re) {
  const float s = log_re * log_re;
  return s > 0x1p126f ? 0x1p126f : s;
}

__device__ __forceinline__ int row_len(const Args& p, int b) {
  if (!p.lens) return p.L;
  return min(max(p.lens[b], 0), p.L);
}

// Where steps 4 j .. 4 j + 3 of lane `seg` lie in a tile of LDS, in floats: the
// 16 lanes read 16 bytes each from all banks.
template <int ST>
__device__ __forceinline__ int slot(int seg, int j) {
  if (ST == 8) return seg * 8 + 4 * (j ^ (seg >> 3));
  return seg * 4;
}

template <int ST>
__device__ __forceinline__ void read_steps(const float* tile, int seg, float* out) {
#pragma unroll
  for (int j = 0; j < ST / 4; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(tile + slot<ST>(seg, j));
    out[4 * j] = v.x;
    out[4 * j + 1] = v.y;
    out[4 * j + 2] = v.z;
    out[4 * j + 3] = v.w;
  }
}

// Eight steps from t (a multiple of 8, in the tile) to where they are read.
template <int ST>
__device__ __forceinline__ void write_steps(float* tile, int t, const float* v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int q = t / 4 + k;
    float* to = tile + slot<ST>(q / (ST / 4), q % (ST / 4));
    *reinterpret_cast<float4*>(to) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  }
}

// Which batch row, group, row block and segment a workgroup works on.
struct Place {
  int b, g, rb, seg;
  __device__ __forceinline__ Place(const Args& p) {
    unsigned k = blockIdx.x;
    seg = (int)(k % (unsigned)p.nseg);
    k /= (unsigned)p.nseg;
    rb = (int)(k % (unsigned)p.nrb);
    k /= (unsigned)p.nrb;
    g = (int)(k % (unsigned)p.G);
    b = (int)(k / (unsigned)p.G);
  }
};

// A lane number the compiler knows nothing of: addresses derived from it are
// formed where they are used instead of being kept in registers through a loop.
__device__ __forceinline__ int opaque(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// An address the workgroup shares (in scalar registers) plus a lane's own 32 bits
// of bytes: 32 rows of 2^24 steps of 4 bytes.
// The lane's part is made opaque: as loop-invariant sums the compiler would keep
// every tensor's whole address in vector registers.
template <typename T>
__device__ __forceinline__ T* spot(T* shared, uint32_t bytes) {
  return reinterpret_cast<T*>(
      reinterpret_cast<char*>(const_cast<typename std::remove_const<T>::type*>(shared)) +
      (uint32_t)opaque((int)bytes));
}

// The group's B and C over one tile and kModes modes, on their way to LDS.
template <typename T, int NT, int TILE, bool BOTH>
struct Stage {
  static constexpr int kChunks = (BOTH ? 2 : 1) * kModes * (TILE / 8);
  static constexpr int IT = (kChunks + NT - 1) / NT;
  Packed<T, 8> v[IT];
  // modes n0 .. of the tile from t0; steps at or past len are 0
  __device__ __forceinline__ void fetch(const T* Bm, const T* Cm, int N, int L, int n0, int t0,
                                        int len) {
    const size_t first = (size_t)n0 * L + t0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = opaque((int)threadIdx.x) + i * NT;
      const int t = (k % (TILE / 8)) * 8, n = k / (TILE / 8) % kModes;
      const bool second = BOTH && k >= kChunks / 2;
      const int nv = (IT * NT == kChunks || k < kChunks) && n0 + n < N ? len - t0 - t : 0;
      const T* from = spot((second ? Cm : Bm) + first, (uint32_t)(n * L + t) * sizeof(T));
      if (nv >= 8)
        v[i].load(from);
      else
        v[i].load(from, max(nv, 0), (T)0.f);
    }
  }
  __device__ __forceinline__ void put(float (*to)[kModes][TILE]) const {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = opaque((int)threadIdx.x) + i * NT;
      if (IT * NT != kChunks && k >= kChunks) break;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = v[i][j];
      write_steps<TILE / kSeg>(to[BOTH && k >= kChunks / 2 ? 1 : 0][k / (TILE / 8) % kModes],
                               k % (TILE / 8) * 8, f);
    }
  }
};

// A lane's steps of one row as they lie in memory; row0: the workgroup's first
// row at the tile's first step.
template <typename T, int SP>
struct Lane {
  Packed<T, SP> v;
  __device__ __forceinline__ void fetch(const T* row0, uint32_t own, int nv) {
    if (nv >= SP)
      v.load(spot(row0, own));
    else
      v.load(spot(row0, own), max(nv, 0), (T)0.f);
  }
};

__host__ __device__ inline int padded(int N) { return (N + kModes - 1) / kModes * kModes; }

// The states entering a lane's first step, of M modes side by side.  a: decays,
// b: drives, P: decay over the lane's steps; carry: in a row's first lane the
// state entering the tile, in the others 0.  end: in its last lane the state
// after the tile.
template <int ST, int M>
__device__ __forceinline__ void enter_forward(const float (&a)[M][ST], const float (&b)[M][ST],
                                              float (&P)[M], const float (&carry)[M],
                                              float (&x)[M], float (&end)[M]) {
#pragma unroll
  for (int i = 0; i < M; ++i) end[i] = b[i][0];
#pragma unroll
  for (int j = 1; j < ST; ++j)
#pragma unroll
    for (int i = 0; i < M; ++i) end[i] = fmaf(a[i][j], end[i], b[i][j]);
#pragma unroll
  for (int i = 0; i < M; ++i) end[i] = fmaf(P[i], carry[i], end[i]);
  row_scan<false>(P, end, x);
#pragma unroll
  for (int i = 0; i < M; ++i) x[i] += carry[i];
}

// A workgroup's values of every row and mode, in LDS: a row's first (or last)
// lane has the value, the others find zeros to read and a place to write that
// nobody reads, at the same distances: no branch and no address per mode.
// pitch: modes, rounded up to what the waves take at once.
struct Cells {
  float* at;  // [R][pitch], then pitch zeros, then pitch spare
  int R, pitch;
  __device__ __forceinline__ float* row(int r) const { return at + r * pitch; }
  __device__ __forceinline__ float* from(int r, bool mine) const { return row(mine ? r : R); }
  __device__ __forceinline__ float* to(int r, bool mine) const { return row(mine ? r : R + 1); }
};

// Forward over a row or a segment of it.  RW groups of four rows, the modes of
// each shared out among NW waves: with NW > 1 every wave forms a part of the
// lanes' step sizes, and of their outputs.  AGG: only the segment's ends.
template <typename T, int ST, int RW, int NW, bool AGG>
__global__ __launch_bounds__(64 * RW * NW) __attribute__((amdgpu_waves_per_eu(4)))
void selective_fwd_kernel(Args p) {
  constexpr int NT = 64 * RW * NW, R = 4 * RW, TILE = kSeg * ST, SP = ST / NW;
  constexpr int QS = ST / 4, QP = SP / 4;  // a lane's, and its own part's, groups of four steps
  static_assert(SP % 4 == 0, "the waves of a row exchange 16 bytes a lane");
  __shared__ float bc[2][AGG ? 1 : 2][kModes][TILE];
  __shared__ float4 xch[NW > 1 ? RW : 1][2][NW > 1 ? QS : 1][NW > 1 ? 64 : 1];
  constexpr bool kJoinY = NW > 1 && !AGG;
  __shared__ float4 yred[kJoinY ? RW * NW : 1][kJoinY ? QS : 1][kJoinY ? 64 : 1];
  extern __shared__ float dyn[];
  const int NP = padded(p.N);
  const Cells kap{dyn, R, NP}, car{dyn + R * NP, R, NP};  // log_re^2; the state entering the tile
  const Place at(p);
  if (AGG && at.seg == p.nseg - 1) return;  // nobody joins the last segment
  const int lane = threadIdx.x & 63, seg = lane & (kSeg - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = wave / NW, nw = wave % NW;
  const int r = rg * 4 + lane / kSeg;  // the lane's row in the workgroup
  const bool live = at.rb * R + r < p.HG, first = seg == 0;
  const int h = at.g * p.HG + min(at.rb * R + r, p.HG - 1);
  const int len = row_len(p, at.b);
  const int ntile = (p.L + TILE - 1) / TILE;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  const int t_live = min(t_hi, (len + TILE - 1) / TILE);
  const size_t row0 = (size_t)at.b * p.H + at.g * p.HG + at.rb * R;  // the workgroup's first row
  const int nrow = min(R, p.HG - at.rb * R);
  // the waves of a row group take turns with its modes
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int q = rg * 4 + k;
    for (int n = lane * NW + nw; n < NP; n += 64 * NW) {
      float c = 0.f, s = 0.f;
      if (q < nrow && n < p.N) {
        s = square_of(p.log_re[(size_t)(row0 - (size_t)at.b * p.H + q) * p.N + n]) * kLog2e;
        if (!AGG && p.nseg > 1)
          c = p.agg[((row0 + q) * p.nseg + at.seg) * p.N + n];
        else if (!AGG && p.x0)
          c = p.x0[(row0 + q) * p.N + n];
      }
      kap.row(q)[n] = s;
      car.row(q)[n] = c;
    }
  }
  for (int n = threadIdx.x; n < NP; n += NT) car.row(R)[n] = 0.f;  // before the first barrier
  const float* krow = kap.row(r) + nw;
  const float* from = car.from(r, first) + nw;
  float* to = car.to(r, seg == kSeg - 1) + nw;
  const size_t first_row = (size_t)(at.g * p.HG + at.rb * R) * p.L;
  const T* u = static_cast<const T*>(p.u) + (size_t)(at.b * p.su) + first_row;
  const T* delta = static_cast<const T*>(p.delta) + (size_t)(at.b * p.sd) + first_row;
  const T* z = static_cast<const T*>(p.z) + (p.z ? (size_t)(at.b * p.sz) + first_row : 0);
  const T* Bm = static_cast<const T*>(p.Bm) + (size_t)(at.b * p.sB) + (size_t)at.g * p.N * p.L;
  const T* Cm = static_cast<const T*>(p.Cm) + (size_t)(at.b * p.sC) + (size_t)at.g * p.N * p.L;
  T* out = static_cast<T*>(p.y) + row0 * p.L;
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  const float D = !AGG && p.D ? p.D[h] : 0.f;
  const int nblk = (p.N + kModes - 1) / kModes;
  const int off = seg * ST + nw * SP;  // the lane's own part of a tile
  const uint32_t mine = ((uint32_t)min(r, nrow - 1) * (uint32_t)p.L + off) * (uint32_t)sizeof(T);
  Stage<T, NT, TILE, !AGG> stage;
  Lane<T, SP> un, dn;
  if (t_lo < t_live) {
    const int t = t_lo * TILE;
    stage.fetch(Bm, Cm, p.N, p.L, 0, t, len);
    dn.fetch(delta + t, mine, len - t - off);
    un.fetch(u + t, mine, len - t - off);
  }
  float Sseg = 0.f;
  int buf = 0;
  for (int tile = t_lo; tile < t_live; ++tile) {
    const int t0 = tile * TILE, nv = len - t0 - off, ln = opaque(lane);
    // the states entering a chunk, for the backward pass
    if (!AGG && p.bounds && (t0 & (kKeep - 1)) == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = rg * 4 + k;
        if (q < nrow)
          for (int n = ln * NW + nw; n < p.N; n += 64 * NW)
            p.bounds[((row0 + q) * p.nchunk + t0 / kKeep) * p.N + n] = car.row(q)[n];
      }
    }
    Lane<T, SP> zc;
    float dt[ST], du[ST], y[ST], skip[SP];
    {
      float own[2][SP];
#pragma unroll
      for (int j = 0; j < SP; ++j) {
        own[0][j] = softplus(dn.v[j] + bias);
        own[1][j] = own[0][j] * un.v[j];
        skip[j] = D * un.v[j];
      }
      if (t0 + TILE > len) {
#pragma unroll
        for (int j = 0; j < SP; ++j) {
          own[0][j] = j < nv ? own[0][j] : 0.f;
          own[1][j] = j < nv ? own[1][j] : 0.f;
        }
      }
      if constexpr (NW == 1) {
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          dt[j] = own[0][j];
          du[j] = own[1][j];
          y[j] = skip[j];
        }
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < QP; ++i)
            xch[rg][m][nw * QP + i][ln] = make_float4(own[m][4 * i], own[m][4 * i + 1],
                                                        own[m][4 * i + 2], own[m][4 * i + 3]);
#pragma unroll
        for (int j = 0; j < ST; ++j) y[j] = 0.f;
      }
    }
    // the gate is read for this tile's end, the rest for the next tile
    if (!AGG && p.z) zc.fetch(z + t0, mine, nv);
    if (tile + 1 < t_live) {
      const int t = t0 + TILE;
      dn.fetch(delta + t, mine, len - t - off);
      un.fetch(u + t, mine, len - t - off);
    }
    float S = 0.f;
    for (int blk = 0; blk < nblk; ++blk) {
      stage.put(bc[buf]);
      // one barrier a stage: the buffers alternate, and a wave past this one
      // has read the other
      __syncthreads();
      if (blk + 1 < nblk)
        stage.fetch(Bm, Cm, p.N, p.L, (blk + 1) * kModes, t0, len);
      else if (tile + 1 < t_live)
        stage.fetch(Bm, Cm, p.N, p.L, 0, t0 + TILE, len);
      if (blk == 0) {
        if constexpr (NW > 1) {
#pragma unroll
          for (int k = 0; k < QS; ++k) {
            const float4 a = xch[rg][0][k][ln], b = xch[rg][1][k][ln];
            const float va[4] = {a.x, a.y, a.z, a.w}, vb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              dt[4 * k + j] = va[j];
              du[4 * k + j] = vb[j];
            }
          }
        }
#pragma unroll
        for (int j = 0; j < ST; ++j) S += dt[j];
        if (AGG) Sseg += S;
      }
      const int n0 = blk * kModes, nm = p.N - n0;
      // two modes at a time: the passes are chains, and two fill each other's
      // waits.  Modes past the last one are zeros.
      const auto walk = [&](auto step) {
        constexpr int M = kPair, m0 = decltype(step)::value * M * NW;
        __builtin_amdgcn_sched_barrier(0);  // steps mixed together would not fit the registers
        float P[M], carry[M], x[M], end[M], v[M][ST], a[M][ST], b[M][ST];
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const float k = krow[n0 + m0 + i * NW];
          carry[i] = from[n0 + m0 + i * NW];
          read_steps<ST>(bc[buf][0][m0 + i * NW + nw], seg, b[i]);
#pragma unroll
          for (int j = 0; j < ST; ++j) {
            a[i][j] = exp2_fast(-k * dt[j]);
            b[i][j] *= du[j];
          }
          P[i] = exp2_fast(-k * S);
        }
        enter_forward<ST, M>(a, b, P, carry, x, end);
#pragma unroll
        for (int i = 0; i < M; ++i) to[n0 + m0 + i * NW] = end[i];
        if (AGG) return;
#pragma unroll
        for (int i = 0; i < M; ++i) read_steps<ST>(bc[buf][AGG ? 0 : 1][m0 + i * NW + nw], seg, v[i]);
#pragma unroll
        for (int j = 0; j < ST; ++j)
#pragma unroll
          for (int i = 0; i < M; ++i) {
            x[i] = fmaf(a[i][j], x[i], b[i][j]);
            y[j] = fmaf(v[i][j], x[i], y[j]);
          }
      };
      walk(std::integral_constant<int, 0>());
      if (nm > kPair * NW) walk(std::integral_constant<int, 1>());
      if constexpr (kModes > 2 * kPair * NW) {
        if (nm > 2 * kPair * NW) walk(std::integral_constant<int, 2>());
        if (nm > 3 * kPair * NW) walk(std::integral_constant<int, 3>());
      }
      buf ^= 1;
    }
    if constexpr (AGG) {
      if (NW > 1) __syncthreads();  // before the next tile's step sizes take this one's place
    } else {
      float own[SP];
      if constexpr (kJoinY) {
        // the next tile's first barrier keeps these from being overwritten too early
#pragma unroll
        for (int k = 0; k < QS; ++k)
          yred[wave][k][ln] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < SP; ++j) own[j] = skip[j];
#pragma unroll
        for (int k = 0; k < NW; ++k)
#pragma unroll
          for (int i = 0; i < QP; ++i) {
            const float4 a = yred[rg * NW + k][nw * QP + i][ln];
            own[4 * i] += a.x;
            own[4 * i + 1] += a.y;
            own[4 * i + 2] += a.z;
            own[4 * i + 3] += a.w;
          }
      } else {
#pragma unroll
        for (int j = 0; j < SP; ++j) own[j] = y[j];
      }
#pragma unroll
      for (int j = 0; j < SP; ++j) {
        float rest;
        if (p.z) own[j] *= zc.v[j] * sigmoid_pair(zc.v[j], &rest);
      }
      if (t0 + TILE > len) {
#pragma unroll
        for (int j = 0; j < SP; ++j) own[j] = j < nv ? own[j] : 0.f;
      }
      if (live) store_n<T, SP>(spot(out + t0, mine), p.L - t0 - off, own);
    }
  }
  if (AGG) {
    const float s = row_total(Sseg);
    if (live && first && nw == 0) p.aggS[(row0 + r) * p.nseg + at.seg] = s;
  } else {
    // behind the rows' end: outputs are 0, the states stay
    for (int tile = max(t_lo, t_live); tile < t_hi; ++tile) {
      const int t0 = tile * TILE;
      float zero[SP];
#pragma unroll
      for (int j = 0; j < SP; ++j) zero[j] = 0.f;
      if (live) store_n<T, SP>(spot(out + t0, mine), p.L - t0 - off, zero);
    }
  }
  // what leaves: the state after the row, or the segment's own part of it
  float* out_x = AGG ? p.agg + (size_t)at.seg * p.N : at.seg == p.nseg - 1 ? p.xT : nullptr;
  if (out_x) {
    const size_t pitch = (size_t)(AGG ? p.nseg : 1) * p.N;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int q = rg * 4 + k;
      if (q < nrow)
        for (int n = lane * NW + nw; n < p.N; n += 64 * NW)
          out_x[(row0 + q) * pitch + n] = car.row(q)[n];
    }
  }
}

// What enters each segment of a split row: the segments' ends joined in order,
// a mode to a thread (REV: from the last to the first, `start` being the
// gradient of the state after the row).
template <bool REV>
__global__ __launch_bounds__(256) void selective_join_kernel(float* agg, const float* aggS,
                                                             const float* log_re,
                                                             const float* start, long rows, int H,
                                                             int N, int nseg) {
  const long k = (long)blockIdx.x * 256 + threadIdx.x;
  if (k >= rows * N) return;
  const long row = k / N;
  const int n = (int)(k - row * N);
  const float kap = square_of(log_re[(row % H) * N + n]) * kLog2e;
  float c = start ? start[k] : 0.f;
  float* v = agg + row * nseg * N + n;
  const float* s = aggS + row * nseg;
  for (int j = 0; j < nseg; ++j) {
    const int i = REV ? nseg - 1 - j : j;
    const float e = v[(size_t)i * N];
    v[(size_t)i * N] = c;
    if (j + 1 < nseg) c = fmaf(exp2_fast(-kap * s[i]), c, e);
  }
}

// Four lanes' rows added up: quads v[m], v[4 + m], v[8 + m], v[12 + m] over the
// wave's four rows, row k of lanes getting the sum of v[4 k + m].
__device__ __forceinline__ void swap_halves(float& a, float& b) {
  const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  a = __uint_as_float(t[0]);
  b = __uint_as_float(t[1]);
}
__device__ __forceinline__ void swap_rows(float& a, float& b) {
  const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  a = __uint_as_float(t[0]);
  b = __uint_as_float(t[1]);
}
// v0, v2 to the halves, v1, v3 likewise; then rows: lanes of row k get the sum of vk.
__device__ __forceinline__ float rows_quad(float v0, float v1, float v2, float v3) {
  swap_halves(v0, v2);
  swap_halves(v1, v3);
  float a = v0 + v2, b = v1 + v3;
  swap_rows(a, b);
  return a + b;
}

// A segment's part of the state gradient entering it from the right, and the
// sum of its step sizes.
template <typename T, int ST, int RW>
__global__ __launch_bounds__(64 * RW) void selective_bwd_agg_kernel(Args p) {
  constexpr int NT = 64 * RW, R = 4 * RW, RP = R + 1, TILE = kSeg * ST;
  __shared__ float bc[2][1][kModes][TILE];
  extern __shared__ float dyn[];
  float* kap = dyn;
  float* car = dyn + p.N * RP;
  const Place at(p);
  if (at.seg == 0) return;  // nobody joins the first segment
  const int lane = threadIdx.x & 63, seg = lane & (kSeg - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = wave * 4 + lane / kSeg;
  const bool live = at.rb * R + r < p.HG, last = seg == kSeg - 1;
  const int h = at.g * p.HG + min(at.rb * R + r, p.HG - 1);
  const int len = row_len(p, at.b);
  const int ntile = (p.L + TILE - 1) / TILE;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  const int t_live = min(t_hi, (len + TILE - 1) / TILE);
  const size_t row0 = (size_t)at.b * p.H + at.g * p.HG + at.rb * R;
  const int nrow = min(R, p.HG - at.rb * R);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int q = wave * 4 + k;
    for (int n = lane; n < p.N; n += 64) {
      kap[n * RP + q] =
          q < nrow
              ? square_of(p.log_re[(size_t)(row0 - (size_t)at.b * p.H + q) * p.N + n]) * kLog2e
              : 0.f;
      car[n * RP + q] = 0.f;
    }
  }
  const size_t first_row = (size_t)(at.g * p.HG + at.rb * R) * p.L;
  const T* delta = static_cast<const T*>(p.delta) + (size_t)(at.b * p.sd) + first_row;
  const T* z = static_cast<const T*>(p.z) + (p.z ? (size_t)(at.b * p.sz) + first_row : 0);
  const T* dy = static_cast<const T*>(p.dy) + row0 * p.L;
  const T* Cm = static_cast<const T*>(p.Cm) + (size_t)(at.b * p.sC) + (size_t)at.g * p.N * p.L;
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  const int nblk = (p.N + kModes - 1) / kModes;
  const int off = seg * ST;
  const uint32_t mine = ((uint32_t)min(r, nrow - 1) * (uint32_t)p.L + off) * (uint32_t)sizeof(T);
  Stage<T, NT, TILE, false> stage;
  if (t_lo < t_live) stage.fetch(Cm, Cm, p.N, p.L, 0, (t_live - 1) * TILE, len);
  float Sseg = 0.f;
  int buf = 0;
  for (int tile = t_live - 1; tile >= t_lo; --tile) {
    const int t0 = tile * TILE, nv = len - t0 - off;
    Lane<T, ST> dv, zv, gv;
    dv.fetch(delta + t0, mine, nv);
    gv.fetch(dy + t0, mine, nv);
    if (p.z) zv.fetch(z + t0, mine, nv);
    float dt[ST], gy[ST], S = 0.f;
#pragma unroll
    for (int j = 0; j < ST; ++j) {
      const float d = softplus(dv.v[j] + bias);
      float g = gv.v[j], rest;
      if (p.z) g *= zv.v[j] * sigmoid_pair(zv.v[j], &rest);
      dt[j] = j < nv ? d : 0.f;
      gy[j] = j < nv && live ? g : 0.f;
      S += dt[j];
    }
    Sseg += S;
    for (int blk = 0; blk < nblk; ++blk) {
      stage.put(bc[buf]);
      __syncthreads();
      if (blk + 1 < nblk)
        stage.fetch(Cm, Cm, p.N, p.L, (blk + 1) * kModes, t0, len);
      else if (tile > t_lo)
        stage.fetch(Cm, Cm, p.N, p.L, 0, t0 - TILE, len);
      const int n0 = blk * kModes, nm = min(kModes, p.N - n0);
      for (int m = 0; m < nm; ++m) {
        float* cell = car + (n0 + m) * RP + r;
        const float k = kap[(n0 + m) * RP + r], carry = *cell;
        float v[ST];
        read_steps<ST>(bc[buf][0][m], seg, v);
        float F = 0.f;
#pragma unroll
        for (int j = ST - 1; j >= 0; --j)
          F = exp2_fast(-k * dt[j]) * fmaf(v[j], gy[j], F);
        float P[1] = {exp2_fast(-k * S)}, V[1] = {fmaf(P[0], last ? carry : 0.f, F)}, in[1];
        row_scan<true>(P, V, in);
        if (seg == 0) *cell = V[0];
      }
      buf ^= 1;
    }
  }
  const float s = row_total(Sseg);
  if (live && seg == 0) p.aggS[(row0 + r) * p.nseg + at.seg] = s;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int q = wave * 4 + k;
    if (q < nrow)
      for (int n = lane; n < p.N; n += 64)
        p.agg[((row0 + q) * p.nseg + at.seg) * p.N + n] = car[n * RP + q];
  }
}

// Backward over a row or a segment of it, from its end: every tile's states are
// formed again from the kept one.  The sums over the group's rows (dB, dC) are
// added up over a wave's four rows in registers, over the workgroup's waves
// through LDS, two modes at a time, and left for the last kernel.
template <typename T, int ST, int RW, bool Z>
__global__ __launch_bounds__(64 * RW) void selective_bwd_kernel(Args p) {
  constexpr int NT = 64 * RW, R = 4 * RW, RP = R + 1, TILE = kSeg * ST, Q = ST / 4;
  typedef float Pair __attribute__((ext_vector_type(2)));
  typedef typename std::conditional<Q == 2, Pair, float>::type Part;  // Q steps
  __shared__ float bc[2][2][kModes][TILE];
  __shared__ Part slab[2][RW][2][2][64];
  extern __shared__ float dyn[];
  float* kap = dyn;                  // [N][RP]
  float* car = dyn + p.N * RP;       // [N][RP] state gradient entering the tile
  float* dre = dyn + 2 * p.N * RP;   // [N][RP] sum of w dt, and a spare word
  const Place at(p);
  const int lane = threadIdx.x & 63, seg = lane & (kSeg - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = wave * 4 + lane / kSeg;
  const bool live = at.rb * R + r < p.HG, first = seg == 0, last = seg == kSeg - 1;
  const int h = at.g * p.HG + min(at.rb * R + r, p.HG - 1);
  const int len = row_len(p, at.b);
  const int ntile = (p.L + TILE - 1) / TILE;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  const int t_live = min(t_hi, (len + TILE - 1) / TILE);
  const size_t row0 = (size_t)at.b * p.H + at.g * p.HG + at.rb * R;
  const int nrow = min(R, p.HG - at.rb * R);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int q = wave * 4 + k;
    for (int n = lane; n < p.N; n += 64) {
      float c = 0.f, s = 0.f;
      if (q < nrow) {
        s = square_of(p.log_re[(size_t)(row0 - (size_t)at.b * p.H + q) * p.N + n]) * kLog2e;
        if (p.nseg > 1)
          c = p.agg[((row0 + q) * p.nseg + at.seg) * p.N + n];
        else if (p.dx)
          c = p.dx[(row0 + q) * p.N + n];
      }
      kap[n * RP + q] = s;
      car[n * RP + q] = c;
      dre[n * RP + q] = 0.f;
    }
  }
  const size_t first_row = (size_t)(at.g * p.HG + at.rb * R) * p.L;
  const T* u = static_cast<const T*>(p.u) + (size_t)(at.b * p.su) + first_row;
  const T* delta = static_cast<const T*>(p.delta) + (size_t)(at.b * p.sd) + first_row;
  const T* z = static_cast<const T*>(p.z) + (Z ? (size_t)(at.b * p.sz) + first_row : 0);
  const T* dy = static_cast<const T*>(p.dy) + row0 * p.L;
  T* du = static_cast<T*>(p.du) + (size_t)(at.b * p.sdu) + first_row;
  T* ddelta = static_cast<T*>(p.ddelta) + (size_t)(at.b * p.sdd) + first_row;
  T* dz = static_cast<T*>(p.dz) + (Z ? (size_t)(at.b * p.sdz) + first_row : 0);
  const T* Bm = static_cast<const T*>(p.Bm) + (size_t)(at.b * p.sB) + (size_t)at.g * p.N * p.L;
  const T* Cm = static_cast<const T*>(p.Cm) + (size_t)(at.b * p.sC) + (size_t)at.g * p.N * p.L;
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f, D = p.D ? p.D[h] : 0.f;
  const int nblk = (p.N + kModes - 1) / kModes;
  const int off = seg * ST;
  const uint32_t mine = ((uint32_t)min(r, nrow - 1) * (uint32_t)p.L + off) * (uint32_t)sizeof(T);
  const int Lp = p.nchunk * kKeep;
  float* part = p.part_bc +
                (((size_t)at.rb * p.B + at.b) * p.G + at.g) * 2 * p.N * (size_t)Lp;
  // the lanes that put a row's values; the others take the spare word: no branch
  const int put_c = first ? p.N * RP + r : 3 * p.N * RP, pitch_c = first ? RP : 0;
  const int put_d = first ? 2 * p.N * RP + r : 3 * p.N * RP, pitch_d = first ? RP : 0;
  // behind the rows' end: no gradients
  for (int tile = t_hi - 1; tile >= max(t_lo, t_live); --tile) {
    const int t0 = tile * TILE, ns = p.L - t0 - off;
    float zero[ST];
#pragma unroll
    for (int j = 0; j < ST; ++j) zero[j] = 0.f;
    if (live) {
      store_n<T, ST>(spot(du + t0, mine), ns, zero);
      store_n<T, ST>(spot(ddelta + t0, mine), ns, zero);
      if (Z) store_n<T, ST>(spot(dz + t0, mine), ns, zero);
    }
  }
  Stage<T, NT, TILE, true> stage;
  // the kept states of a stage's modes, one to each of a row's first lanes
  float starts = 0.f;
  const auto fetch_starts = [&](int n0, int t0) {
    starts = 0.f;
    if (live && seg < kModes && n0 + seg < p.N)
      starts = p.bounds[((row0 + r) * p.nchunk + t0 / kKeep) * p.N + n0 + seg];
  };
  if (t_lo < t_live) {
    stage.fetch(Bm, Cm, p.N, p.L, 0, (t_live - 1) * TILE, len);
    fetch_starts(0, (t_live - 1) * TILE);
  }
  float sumD = 0.f, sumb = 0.f;
  int buf = 0, sb = 0;
  for (int tile = t_live - 1; tile >= t_lo; --tile) {
    const int t0 = tile * TILE, nv = len - t0 - off;
    float dt[ST], dtu[ST], gy[ST], y[ST], q[ST], w[ST], S = 0.f;
    {
      Lane<T, ST> uv, dv, zv, gv;
      uv.fetch(u + t0, mine, nv);
      dv.fetch(delta + t0, mine, nv);
      gv.fetch(dy + t0, mine, nv);
      if (Z) zv.fetch(z + t0, mine, nv);
#pragma unroll
      for (int j = 0; j < ST; ++j) {
        const float d = softplus(dv.v[j] + bias);
        float g = gv.v[j], rest;
        if (Z) g *= zv.v[j] * sigmoid_pair(zv.v[j], &rest);
        dt[j] = d;
        dtu[j] = d * uv.v[j];
        gy[j] = g;
        y[j] = D * uv.v[j];
        q[j] = w[j] = 0.f;
      }
      if (t0 + TILE > len || !live) {
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          dt[j] = j < nv ? dt[j] : 0.f;
          dtu[j] = j < nv && live ? dtu[j] : 0.f;
          gy[j] = j < nv && live ? gy[j] : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < ST; ++j) S += dt[j];
    }
    for (int blk = 0; blk < nblk; ++blk) {
      stage.put(bc[buf]);
      float start = starts;
      __syncthreads();
      if (blk + 1 < nblk) {
        stage.fetch(Bm, Cm, p.N, p.L, (blk + 1) * kModes, t0, len);
        fetch_starts((blk + 1) * kModes, t0);
      } else if (tile > t_lo) {
        stage.fetch(Bm, Cm, p.N, p.L, 0, t0 - TILE, len);
        fetch_starts(0, t0 - TILE);
      }
      const int n0 = blk * kModes, nm = min(kModes, p.N - n0);
      for (int m = 0; m < nm; ++m) {
        const int n = n0 + m;
        const float k = kap[n * RP + r], carry = car[n * RP + r], was = dre[n * RP + r];
        float v[ST], a[1][ST], ax[ST], c[1][ST], g[ST];
        read_steps<ST>(bc[buf][0][m], seg, v);
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          a[0][j] = exp2_fast(-k * dt[j]);
          c[0][j] = dtu[j] * v[j];
        }
        const float decay = exp2_fast(-k * S);
        float P[1] = {decay}, V[1], xs[1];
        const float enter[1] = {first ? start : 0.f};
        enter_forward<ST, 1>(a, c, P, enter, xs, V);
        float x = xs[0];
        start = row_move<kRowShl + 1>(start);  // the next mode's to the first lane
        float cv[ST];
        read_steps<ST>(bc[buf][1][m], seg, cv);
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          ax[j] = a[0][j] * x;
          x = ax[j] + c[0][j];
          if (Z) y[j] = fmaf(cv[j], x, y[j]);
          g[j] = gy[j] * x;
          c[0][j] = cv[j] * gy[j];
        }
        const auto leave = [&](int which) {
          float o[Q];
#pragma unroll
          for (int i = 0; i < Q; ++i) o[i] = rows_quad(g[i], g[Q + i], g[2 * Q + i], g[3 * Q + i]);
          Part to;
          if constexpr (Q == 2)
            to = Part{o[0], o[1]};
          else
            to = o[0];
          slab[sb][wave][m & 1][which][lane] = to;
        };
        leave(1);
        // against time
        float F = c[0][ST - 1];
#pragma unroll
        for (int j = ST - 2; j >= 0; --j) F = fmaf(a[0][j + 1], F, c[0][j]);
        F *= a[0][0];
        const float right = last ? carry : 0.f;
        P[0] = decay;
        V[0] = fmaf(decay, right, F);
        row_scan<true>(P, V, xs);
        dyn[put_c + n * pitch_c] = V[0];
        float G = xs[0] + right;
        float acc = 0.f;
#pragma unroll
        for (int j = ST - 1; j >= 0; --j) {
          G = j == ST - 1 ? G + c[0][j] : fmaf(a[0][(j + 1) % ST], G, c[0][j]);
          const float wx = G * ax[j];
          g[j] = G * dtu[j];
          q[j] = fmaf(G, v[j], q[j]);
          w[j] = fmaf(k, wx, w[j]);
          acc = fmaf(wx, dt[j], acc);
        }
        leave(0);
        dyn[put_d + n * pitch_d] = was + row_total(acc);
        if ((m & 1) || m + 1 == nm) {
          // one barrier for two modes: the slabs alternate
          __syncthreads();
          const int count = 128 * ((m & 1) + 1);
          for (int i = threadIdx.x; i < count; i += NT) {
            const int e = i & 63, which = i / 64 & 1, mm = i / 128;
            Part sum = slab[sb][0][mm][which][e];
#pragma unroll
            for (int o = 1; o < RW; ++o) sum += slab[sb][o][mm][which][e];
            const int st = (e & 15) * ST + (e >> 4) * Q;
            *reinterpret_cast<Part*>(part + (size_t)(which * p.N + n0 + (m & ~1) + mm) * Lp + t0 +
                                     st) = sum;
          }
          sb ^= 1;
        }
      }
      buf ^= 1;
    }
    // the inputs again, from a cache: held through the modes they would not fit the registers
    Lane<T, ST> uv, dv, zv, gv;
    uv.fetch(u + t0, mine, nv);
    dv.fetch(delta + t0, mine, nv);
    if (Z) {
      gv.fetch(dy + t0, mine, nv);
      zv.fetch(z + t0, mine, nv);
    }
    float o[3][ST];
#pragma unroll
    for (int j = 0; j < ST; ++j) {
      const float uj = uv.v[j];
      float rest;
      const float d = fmaf(uj, q[j], -0.69314718056f * w[j]) * sigmoid_pair(dv.v[j] + bias, &rest);
      o[0][j] = j < nv ? fmaf(dt[j], q[j], D * gy[j]) : 0.f;
      o[1][j] = j < nv ? d : 0.f;
      if (j < nv && live) {
        sumD = fmaf(gy[j], uj, sumD);
        sumb += d;
      }
      if (Z) {
        const float s = sigmoid_pair(zv.v[j], &rest);
        const float e = gv.v[j] * y[j] * fmaf(zv.v[j] * s, rest, s);
        o[2][j] = j < nv ? e : 0.f;
      }
    }
    if (live) {
      const int ns = p.L - t0 - off;
      store_n<T, ST>(spot(du + t0, mine), ns, o[0]);
      store_n<T, ST>(spot(ddelta + t0, mine), ns, o[1]);
      if (Z) store_n<T, ST>(spot(dz + t0, mine), ns, o[2]);
    }
  }
  sumD = row_total(sumD);
  sumb = row_total(sumb);
  if (live && first) {
    float* to = p.part_h + ((row0 + r) * p.nseg + at.seg) * 2;
    to[0] = sumD;
    to[1] = sumb;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = wave * 4 + k;
    if (i < nrow)
      for (int n = lane; n < p.N; n += 64) {
        p.part_n[((row0 + i) * p.nseg + at.seg) * p.N + n] = dre[n * RP + i];
        if (p.dx0 && at.seg == 0) p.dx0[(row0 + i) * p.N + n] = car[n * RP + i];
      }
  }
}

// dB and dC: the row blocks' parts in order; 4 steps to a thread.
template <typename T>
__global__ __launch_bounds__(256) void selective_dbc_kernel(Args p) {
  const int per = (p.L + 1023) / 1024;  // workgroups of a row of steps
  const unsigned k = blockIdx.x / (unsigned)per;  // ((b G + g) 2 + which) N + n
  const int t = ((int)(blockIdx.x - k * per) * 256 + (int)threadIdx.x) * 4;
  if (t >= p.L) return;
  const unsigned n = k % (unsigned)p.N, bg2 = k / (unsigned)p.N;
  const int which = bg2 & 1;
  const unsigned bg = bg2 >> 1;
  const int b = bg / (unsigned)p.G, g = bg - b * p.G;
  const int Lp = p.nchunk * kKeep, len = row_len(p, b);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (t < len) {
    const size_t step = (size_t)p.B * p.G * 2 * p.N * Lp;
    const float* v = p.part_bc + (size_t)k * Lp + t;
    for (int i = 0; i < p.nrb; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(v + i * step);
      s[0] += f.x;
      s[1] += f.y;
      s[2] += f.z;
      s[3] += f.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = t + j < len ? s[j] : 0.f;
  }
  T* to = static_cast<T*>(which ? p.dC : p.dB) + (size_t)(b * (which ? p.sdC : p.sdB)) +
          ((size_t)g * p.N + n) * p.L + t;
  store_n<T, 4>(to, p.L - t, s);
}

// The parameters' gradients: sums over the batch and segments in a fixed order,
// in float64; 16 lanes to a value: N of dlog_re, then dD and ddt_bias, of a channel.
__global__ __launch_bounds__(256) void selective_param_kernel(Args p) {
  const long k = ((long)blockIdx.x * 256 + threadIdx.x) / 16;
  const int sub = threadIdx.x & 15;
  if (k >= (long)p.H * (p.N + 2)) return;
  const int h = (int)(k / (p.N + 2)), n = (int)(k - (long)h * (p.N + 2));
  double s = 0.0;
  const long count = (long)p.B * p.nseg;
  for (long i = sub; i < count; i += 16) {
    const long b = i / p.nseg, at = (b * p.H + h) * p.nseg + (i - b * p.nseg);
    s += (double)(n < p.N ? p.part_n[at * p.N + n] : p.part_h[at * 2 + (n - p.N)]);
  }
  for (int o = 1; o < 16; o <<= 1) s += __shfl_xor(s, o);
  if (sub) return;
  if (n < p.N)  // nothing to add up is 0, whatever the parameter
    p.dlog_re[(size_t)h * p.N + n] =
        (float)(s != 0.0 ? -2.0 * (double)p.log_re[(size_t)h * p.N + n] * s : 0.0);
  else if (n == p.N && p.dD)
    p.dD[h] = (float)s;
  else if (n == p.N + 1 && p.ddt_bias)
    p.ddt_bias[h] = (float)s;
}

// One token: `lpr` lanes to a row (a power of two, at most 64), four modes each.
template <typename T>
__global__ __launch_bounds__(256) void selective_step_kernel(Args p, int lpr) {
  const long row = (long)blockIdx.x * (256 / lpr) + threadIdx.x / lpr;
  const int l = threadIdx.x % lpr;
  const bool in = row < (long)p.B * p.H;
  const long b = in ? row / p.H : 0;
  const int h = in ? (int)(row - b * p.H) : 0;
  const bool live = in && (!p.lens || p.lens[b] > 0);
  const int n = 4 * l, m = in ? min(max(p.N - n, 0), 4) : 0, nv = live ? m : 0;
  const size_t xo = (size_t)(in ? row : 0) * p.N + n;
  const size_t bc = (size_t)(h / p.HG) * p.N + n;
  float x[4], k[4], Bv[4], Cv[4];
  load_n<float, 4>(p.x0 + xo, p.x0 ? m : 0, x);
  load_n<float, 4>(p.log_re + (size_t)h * p.N + n, nv, k);
  load_n<T, 4>(static_cast<const T*>(p.Bm) + (size_t)(b * p.sB) + bc, nv, Bv);
  load_n<T, 4>(static_cast<const T*>(p.Cm) + (size_t)(b * p.sC) + bc, nv, Cv);
  float u = 0.f, d = 0.f, z = 0.f;
  if (live) {
    u = (float)static_cast<const T*>(p.u)[(size_t)(b * p.su) + h];
    d = (float)static_cast<const T*>(p.delta)[(size_t)(b * p.sd) + h];
    if (p.z) z = (float)static_cast<const T*>(p.z)[(size_t)(b * p.sz) + h];
  }
  const float dt = softplus(d + (p.dt_bias ? p.dt_bias[h] : 0.f));
  float y = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < nv) {
      x[j] = fmaf(exp2_fast(-(square_of(k[j]) * kLog2e) * dt), x[j], dt * u * Bv[j]);
      y = fmaf(Cv[j], x[j], y);
    }
  }
  if (p.xT) store_n<float, 4>(p.xT + xo, m, x);
  for (int o = 1; o < lpr; o <<= 1) y += __shfl_xor(y, o);
  if (!in || l) return;
  if (p.D) y = fmaf(p.D[h], u, y);
  float rest;
  if (p.z) y *= z * sigmoid_pair(z, &rest);
  static_cast<T*>(p.y)[row] = (T)(live ? y : 0.f);
}

// How rows go to workgroups.
struct Plan {
  int st;         // steps of a lane: 8, or 4 where rows have at most 64 steps
  int rw;         // groups of four rows
  int nrb;        // row blocks of a group of channels
  int nseg, seg_tiles;
};

Plan plan_of(int B, int H, int G, int N, int L, bool backward) {
  Plan p{8, 8, 1, 1, 1};
  if (L <= 64) p.st = 4;
  const int tile = kSeg * p.st, ntile = std::max(1, (L + tile - 1) / tile), hg = H / G;
  if (!backward && p.st == 8) p.rw = 4;
  p.nrb = (hg + 4 * p.rw - 1) / (4 * p.rw);
  const long have = std::max(1L, (long)B * G * p.nrb);
  const long want = have >= 256 ? 1 : std::min<long>(ntile, 512 / have);
  p.seg_tiles = (int)((ntile + want - 1) / want);
  p.nseg = (ntile + p.seg_tiles - 1) / p.seg_tiles;
  return p;
}

Args make_args(const SelectiveCall& c, const Plan& pl) {
  Args a{};
  a.u = c.u;
  a.delta = c.delta;
  a.z = c.z;
  a.Bm = c.Bm;
  a.Cm = c.Cm;
  a.su = c.stride_u;
  a.sd = c.stride_delta;
  a.sz = c.stride_z;
  a.sB = c.stride_B;
  a.sC = c.stride_C;
  a.log_re = c.log_re;
  a.D = c.D;
  a.dt_bias = c.dt_bias;
  a.lens = c.lens;
  a.B = c.B;
  a.H = c.H;
  a.G = c.G;
  a.N = c.N;
  a.L = c.L;
  a.HG = c.H / c.G;
  a.x0 = c.x0;
  a.xT = c.xT;
  a.y = c.y;
  a.bounds = static_cast<float*>(c.ckpt);
  a.nchunk = (c.L + kKeep - 1) / kKeep;
  a.nrb = pl.nrb;
  a.nseg = pl.nseg;
  a.seg_tiles = pl.seg_tiles;
  a.dy = c.dy;
  a.dx = c.dx;
  a.du = c.du;
  a.ddelta = c.ddelta;
  a.dz = c.dz;
  a.dB = c.dB;
  a.dC = c.dC;
  a.sdu = c.stride_du;
  a.sdd = c.stride_ddelta;
  a.sdz = c.stride_dz;
  a.sdB = c.stride_dB;
  a.sdC = c.stride_dC;
  a.dlog_re = c.dlog_re;
  a.dD = c.dD;
  a.ddt_bias = c.ddt_bias;
  a.dx0 = c.dx0;
  return a;
}

// The workspace's parts; the backward pass's after the split rows'.
struct Layout {
  size_t agg, aggS, bc, n, h, total;
};

Layout layout_of(const Plan& pl, int B, int H, int G, int N, int L, bool backward) {
  const size_t rows = (size_t)B * H;
  Layout o{};
  size_t at = 0;
  const auto take = [&](size_t floats) {
    const size_t here = at;
    at += align_up(floats * sizeof(float), 256);
    return here;
  };
  o.agg = take(pl.nseg > 1 ? rows * pl.nseg * N : 0);
  o.aggS = take(pl.nseg > 1 ? rows * pl.nseg : 0);
  if (backward) {
    o.bc = take((size_t)pl.nrb * B * G * 2 * N * ((size_t)(L + kKeep - 1) / kKeep * kKeep));
    o.n = take(rows * pl.nseg * N);
    o.h = take(rows * pl.nseg * 2);
  }
  o.total = at;
  return o;
}

void place(Args& a, const SelectiveCall& c, const Layout& o) {
  char* ws = static_cast<char*>(c.ws);
  a.agg = reinterpret_cast<float*>(ws + o.agg);
  a.aggS = reinterpret_cast<float*>(ws + o.aggS);
  a.part_bc = reinterpret_cast<float*>(ws + o.bc);
  a.part_n = reinterpret_cast<float*>(ws + o.n);
  a.part_h = reinterpret_cast<float*>(ws + o.h);
}

unsigned blocks_of(long n) { return (unsigned)((n + 255) / 256); }

template <typename T, int ST, int RW, int NW>
hipError_t forward(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)a.B * a.G * a.nrb * a.nseg), block(64 * RW * NW);
  const size_t lds = (size_t)padded(a.N) * (2 * 4 * RW + 2) * sizeof(float);
  if (a.nseg > 1) {
    hipLaunchKernelGGL((selective_fwd_kernel<T, ST, RW, NW, true>), grid, block, lds, st, a);
    hipLaunchKernelGGL((selective_join_kernel<false>), dim3(blocks_of((long)a.B * a.H * a.N)),
                       dim3(256), 0, st, a.agg, a.aggS, a.log_re, a.x0, (long)a.B * a.H, a.H, a.N,
                       a.nseg);
  }
  hipLaunchKernelGGL((selective_fwd_kernel<T, ST, RW, NW, false>), grid, block, lds, st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_forward(const SelectiveCall& c, hipStream_t st) {
  const Plan pl = plan_of(c.B, c.H, c.G, c.N, c.L, false);
  Args a = make_args(c, pl);
  place(a, c, layout_of(pl, c.B, c.H, c.G, c.N, c.L, false));
  return pl.st == 4 ? forward<T, 4, 8, 1>(a, st) : forward<T, 8, 4, 2>(a, st);
}

template <typename T, int ST, int RW>
hipError_t backward(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)a.B * a.G * a.nrb * a.nseg), block(64 * RW);
  const size_t lds = (size_t)a.N * (4 * RW + 1) * sizeof(float);
  if (a.nseg > 1) {
    hipLaunchKernelGGL((selective_bwd_agg_kernel<T, ST, RW>), grid, block, 2 * lds, st, a);
    hipLaunchKernelGGL((selective_join_kernel<true>), dim3(blocks_of((long)a.B * a.H * a.N)),
                       dim3(256), 0, st, a.agg, a.aggS, a.log_re, a.dx, (long)a.B * a.H, a.H, a.N,
                       a.nseg);
  }
  if (a.z)
    hipLaunchKernelGGL((selective_bwd_kernel<T, ST, RW, true>), grid, block, 3 * lds + 4, st, a);
  else
    hipLaunchKernelGGL((selective_bwd_kernel<T, ST, RW, false>), grid, block, 3 * lds + 4, st, a);
  if (a.L > 0)
    hipLaunchKernelGGL((selective_dbc_kernel<T>),
                       dim3((unsigned)a.B * a.G * 2 * a.N * (unsigned)((a.L + 1023) / 1024)),
                       dim3(256), 0, st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_backward(const SelectiveCall& c, hipStream_t st) {
  const Plan pl = plan_of(c.B, c.H, c.G, c.N, c.L, true);
  Args a = make_args(c, pl);
  place(a, c, layout_of(pl, c.B, c.H, c.G, c.N, c.L, true));
  if (c.B > 0) {
    const hipError_t e = pl.st == 4 ? backward<T, 4, 8>(a, st) : backward<T, 8, 8>(a, st);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(selective_param_kernel, dim3(blocks_of((long)c.H * (c.N + 2) * 16)), dim3(256),
                     0, st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_step(const SelectiveCall& c, hipStream_t st) {
  const Args a = make_args(c, Plan{8, 8, 1, 1, 1});
  int lpr = 1;
  while (lpr * 4 < c.N) lpr *= 2;
  const long rows = (long)c.B * c.H, per = 256 / lpr;
  hipLaunchKernelGGL((selective_step_kernel<T>), dim3((unsigned)((rows + per - 1) / per)),
                     dim3(256), 0, st, a, lpr);
  return hipGetLastError();
}

}  // namespace

size_t selective_workspace(int B, int H, int G, int N, int L, bool backward) {
  return layout_of(plan_of(B, H, G, N, L, backward), B, H, G, N, L, backward).total;
}

size_t selective_ckpt(int B, int H, int N, int L) {
  return align_up((size_t)B * H * ((L + kKeep - 1) / kKeep) * N * sizeof(float), 256);
}

hipError_t launch_selective_forward(const SelectiveCall& c, int dtype, hipStream_t st) {
  switch (dtype) {
    case 0: return run_forward<float>(c, st);
    case 1: return run_forward<__bf16>(c, st);
    default: return run_forward<_Float16>(c, st);
  }
}

hipError_t launch_selective_backward(const SelectiveCall& c, int dtype, hipStream_t st) {
  switch (dtype) {
    case 0: return run_backward<float>(c, st);
    case 1: return run_backward<__bf16>(c, st);
    default: return run_backward<_Float16>(c, st);
  }
}

hipError_t launch_selective_step(const SelectiveCall& c, int dtype, hipStream_t st) {
  switch (dtype) {
    case 0: return run_step<float>(c, st);
    case 1: return run_step<__bf16>(c, st);
    default: return run_step<_Float16>(c, st);
  }
}

}  // namespace dssm
