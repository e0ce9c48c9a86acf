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
// Layout.  A row (b, h) takes 16 lanes, ST = 8 consecutive steps each; a wave four
// rows.  16 lanes are what the data-parallel primitives shift and rotate within:
// joining the lanes of a mode takes 8 vector operations, one per step.  The modes
// are walked two at a time, a lane's decays and drives of them in registers, and
// two waves share the modes of a row.  With 16 steps to a lane and one wave the
// joins cost half, but the registers leave two waves per SIMD instead of four, and
// instructions issue slower for it: forward the same (0.20 ms of 4 x 2048 rows of
// 4096 steps and 16 modes), backward 643 us against 595.  B and C are the same for
// all rows of a group: the workgroup's tile of them lies in LDS as float32.
//
// What bounds it is the vector unit (busy in 76% of the cycles, either direction): a
// product for the exponent, the exponential (its own rate a quarter), the drive, two
// passes of the recurrence (one to join the lanes, one from the joined state), the
// join and the read-out, about 7 operations and an exponential per mode and step; the
// backward pass forms the states again, walks their gradients the other way and sums
// two products over rows, about 19 and an
// exponential; and what is done once a step (inputs, gates, turns through LDS) takes
// a third of the time at 16 modes.  4 x 2048 rows of 4096 steps and 16 modes in bf16
// with a gate: forward 0.21 ms (0.27 GB of tensors take 0.05), backward 0.61 + 0.07 ms
// to add the row blocks' dB and dC.  At the 128 registers that four waves per SIMD
// leave, the output kernel keeps 10 to 17 in scratch and the backward kernel 17 to 28.
// The backward pass's LDS, 64 KB and 208 bytes a mode, holds two workgroups to a
// compute unit up to 72 modes and one beyond (B=4 H=2048 L=2048 bf16, a training step's
// us per mode: 64 modes 20.7, 72 20.4, 80 24.0, 128 22.9).
//
// Decays are float32, also those next to 1, and a lane multiplies its 8; from lane to
// lane and tile to tile a state decays by one exponential of the summed step sizes, so
// that a long memory does not pile up a rounding per step.
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
constexpr int kSumTiles = 16;  // tiles whose sums for the parameters are one float32 part
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
  // a row's (backward: a slab's) tiles in nseg segments of seg_tiles
  int nrb, nseg, seg_tiles;
  int pair0;              // the launch's first pair of batch row and group
  float* agg;             // [rows][nseg][N]: ends of the segments, then what enters them
  float* aggS;            // [rows][nseg]: sum of dt
  // backward
  const void* dy;
  const float* dx;
  void *du, *ddelta, *dz, *dB, *dC;
  long long sdu, sdd, sdz, sdB, sdC;
  float *dlog_re, *dD, *ddt_bias, *dx0;
  int npair, tile0, tile1;  // the launch's pairs; the slab's tiles
  int steps;              // of a row of part_bc
  // parts of a row's sums: in all, before this slab, of a segment
  int nparts, part0, seg_parts;
  float* part_bc;         // [nrb][npair][2][N][steps]
  float* part_n;          // [rows][nparts][N]
  float* part_h;          // [rows][nparts][2]
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
// on [0, 1] the polynomial of least relative error (6e-8 with its coefficients in
// float32).  Steps of 1e-3 and less are what the map is used with: log2(1 + t)
// would keep ten bits of them, and this takes half the operations of the series
// of t / (2 + t).  The exponent is one rounded product, so a step below 1 carries
// (1.25 |v| + 6) 2^-24: at 1e-3 at most 5e-7 beside exp2's own 2^-23, 21 bits, as the
// rounded sum of delta and bias leaves it (2.4e-7 there).  Putting back what the product
// loses would halve that and cost 0.3 to 1.4% of every pass over a sequence.
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

// A sum of step sizes, kept finite: resets (steps of 2^127, say) side by side pass
// float32, and a mode with log_re 0 decays by no step however long.  One instruction,
// which takes NaN for 0: the decays of the steps themselves carry it.
__device__ __forceinline__ float finite_sum(float s) {
  return __builtin_amdgcn_fmed3f(s, 0.f, 0x1.fffffep127f);
}

// What stands for log_re^2 in the modes and rows that only fill a workgroup: their
// states are 0 whatever the step, and at 0 a step past float32 would make NaN.
constexpr float kFill = 1.f;

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

__device__ __forceinline__ void put_quad(float* to, const float* v) {
  *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void add_quad(const float* from, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(from);
  v[0] += a.x;
  v[1] += a.y;
  v[2] += a.z;
  v[3] += a.w;
}
// Four steps, the q-th of the tile, to where they are read.
template <int ST>
__device__ __forceinline__ void write_quad(float* tile, int q, const float* v) {
  put_quad(tile + slot<ST>(q / (ST / 4), q % (ST / 4)), v);
}

// Which batch row, group, row block and segment a workgroup works on.
struct Place {
  int b, g, rb, seg;
  __device__ __forceinline__ Place(const Args& p) {
    unsigned k = blockIdx.x;
    seg = (int)(k % (unsigned)p.nseg);
    k /= (unsigned)p.nseg;
    rb = (int)(k % (unsigned)p.nrb);
    k = k / (unsigned)p.nrb + (unsigned)p.pair0;
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

// The group's B and C over one tile and kModes modes, on their way to LDS: 8
// steps of a mode to a thread.
template <typename T, int NT, int TILE, bool BOTH>
struct Stage {
  static constexpr int ST = TILE / kSeg, kRow = TILE / 8, kHalf = kModes * kRow;
  static constexpr int kChunks = (BOTH ? 2 : 1) * kHalf, IT = (kChunks + NT - 1) / NT;
  Packed<T, 8> v[IT];
  // modes n0 .. of the tile from t0; steps at or past len are 0
  __device__ __forceinline__ void fetch(const T* Bm, const T* Cm, int N, int L, int n0, int t0,
                                        int len) {
    const size_t from = (size_t)n0 * L + t0;
    const bool whole = t0 + TILE <= len && n0 + kModes <= N;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = (int)threadIdx.x + i * NT;
      // whole waves take B or C, so that the choice is a scalar's
      const bool second = BOTH && __builtin_amdgcn_readfirstlane(k / kHalf) != 0;
      const int t = k % kRow * 8, n = k / kRow % kModes;
      const T* p = spot((second ? Cm : Bm) + from, (uint32_t)(n * L + t) * sizeof(T));
      if (IT * NT != kChunks && k >= kChunks) break;
      if (whole) {
        v[i].load(p);
      } else {
        const int nv = n0 + n < N ? len - t0 - t : 0;
        v[i].load(p, max(nv, 0), (T)0.f);
      }
    }
  }
  __device__ __forceinline__ void put(float (*to)[kModes][TILE]) const {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = (int)threadIdx.x + i * NT;
      if (IT * NT != kChunks && k >= kChunks) break;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = v[i][j];
      float* tile = to[0][0] + k / kRow * TILE;
      write_quad<ST>(tile, k % kRow * 2, f);
      write_quad<ST>(tile, k % kRow * 2 + 1, f + 4);
    }
  }
};

// A lane's steps of one row as they lie in memory; row0: the workgroup's first
// row at the tile's first step; whole: the workgroup's tile has no end in it.
template <typename T, int SP>
struct Lane {
  Packed<T, SP> v;
  __device__ __forceinline__ void fetch(const T* row0, uint32_t own, int nv, bool whole) {
    if (whole)
      v.load(spot(row0, own));
    else
      v.load(spot(row0, own), max(nv, 0), (T)0.f);
  }
};

template <typename T, int SP>
__device__ __forceinline__ void store_lane(T* row0, uint32_t own, int ns, bool whole,
                                           const float* v) {
  store_n<T, SP>(spot(row0, own), whole ? SP : ns, v);
}

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

// What a workgroup of RW groups of four rows and NW waves to each works on.  A
// lane walks the modes over ST steps of one row (r); what is formed once per
// step (step sizes, gates, outputs) it does for four steps of row `own`, 32
// (16) neighbouring lanes to a row, so that memory is met in whole lines.  The
// two are the same where NW == 1.
template <int ST, int RW, int NW>
struct Lanes {
  static constexpr int NT = 64 * RW * NW, R = 4 * RW, TILE = kSeg * ST, LPR = TILE / 4;
  static_assert(NW * 64 == 4 * LPR, "every step is some lane's own");
  int lane, seg, rg, nw, r, own, step;  // step: the lane's own first one in a tile
  __device__ __forceinline__ Lanes() {
    lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    seg = lane & (kSeg - 1);
    rg = wave / NW;
    nw = wave % NW;
    r = rg * 4 + lane / kSeg;
    own = rg * 4 + (nw * 64 + lane) / LPR;
    step = lane % LPR * 4;
  }
};

// Forward over a row or a segment of it; the modes of a group of rows are shared
// out among its NW waves.  AGG: only the segment's ends.
template <typename T, int ST, int RW, int NW, bool AGG>
__global__ __launch_bounds__(64 * RW * NW) __attribute__((amdgpu_waves_per_eu(4)))
void selective_fwd_kernel(Args p) {
  typedef Lanes<ST, RW, NW> Work;
  constexpr int NT = Work::NT, R = Work::R, TILE = Work::TILE;
  __shared__ float bc[2][AGG ? 1 : 2][kModes][TILE];
  // step sizes and drives of the rows; their outputs, a wave's part each
  __shared__ float xch[NW > 1 ? 2 : 1][NW > 1 ? R : 1][TILE];
  constexpr bool kJoinY = NW > 1 && !AGG;
  __shared__ float yred[kJoinY ? NW : 1][kJoinY ? R : 1][TILE];
  extern __shared__ float dyn[];
  const int NP = padded(p.N);
  const Cells kap{dyn, R, NP}, car{dyn + R * NP, R, NP};  // log_re^2; the state entering the tile
  const Place at(p);
  if (AGG && at.seg == p.nseg - 1) return;  // nobody joins the last segment
  const Work w;
  const int seg = w.seg, nw = w.nw, r = w.r, lane = w.lane;
  const int len = row_len(p, at.b);
  const int ntile = (p.L + TILE - 1) / TILE;
  const int t_lo = at.seg * p.seg_tiles, t_hi = min(ntile, t_lo + p.seg_tiles);
  const int t_live = min(t_hi, (len + TILE - 1) / TILE);
  const int h0 = at.g * p.HG + at.rb * R, nrow = min(R, p.HG - at.rb * R);
  const size_t row0 = (size_t)at.b * p.H + h0;  // the workgroup's first row
  // the waves of a row group take turns with its modes
  for (int n = (lane & 15) * NW + nw; n < NP; n += 16 * NW) {
    float c = 0.f, s = kFill;
    if (r < nrow && n < p.N) {
      s = square_of(p.log_re[(size_t)(h0 + r) * p.N + n]) * kLog2e;
      if (!AGG && p.nseg > 1)
        c = p.agg[((row0 + r) * p.nseg + at.seg) * p.N + n];
      else if (!AGG && p.x0)
        c = p.x0[(row0 + r) * p.N + n];
    }
    kap.row(r)[n] = s;
    car.row(r)[n] = c;
  }
  for (int n = threadIdx.x; n < NP; n += NT) car.row(R)[n] = 0.f;  // before the first barrier
  const float* krow = kap.row(r) + nw;
  const float* from = car.from(r, seg == 0) + nw;
  float* to = car.to(r, seg == kSeg - 1) + nw;
  const size_t first_row = (size_t)h0 * p.L;
  const T* u = static_cast<const T*>(p.u) + (size_t)(at.b * p.su) + first_row;
  const T* delta = static_cast<const T*>(p.delta) + (size_t)(at.b * p.sd) + first_row;
  const T* z = static_cast<const T*>(p.z) + (p.z ? (size_t)(at.b * p.sz) + first_row : 0);
  const T* Bm = static_cast<const T*>(p.Bm) + (size_t)(at.b * p.sB) + (size_t)at.g * p.N * p.L;
  const T* Cm = static_cast<const T*>(p.Cm) + (size_t)(at.b * p.sC) + (size_t)at.g * p.N * p.L;
  T* out = static_cast<T*>(p.y) + row0 * p.L;
  const int h = h0 + min(w.own, nrow - 1);
  const bool live = w.own < nrow;
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  const float D = !AGG && p.D ? p.D[h] : 0.f;
  const int nblk = (p.N + kModes - 1) / kModes;
  const uint32_t mine =
      ((uint32_t)min(w.own, nrow - 1) * (uint32_t)p.L + w.step) * (uint32_t)sizeof(T);
  Stage<T, NT, TILE, !AGG> stage;
  Lane<T, 4> un, dn;
  if (t_lo < t_live) {
    const int t = t_lo * TILE;
    stage.fetch(Bm, Cm, p.N, p.L, 0, t, len);
    dn.fetch(delta + t, mine, len - t - w.step, t + TILE <= len);
    un.fetch(u + t, mine, len - t - w.step, t + TILE <= len);
  }
  // where the lane's own steps, and those it walks, lie among a tile's rows
  const int own_at = w.own * TILE + slot<ST>(w.step / ST, w.step % ST / 4), walk_at = r * TILE;
  uint32_t keep_at = ((uint32_t)r * p.nchunk * p.N + (lane & 15) * NW + nw) * 4u;
  float Sseg = 0.f;
  int buf = 0;
  for (int tile = t_lo; tile < t_live; ++tile) {
    const int t0 = tile * TILE, nv = len - t0 - w.step;
    const bool whole = t0 + TILE <= len;
    // the states entering a chunk, for the backward pass
    if (!AGG && p.bounds && (t0 & (kKeep - 1)) == 0) {
      float* keep = p.bounds + (row0 * p.nchunk + t0 / kKeep) * p.N;
      if (r < nrow)
        for (int n = (lane & 15) * NW + nw, k = 0; n < p.N; n += 16 * NW, k += 64 * NW)
          *spot(keep, keep_at + k) = car.row(r)[n];
    }
    Lane<T, 4> zc;
    float dt[ST], du[ST], y[ST], skip[4];
    {
      float own[2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        own[0][j] = softplus(dn.v[j] + bias);
        own[1][j] = own[0][j] * un.v[j];
        skip[j] = D * un.v[j];
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          own[0][j] = j < nv ? own[0][j] : 0.f;
          own[1][j] = j < nv ? own[1][j] : 0.f;
        }
      }
      if constexpr (NW == 1) {
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          dt[j] = own[0][j];
          du[j] = own[1][j];
        }
      } else {
        put_quad(xch[0][0] + own_at, own[0]);
        put_quad(xch[1][0] + own_at, own[1]);
      }
    }
#pragma unroll
    for (int j = 0; j < ST; ++j) y[j] = 0.f;
    // the gate is read for this tile's end, the rest for the next tile
    if (!AGG && p.z) zc.fetch(z + t0, mine, nv, whole);
    if (tile + 1 < t_live) {
      const int t = t0 + TILE;
      dn.fetch(delta + t, mine, len - t - w.step, t + TILE <= len);
      un.fetch(u + t, mine, len - t - w.step, t + TILE <= len);
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
          read_steps<ST>(xch[0][0] + walk_at, seg, dt);
          read_steps<ST>(xch[1][0] + walk_at, seg, du);
        }
#pragma unroll
        for (int j = 0; j < ST; ++j) S += dt[j];
        S = finite_sum(S);
        if (AGG) Sseg = finite_sum(Sseg + S);
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
      float own[4];
      if constexpr (kJoinY) {
        // the next tile's first barrier keeps these from being overwritten too early
#pragma unroll
        for (int k = 0; k < ST / 4; ++k)
          put_quad(yred[nw][0] + walk_at + slot<ST>(seg, k), y + 4 * k);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) own[j] = skip[j];
#pragma unroll
        for (int k = 0; k < NW; ++k)
          add_quad(yred[k][0] + own_at, own);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) own[j] = y[j] + skip[j];
      }
      if (p.z) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float rest;
          own[j] *= zc.v[j] * sigmoid_pair(zc.v[j], &rest);
        }
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 4; ++j) own[j] = j < nv ? own[j] : 0.f;
      }
      if (live) store_lane<T, 4>(out + t0, mine, p.L - t0 - w.step, whole, own);
    }
  }
  if (AGG) {
    const float s = finite_sum(row_total(Sseg));
    if (r < nrow && seg == 0 && nw == 0) p.aggS[(row0 + r) * p.nseg + at.seg] = s;
  } else {
    // behind the rows' end: outputs are 0, the states stay
    for (int tile = max(t_lo, t_live); tile < t_hi; ++tile) {
      const int t0 = tile * TILE;
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      if (live) store_n<T, 4>(spot(out + t0, mine), p.L - t0 - w.step, zero);
    }
  }
  // what leaves: the state after the row, or the segment's own part of it
  float* out_x = AGG ? p.agg + (size_t)at.seg * p.N : at.seg == p.nseg - 1 ? p.xT : nullptr;
  if (out_x && r < nrow) {
    const size_t pitch = (size_t)(AGG ? p.nseg : 1) * p.N;
    for (int n = (lane & 15) * NW + nw; n < p.N; n += 16 * NW)
      out_x[(row0 + r) * pitch + n] = car.row(r)[n];
  }
}

// What enters each segment of a split row: the segments' ends joined in order
// (REV: from the last to the first, `start` being the gradient of the state after
// the row).  16 modes of a row to a workgroup, the segments in 16 parts: a part's
// own end first, then what enters the part, then its segments (128 rows of 16
// modes and 256 segments: 6 us, one thread walking a mode's segments 22).
template <bool REV>
__global__ __launch_bounds__(256) void selective_join_kernel(float* agg, const float* aggS,
                                                             const float* log_re,
                                                             const float* start, int H, int N,
                                                             int nseg) {
  __shared__ float2 ends[16][16];
  const int nb = (N + 15) / 16;
  const long row = blockIdx.x / (unsigned)nb;
  const int m = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int n = (int)(blockIdx.x - (unsigned)row * nb) * 16 + m, at = min(n, N - 1);
  const float kap = square_of(log_re[(row % H) * N + at]) * kLog2e;
  float* v = agg + row * nseg * N + at;
  const float* s = aggS + row * nseg;
  const int per = (nseg + 15) / 16, lo = part * per, hi = min(nseg, lo + per);
  // the segment nobody joins, the last in order, has no end of its own
  const auto segment = [&](int j) { return REV ? nseg - 1 - j : j; };
  // steps of no length decay nothing, whatever the parameter
  const auto decay = [&](float d) { return d == 0.f ? 1.f : exp2_fast(-kap * d); };
  float S = 0.f, V = 0.f;
#pragma unroll 4
  for (int j = lo; j < hi; ++j) {
    const int i = segment(j);
    const float d = j + 1 < nseg ? s[i] : 0.f, e = j + 1 < nseg ? v[(size_t)i * N] : 0.f;
    V = fmaf(decay(d), V, e);
    S = finite_sum(S + d);
  }
  ends[part][m] = make_float2(S, V);
  __syncthreads();
  float c = start ? start[row * N + at] : 0.f;
  for (int k = 0; k < part; ++k) c = fmaf(decay(ends[k][m].x), c, ends[k][m].y);
#pragma unroll 4
  for (int j = lo; j < hi; ++j) {
    const int i = segment(j);
    const float d = j + 1 < nseg ? s[i] : 0.f, e = j + 1 < nseg ? v[(size_t)i * N] : 0.f;
    if (n < N) v[(size_t)i * N] = c;
    c = fmaf(decay(d), c, e);
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
  const int t_lo = p.tile0 + at.seg * p.seg_tiles, t_hi = min(p.tile1, t_lo + p.seg_tiles);
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
              : kFill;
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
    const bool whole = t0 + TILE <= len;
    Lane<T, ST> dv, zv, gv;
    dv.fetch(delta + t0, mine, nv, whole);
    gv.fetch(dy + t0, mine, nv, whole);
    if (p.z) zv.fetch(z + t0, mine, nv, whole);
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
    S = finite_sum(S);
    Sseg = finite_sum(Sseg + S);
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
  const float s = finite_sum(row_total(Sseg));
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
// added up over a wave's four rows in registers, over the workgroup's row groups
// through LDS, and left for a kernel of its own.
template <typename T, int ST, int RW, int NW, bool Z>
__global__ __launch_bounds__(64 * RW * NW) __attribute__((amdgpu_waves_per_eu(4)))
void selective_bwd_kernel(Args p) {
  typedef Lanes<ST, RW, NW> Work;
  constexpr int NT = Work::NT, R = Work::R, TILE = Work::TILE, Q = ST / 4;
  typedef float Pair __attribute__((ext_vector_type(2)));
  typedef typename std::conditional<Q == 2, Pair, float>::type Part;  // Q steps
  __shared__ float bc[2][kModes][TILE];
  __shared__ Part slab[RW][kModes][2][64];
  // step sizes, drives and the output's gradients of the rows; at a tile's end the
  // waves' sums over their modes
  __shared__ float xch[NW > 1 ? 3 * (NW - 1) : 1][NW > 1 ? R : 1][TILE];
  extern __shared__ float dyn[];
  const int NP = padded(p.N);
  const Cells kap{dyn, R, NP};                  // log_re^2
  const Cells car{dyn + R * NP, R, NP};         // state gradient entering the tile
  const Cells dre{dyn + (2 * R + 2) * NP, R, NP};  // sum of w dt
  const Place at(p);
  const Work w_;
  const int seg = w_.seg, rg = w_.rg, nw = w_.nw, r = w_.r, lane = w_.lane;
  const int len = row_len(p, at.b);
  const int t_lo = p.tile0 + at.seg * p.seg_tiles, t_hi = min(p.tile1, t_lo + p.seg_tiles);
  const int t_live = min(t_hi, (len + TILE - 1) / TILE);
  const int h0 = at.g * p.HG + at.rb * R, nrow = min(R, p.HG - at.rb * R);
  const size_t row0 = (size_t)at.b * p.H + h0;
  for (int n = (lane & 15) * NW + nw; n < NP; n += 16 * NW) {
    float c = 0.f, s = kFill;
    if (r < nrow && n < p.N) {
      s = square_of(p.log_re[(size_t)(h0 + r) * p.N + n]) * kLog2e;
      if (p.nseg > 1)
        c = p.agg[((row0 + r) * p.nseg + at.seg) * p.N + n];
      else if (p.dx)
        c = p.dx[(row0 + r) * p.N + n];
    }
    kap.row(r)[n] = s;
    car.row(r)[n] = c;
    dre.row(r)[n] = 0.f;
  }
  for (int n = threadIdx.x; n < NP; n += NT) car.row(R)[n] = 0.f;  // before the first barrier
  const float* krow = kap.row(r) + nw;
  const float* from = car.from(r, seg == kSeg - 1) + nw;
  float* to = car.to(r, seg == 0) + nw;
  const float* dre_row = dre.row(r) + nw;
  float* dre_to = dre.to(r, seg == 0) + nw;
  const size_t first_row = (size_t)h0 * p.L;
  const T* u = static_cast<const T*>(p.u) + (size_t)(at.b * p.su) + first_row;
  const T* delta = static_cast<const T*>(p.delta) + (size_t)(at.b * p.sd) + first_row;
  const T* z = static_cast<const T*>(p.z) + (Z ? (size_t)(at.b * p.sz) + first_row : 0);
  const T* dy = static_cast<const T*>(p.dy) + row0 * p.L;
  T* du = static_cast<T*>(p.du) + (size_t)(at.b * p.sdu) + first_row;
  T* ddelta = static_cast<T*>(p.ddelta) + (size_t)(at.b * p.sdd) + first_row;
  T* dz = static_cast<T*>(p.dz) + (Z ? (size_t)(at.b * p.sdz) + first_row : 0);
  const T* Bm = static_cast<const T*>(p.Bm) + (size_t)(at.b * p.sB) + (size_t)at.g * p.N * p.L;
  const T* Cm = static_cast<const T*>(p.Cm) + (size_t)(at.b * p.sC) + (size_t)at.g * p.N * p.L;
  const int h = h0 + min(w_.own, nrow - 1);
  const bool live = w_.own < nrow;
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f, D = p.D ? p.D[h] : 0.f;
  const int nblk = (p.N + kModes - 1) / kModes;
  const uint32_t mine =
      ((uint32_t)min(w_.own, nrow - 1) * (uint32_t)p.L + w_.step) * (uint32_t)sizeof(T);
  const int first = p.tile0 * TILE;
  float* part = p.part_bc + ((size_t)at.rb * p.npair + (at.b * p.G + at.g - p.pair0)) * 2 * p.N *
                                (size_t)p.steps;
  // where the lane's own steps, and those it walks, lie among a tile's rows
  const int own_at = w_.own * TILE + slot<ST>(w_.step / ST, w_.step % ST / 4), walk_at = r * TILE;
  const uint32_t keep_at = ((uint32_t)r * p.nchunk * p.N + seg * NW + nw) * 4u;
  // behind the rows' end: no gradients
  for (int tile = t_hi - 1; tile >= max(t_lo, t_live); --tile) {
    const int t0 = tile * TILE, ns = p.L - t0 - w_.step;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
      store_n<T, 4>(spot(du + t0, mine), ns, zero);
      store_n<T, 4>(spot(ddelta + t0, mine), ns, zero);
      if (Z) store_n<T, 4>(spot(dz + t0, mine), ns, zero);
    }
  }
  Stage<T, NT, TILE, true> stage;
  // the kept states of the wave's modes of a stage, one to each of a row's first lanes
  float starts = 0.f;
  const auto fetch_starts = [&](int n0, int t0) {
    starts = 0.f;
    if (r < nrow && seg < kModes / NW && n0 + seg * NW + nw < p.N)
      starts = *spot(p.bounds + (row0 * p.nchunk + t0 / kKeep) * p.N + n0, keep_at);
  };
  if (t_lo < t_live) {
    stage.fetch(Bm, Cm, p.N, p.L, 0, (t_live - 1) * TILE, len);
    fetch_starts(0, (t_live - 1) * TILE);
  }
  // the parameters' sums over kSumTiles tiles leave, to be added up in float64; a row's
  // own lanes: 16, or two rows of the vector unit's 16
  float sumD = 0.f, sumb = 0.f;
  const auto leave_sums = [&](int which) {
    sumD = row_total(sumD);
    sumb = row_total(sumb);
    if (Work::LPR == 32) {
      sumD = rows_sum(sumD);
      sumb = rows_sum(sumb);
    }
    const int to = p.part0 + at.seg * p.seg_parts + which;
    if (live && w_.step == 0) {
      float* put = p.part_h + ((row0 + w_.own) * p.nparts + to) * 2;
      put[0] = sumD;
      put[1] = sumb;
    }
    sumD = sumb = 0.f;
    if (r < nrow)
      for (int n = (lane & 15) * NW + nw; n < p.N; n += 16 * NW) {
        p.part_n[((row0 + r) * p.nparts + to) * p.N + n] = dre.row(r)[n];
        dre.row(r)[n] = 0.f;
      }
  };
  for (int k = p.seg_parts - 1; t_lo + k * kSumTiles >= t_live && k >= 0; --k) leave_sums(k);
  for (int tile = t_live - 1; tile >= t_lo; --tile) {
    const int t0 = tile * TILE, nv = len - t0 - w_.step;
    const bool whole = t0 + TILE <= len;
    float dt[ST], dtu[ST], gy[ST], y[ST], q[ST], w[ST], S = 0.f;
    {
      Lane<T, 4> uv, dv, zv, gv;
      uv.fetch(u + t0, mine, nv, whole);
      dv.fetch(delta + t0, mine, nv, whole);
      gv.fetch(dy + t0, mine, nv, whole);
      if (Z) zv.fetch(z + t0, mine, nv, whole);
      float own[3][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = softplus(dv.v[j] + bias);
        float g = gv.v[j], rest;
        if (Z) g *= zv.v[j] * sigmoid_pair(zv.v[j], &rest);
        own[0][j] = d;
        own[1][j] = d * uv.v[j];
        own[2][j] = g;
      }
      if (!whole || nrow < R) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          own[0][j] = j < nv && live ? own[0][j] : 0.f;
          own[1][j] = j < nv && live ? own[1][j] : 0.f;
          own[2][j] = j < nv && live ? own[2][j] : 0.f;
        }
      }
      if constexpr (NW == 1) {
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          dt[j] = own[0][j];
          dtu[j] = own[1][j];
          gy[j] = own[2][j];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) put_quad(xch[i][0] + own_at, own[i]);
      }
    }
#pragma unroll
    for (int j = 0; j < ST; ++j) y[j] = q[j] = w[j] = 0.f;
    for (int blk = 0; blk < nblk; ++blk) {
      stage.put(bc);
      float start = starts;
      __syncthreads();
      if (blk + 1 < nblk) {
        stage.fetch(Bm, Cm, p.N, p.L, (blk + 1) * kModes, t0, len);
        fetch_starts((blk + 1) * kModes, t0);
      } else if (tile > t_lo) {
        stage.fetch(Bm, Cm, p.N, p.L, 0, t0 - TILE, len);
        fetch_starts(0, t0 - TILE);
      }
      if (blk == 0) {
        if constexpr (NW > 1) {
          read_steps<ST>(xch[0][0] + walk_at, seg, dt);
          read_steps<ST>(xch[1][0] + walk_at, seg, dtu);
          read_steps<ST>(xch[2][0] + walk_at, seg, gy);
        }
#pragma unroll
        for (int j = 0; j < ST; ++j) S += dt[j];
        S = finite_sum(S);
      }
      const int n0 = blk * kModes, nm = p.N - n0;
      // one mode to each of a row group's waves; modes past the last one are zeros
      const auto walk = [&](auto step) {
        constexpr int m0 = decltype(step)::value * NW;
        __builtin_amdgcn_sched_barrier(0);  // steps mixed together would not fit the registers
        const float k = krow[n0 + m0], right = from[n0 + m0], was = dre_row[n0 + m0];
        float v[ST], a[1][ST], ax[ST], c[1][ST], g[ST];
        read_steps<ST>(bc[0][m0 + nw], seg, v);
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          a[0][j] = exp2_fast(-k * dt[j]);
          c[0][j] = dtu[j] * v[j];
        }
        const float decay = exp2_fast(-k * S);
        float P[1] = {decay}, V[1], xs[1];
        const float enter[1] = {seg == 0 ? start : 0.f};
        enter_forward<ST, 1>(a, c, P, enter, xs, V);
        float x = xs[0];
        start = row_move<kRowShl + 1>(start);  // the next mode's to the first lane
        read_steps<ST>(bc[1][m0 + nw], seg, g);
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          ax[j] = a[0][j] * x;
          x = ax[j] + c[0][j];
          if (Z) y[j] = fmaf(g[j], x, y[j]);
          c[0][j] = g[j] * gy[j];
          g[j] = gy[j] * x;
        }
        const auto leave = [&](int which) {
          float o[Q];
#pragma unroll
          for (int i = 0; i < Q; ++i) o[i] = rows_quad(g[i], g[Q + i], g[2 * Q + i], g[3 * Q + i]);
          Part sum;
          if constexpr (Q == 2)
            sum = Part{o[0], o[1]};
          else
            sum = o[0];
          slab[rg][m0 + nw][which][lane] = sum;
        };
        leave(1);
        // against time
        float F = c[0][ST - 1];
#pragma unroll
        for (int j = ST - 2; j >= 0; --j) F = fmaf(a[0][j + 1], F, c[0][j]);
        P[0] = decay;
        V[0] = fmaf(decay, right, F * a[0][0]);
        row_scan<true>(P, V, xs);
        to[n0 + m0] = V[0];
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
        dre_to[n0 + m0] = was + row_total(acc);
      };
      walk(std::integral_constant<int, 0>());
      if (nm > NW) walk(std::integral_constant<int, 1>());
      if (nm > 2 * NW) walk(std::integral_constant<int, 2>());
      if (nm > 3 * NW) walk(std::integral_constant<int, 3>());
      if constexpr (kModes > 4 * NW) {
        if (nm > 4 * NW) walk(std::integral_constant<int, 4>());
        if (nm > 5 * NW) walk(std::integral_constant<int, 5>());
        if (nm > 6 * NW) walk(std::integral_constant<int, 6>());
        if (nm > 7 * NW) walk(std::integral_constant<int, 7>());
      }
      // between this barrier and the next stage's the sums are read, and B and C replaced
      __syncthreads();
      const int count = 128 * min(kModes, nm);
      for (int i = opaque((int)threadIdx.x); i < count; i += NT) {
        // neighbouring threads take neighbouring steps
        const int e = (i & 3) * 16 + (i >> 2 & 15), which = i / 64 & 1, m = i / 128;
        Part sum = slab[0][m][which][e];
#pragma unroll
        for (int o = 1; o < RW; ++o) sum += slab[o][m][which][e];
        *reinterpret_cast<Part*>(part + (size_t)(which * p.N + n0 + m) * p.steps + (t0 - first) +
                                 (e & 15) * ST + (e >> 4) * Q) = sum;
      }
    }
    // the inputs again, from a cache: held through the modes they would not fit the registers
    Lane<T, 4> uv, dv, zv, gv;
    uv.fetch(u + t0, mine, nv, whole);
    dv.fetch(delta + t0, mine, nv, whole);
    gv.fetch(dy + t0, mine, nv, whole);
    if (Z) zv.fetch(z + t0, mine, nv, whole);
    float own[3][4];
    if constexpr (NW > 1) {
      // the first wave's part, then (after all have read it) the others' onto it; a wave past
      // the modes' barriers has read the step sizes
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) own[i][j] = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        if (nw == k) {
#pragma unroll
          for (int e = 0; e < ST / 4; ++e) {
            const int to = walk_at + slot<ST>(seg, e);
            put_quad(xch[0][0] + to, q + 4 * e);
            put_quad(xch[1][0] + to, w + 4 * e);
            if (Z) put_quad(xch[2][0] + to, y + 4 * e);
          }
        }
        __syncthreads();
        add_quad(xch[0][0] + own_at, own[0]);
        add_quad(xch[1][0] + own_at, own[1]);
        if (Z) add_quad(xch[2][0] + own_at, own[2]);
        __syncthreads();
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        own[0][j] = q[j];
        own[1][j] = w[j];
        own[2][j] = y[j];
      }
    }
    float o[3][4], tileD = 0.f, tileb = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float uj = uv.v[j], pre = dv.v[j] + bias, dtj = softplus(pre);
      float rest, g = gv.v[j];
      if (Z) {
        const float s = sigmoid_pair(zv.v[j], &rest), silu = zv.v[j] * s;
        o[2][j] = g * fmaf(D, uj, own[2][j]) * fmaf(silu, rest, s);
        g *= silu;
      }
      o[0][j] = fmaf(dtj, own[0][j], D * g);
      o[1][j] = fmaf(uj, own[0][j], -0.69314718056f * own[1][j]) * sigmoid_pair(pre, &rest);
      tileD = fmaf(g, j < nv ? uj : 0.f, tileD);
      tileb += j < nv ? o[1][j] : 0.f;
    }
    sumD += tileD;
    sumb += tileb;
    if (!whole) {
#pragma unroll
      for (int i = 0; i < (Z ? 3 : 2); ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = j < nv ? o[i][j] : 0.f;
    }
    if (live) {
      const int ns = p.L - t0 - w_.step;
      store_lane<T, 4>(du + t0, mine, ns, whole, o[0]);
      store_lane<T, 4>(ddelta + t0, mine, ns, whole, o[1]);
      if (Z) store_lane<T, 4>(dz + t0, mine, ns, whole, o[2]);
    }
    if ((tile - t_lo) % kSumTiles == 0) leave_sums((tile - t_lo) / kSumTiles);
  }
  if (p.dx0 && at.seg == 0 && r < nrow)
    for (int n = (lane & 15) * NW + nw; n < p.N; n += 16 * NW)
      p.dx0[(row0 + r) * p.N + n] = car.row(r)[n];
}

// dB and dC of a slab: the row blocks' parts in order; 4 steps to a thread.
template <typename T, int TILE>
__global__ __launch_bounds__(256) void selective_dbc_kernel(Args p) {
  const int first = p.tile0 * TILE, end = min(p.L, p.tile1 * TILE);
  const unsigned per = (end - first + 1023u) / 1024;  // parts of a row of steps
  const unsigned k = blockIdx.x / per;                // (pair 2 + which) N + n
  const int t = first + ((int)(blockIdx.x - k * per) * 256 + (int)threadIdx.x) * 4;
  if (t >= end) return;
  const unsigned n = k % (unsigned)p.N, half = k / (unsigned)p.N;
  const int which = half & 1;
  const unsigned bg = (half >> 1) + (unsigned)p.pair0;
  const int b = bg / (unsigned)p.G, g = bg - b * p.G;
  const int len = row_len(p, b);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (t < len) {
    const size_t block = (size_t)p.npair * 2 * p.N * p.steps;
    const float* v = p.part_bc + (size_t)k * p.steps + (t - first);
    for (int i = 0; i < p.nrb; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(v + i * block);
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
  const long count = (long)p.B * p.nparts;
  for (long i = sub; i < count; i += 16) {
    const long b = i / p.nparts, at = (b * p.H + h) * p.nparts + (i - b * p.nparts);
    s += (double)(n < p.N ? p.part_n[at * p.N + n] : p.part_h[at * 2 + (n - p.N)]);
  }
  for (int o = 1; o < 16; o <<= 1) s += __shfl_xor(s, o);
  if (sub) return;
  if (n < p.N) {
    // nothing to add up is 0, whatever the parameter; so is what a parameter of 0
    // multiplies, whose sum w dt resets may take past float32
    const float lr = p.log_re[(size_t)h * p.N + n];
    p.dlog_re[(size_t)h * p.N + n] =
        (float)(s != 0.0 && lr != 0.f ? -2.0 * (double)lr * s : 0.0);
  } else if (n == p.N && p.dD)
    p.dD[h] = (float)s;
  else if (n == p.N + 1 && p.ddt_bias)
    p.ddt_bias[h] = (float)s;
}

// One token: `lpr` lanes to a row (a power of two, at most 64), four modes each;
// V rows of the batch to a lane, which share the channel's parameters and are all
// asked for at once.
template <typename T, int V>
__global__ __launch_bounds__(256) void selective_step_kernel(Args p, int lpr) {
  // workgroups: a batch row's (or V rows') channels side by side
  const unsigned block = __builtin_amdgcn_readfirstlane(blockIdx.x);
  const unsigned per = (unsigned)(p.H * lpr + 255) / 256, group = block / per;
  const int at = (int)((block - group * per) * 256 + threadIdx.x), b0 = (int)group * V;
  const int l = at & (lpr - 1), row = at / lpr;
  const bool in = row < p.H;
  const int h = in ? row : 0;
  const int n = 4 * l, m = in ? min(max(p.N - n, 0), 4) : 0;
  const size_t bc = (p.G > 1 ? (size_t)(h / p.HG) * p.N : 0) + n;
  float x[V][4], Bv[V][4], Cv[V][4], k[4], u[V], d[V], z[V];
  bool live[V];
  load_n<float, 4>(p.log_re + (size_t)h * p.N + n, m, k);
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f, D = p.D ? p.D[h] : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int b = min(b0 + i, p.B - 1);
    live[i] = b0 + i < p.B && (!p.lens || p.lens[b] > 0);
    const int nv = live[i] ? m : 0;
    load_n<float, 4>(p.x0 + ((size_t)b * p.H + h) * p.N + n, p.x0 && b0 + i < p.B ? m : 0, x[i]);
    load_n<T, 4>(static_cast<const T*>(p.Bm) + (size_t)(b * p.sB) + bc, nv, Bv[i]);
    load_n<T, 4>(static_cast<const T*>(p.Cm) + (size_t)(b * p.sC) + bc, nv, Cv[i]);
    u[i] = d[i] = z[i] = 0.f;
    if (live[i] && in) {
      u[i] = (float)static_cast<const T*>(p.u)[(size_t)(b * p.su) + h];
      d[i] = (float)static_cast<const T*>(p.delta)[(size_t)(b * p.sd) + h];
      if (p.z) z[i] = (float)static_cast<const T*>(p.z)[(size_t)(b * p.sz) + h];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = square_of(k[j]) * kLog2e;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float dt = softplus(d[i] + bias), drive = dt * u[i];
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float next = fmaf(exp2_fast(-k[j] * dt), x[i][j], drive * Bv[i][j]);
      x[i][j] = live[i] ? next : x[i][j];
      y += j < m ? Cv[i][j] * next : 0.f;
    }
    for (int o = 1; o < lpr; o <<= 1) y += __shfl_xor(y, o);
    if (b0 + i >= p.B || !in) continue;
    const size_t to = (size_t)(b0 + i) * p.H + h;
    if (p.xT) store_n<float, 4>(p.xT + to * p.N + n, m, x[i]);
    if (l) continue;
    y = fmaf(D, u[i], y);
    float rest;
    if (p.z) y *= z[i] * sigmoid_pair(z[i], &rest);
    static_cast<T*>(p.y)[to] = (T)(live[i] ? y : 0.f);
  }
}

// How rows go to workgroups.  A workgroup has 16 rows of 8 steps to a lane; rows of
// at most 64 steps fill 4 to a lane, and it has 32 of them (8 x 2048 rows of 64 steps
// and 16 modes, bf16: 10 us forward and 44 backward, with 8 to a lane 19 and 85).
//
// 128 workgroups and fewer leave half the device idle: a row's tiles are cut into
// segments, up to 512 workgroups, whose ends a first pass forms and a small kernel
// joins.  That is half the work again and two launches more, so it needs a row
// long enough.  Measured, whole rows against segments, 16 modes, bf16, in us
// (H channels x L steps):
//   forward   1024 x 512 18 / 22, 1024 x 1024 32 / 24, 2048 x 1024 33 / 34, 2048 x 2048 62 / 52
//   backward  1024 x 256 52 / 55, 1024 x 512  71 / 53, 2048 x 512  91 / 82, 2048 x 2048 225 / 152
// At 192 workgroups (3 x 1024 rows of 4096 steps) whole rows win, 119 / 159 and 405 /
// 417; half as many segments lose (2048 x 4096: 117 and 411 whole, 89 and 244 in 512
// workgroups), 1024 workgroups gain no more.
//
// The backward pass leaves dB and dC of every row block in float32, B G ceil(H / (16 G))
// 2 N L values: at 128 modes 32 times a tensor of 16 bits, were they all held at once.
// A slab of tiles of all rows holds at most kPartFloats of them (one tile's of
// some pairs of batch row and group, where all pairs' are more); the slabs go from the
// last to the first, each from the state gradient that the one behind it leaves (8 x 4096
// rows of 8192 steps and 128 modes: all at once 16 GiB and 37.2 ms, in slabs of 1 GiB
// 38.6, of 2 GiB 37.5).
struct Plan {
  int st;         // steps of a lane
  int rw;         // groups of four rows
  int nrb;        // row blocks of a group of channels
  int nslab, slab_tiles, npair;
  int nseg, seg_tiles, seg_parts;
};
constexpr long kPartFloats = 1L << 29;
constexpr int kSplitSteps = 8;  // steps of a lane of rows that may be split: shorter are one tile

Plan plan_of(int B, int H, int G, int N, int L, bool backward) {
  Plan p{};
  p.st = L <= 64 ? 4 : 8;
  p.rw = 8;
  const int tile = kSeg * p.st, ntile = std::max(1, (L + tile - 1) / tile), hg = H / G;
  if (p.st == 8) p.rw = 4;
  p.nrb = (hg + 4 * p.rw - 1) / (4 * p.rw);
  const long pairs = std::max(1L, (long)B * G), have = pairs * p.nrb;
  p.slab_tiles = ntile;
  p.npair = (int)pairs;
  if (backward) {
    const long least = (long)p.nrb * 2 * N * kKeep;  // a pair's in one tile: 2^27 at most
    const long most = std::min<long>(ntile, std::max(1L, kPartFloats / (pairs * least)));
    p.slab_tiles = (int)((ntile + (ntile + most - 1) / most - 1) / ((ntile + most - 1) / most));
    p.npair = (int)std::min(pairs, kPartFloats / least);
  }
  p.nslab = (ntile + p.slab_tiles - 1) / p.slab_tiles;
  const bool split = p.st == kSplitSteps && have <= 128 && p.slab_tiles >= (backward ? 4 : 8);
  const long want = split ? std::min<long>(p.slab_tiles, 512 / have) : 1;
  p.seg_tiles = (int)((p.slab_tiles + want - 1) / want);
  p.nseg = (p.slab_tiles + p.seg_tiles - 1) / p.seg_tiles;
  p.seg_parts = (p.seg_tiles + kSumTiles - 1) / kSumTiles;
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
  a.nparts = pl.nslab * pl.nseg * pl.seg_parts;
  a.seg_parts = pl.seg_parts;
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
  size_t agg, aggS, carry, bc, n, h, total;
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
    const size_t parts = (size_t)pl.nslab * pl.nseg * pl.seg_parts;
    o.carry = take(pl.nslab > 1 ? rows * N : 0);
    o.bc = take(L ? (size_t)pl.nrb * pl.npair * 2 * N * pl.slab_tiles * kKeep : 0);
    o.n = take(rows * parts * N);
    o.h = take(rows * parts * 2);
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
unsigned join_blocks(const Args& a) { return (unsigned)a.B * a.H * ((a.N + 15) / 16); }

template <typename T, int ST, int RW, int NW>
hipError_t forward(const Args& a, hipStream_t st) {
  const long blocks = (long)a.B * a.G * a.nrb * a.nseg;
  if (!launchable(blocks, 64 * RW * NW)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(64 * RW * NW);
  const size_t lds = (size_t)padded(a.N) * (2 * 4 * RW + 2) * sizeof(float);
  if constexpr (ST == kSplitSteps) {
    if (a.nseg > 1) {
      hipLaunchKernelGGL((selective_fwd_kernel<T, ST, RW, NW, true>), grid, block, lds, st, a);
      hipLaunchKernelGGL((selective_join_kernel<false>), dim3(join_blocks(a)), dim3(256), 0, st,
                         a.agg, a.aggS, a.log_re, a.x0, a.H, a.N, a.nseg);
    }
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

// A slab of the launch's pairs.
template <typename T, int ST, int RW, int NW>
hipError_t backward(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)a.npair * a.nrb * a.nseg), block(64 * RW * NW);
  const size_t lds = (size_t)padded(a.N) * (3 * 4 * RW + 4) * sizeof(float);
  if constexpr (ST == kSplitSteps) {
    if (a.nseg > 1) {
      hipLaunchKernelGGL((selective_bwd_agg_kernel<T, ST, RW>), grid, dim3(64 * RW),
                         2 * (size_t)a.N * (4 * RW + 1) * sizeof(float), st, a);
      hipLaunchKernelGGL((selective_join_kernel<true>), dim3(join_blocks(a)), dim3(256), 0, st,
                         a.agg, a.aggS, a.log_re, a.dx, a.H, a.N, a.nseg);
    }
  }
  if (a.z)
    hipLaunchKernelGGL((selective_bwd_kernel<T, ST, RW, NW, true>), grid, block, lds, st, a);
  else
    hipLaunchKernelGGL((selective_bwd_kernel<T, ST, RW, NW, false>), grid, block, lds, st, a);
  const int steps = std::min(a.L, a.tile1 * kSeg * ST) - a.tile0 * kSeg * ST;
  if (steps > 0)
    hipLaunchKernelGGL((selective_dbc_kernel<T, kSeg * ST>),
                       dim3((unsigned)a.npair * 2 * a.N * ((steps + 1023u) / 1024)), dim3(256), 0,
                       st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_backward(const SelectiveCall& c, hipStream_t st) {
  const Plan pl = plan_of(c.B, c.H, c.G, c.N, c.L, true);
  const Layout o = layout_of(pl, c.B, c.H, c.G, c.N, c.L, true);
  Args a = make_args(c, pl);
  place(a, c, o);
  float* carry = reinterpret_cast<float*>(static_cast<char*>(c.ws) + o.carry);
  const long pairs = (long)c.B * c.G;
  if (!launchable(pairs * pl.nrb * pl.nseg, 512)) return hipErrorInvalidConfiguration;
  const int tile = kSeg * pl.st, ntile = (c.L + tile - 1) / tile;
  for (long pair = 0; pair < pairs; pair += pl.npair) {
    a.pair0 = (int)pair;
    a.npair = (int)std::min<long>(pl.npair, pairs - pair);
    for (int slab = pl.nslab - 1; slab >= 0; --slab) {
      a.tile0 = slab * pl.slab_tiles;
      a.tile1 = std::min(ntile, a.tile0 + pl.slab_tiles);
      a.steps = pl.slab_tiles * kKeep;
      a.part0 = slab * pl.nseg * pl.seg_parts;
      a.dx = slab == pl.nslab - 1 ? c.dx : carry;
      a.dx0 = slab == 0 ? c.dx0 : carry;
      const hipError_t e = pl.st == 4 ? backward<T, 4, 8, 1>(a, st) : backward<T, 8, 4, 2>(a, st);
      if (e != hipSuccess) return e;
    }
  }
  hipLaunchKernelGGL(selective_param_kernel, dim3(blocks_of((long)c.H * (c.N + 2) * 16)), dim3(256),
                     0, st, a);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t step(const Args& a, int lpr, hipStream_t st) {
  const long blocks = (long)((a.B + V - 1) / V) * ((a.H * lpr + 255) / 256);
  hipLaunchKernelGGL((selective_step_kernel<T, V>), dim3((unsigned)blocks), dim3(256), 0, st, a, lpr);
  return hipGetLastError();
}

// Memory bounds many rows, and how much of it is under way: two batch rows to a lane
// from 2^20 lanes on (16 modes, bf16, one row to a lane and two: 256 x 4096 rows 33.5
// and 30.4 us, 4.7 TB/s; 64 x 4096 9.7 and 9.1; 32 x 4096 6.2 both).  Fewer are a
// launch's latency, 3.5 us, either way (replayed graphs, states warm).
template <typename T>
hipError_t run_step(const SelectiveCall& c, hipStream_t st) {
  const Args a = make_args(c, Plan{});
  int lpr = 1;
  while (lpr * 4 < c.N) lpr *= 2;
  return (long)c.B * c.H * lpr >= (1L << 20) ? step<T, 2>(a, lpr, st) : step<T, 1>(a, lpr, st);
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
