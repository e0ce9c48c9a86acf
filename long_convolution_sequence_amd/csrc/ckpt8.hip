// Activations in 8 bits: pack and unpack.  Rows of L steps, groups of 64 steps
// as int8 times a power of two (the format is described in seq_common.h).  A
// lane holds 8 steps, 8 lanes a group; both kernels only stream memory.
#include <algorithm>

#include "dssm_internal.h"
#include "seq_common.h"

namespace dssm {
namespace {

// Lane slots of a row: 8 steps each, whole groups (8 slots).
__host__ __device__ inline int row_slots(int L) { return ckpt8_groups(L) * 8; }

// I: the type slots are counted in, 32 bits where they fit (a division of 64
// bits costs more than the rest of a slot's work).
template <typename T, typename I>
__global__ __launch_bounds__(256) void pack_kernel(const T* __restrict__ x, I n, int L,
                                                   int8_t* __restrict__ q8,
                                                   uint8_t* __restrict__ e8) {
  const int slots = row_slots(L);
  const int pitch = ckpt8_row(L), groups = ckpt8_groups(L);
  // n is a multiple of 8: the lanes of a group take part together
  for (I k = (I)blockIdx.x * 256 + threadIdx.x; k < n; k += (I)gridDim.x * 256) {
    const size_t row = k / (I)slots;
    const int t = (int)(k - (I)row * (I)slots) * 8;
    const int ns = min(max(L - t, 0), 8);
    float v[8];
    load_n<T, 8>(x + row * L + t, ns, v);
    uint2 q;
    const int byte = quantise8<T, false>(v, 8, &q);
    if (ns > 0) {
      *reinterpret_cast<uint2*>(q8 + row * pitch + t) = q;
      if ((t & (kGroup - 1)) == 0) e8[row * groups + t / kGroup] = (uint8_t)byte;
    }
  }
}

template <typename T, typename I>
__global__ __launch_bounds__(256) void unpack_kernel(const int8_t* __restrict__ q8,
                                                     const uint8_t* __restrict__ e8, I n, int L,
                                                     T* __restrict__ x) {
  const int slots = (L + 7) / 8;
  const int pitch = ckpt8_row(L), groups = ckpt8_groups(L);
  for (I k = (I)blockIdx.x * 256 + threadIdx.x; k < n; k += (I)gridDim.x * 256) {
    const size_t row = k / (I)slots;
    const int t = (int)(k - (I)row * (I)slots) * 8;
    float v[8];
    dequantise8(*reinterpret_cast<const uint2*>(q8 + row * pitch + t),
                e8[row * groups + t / kGroup], v);
    store_n<T, 8>(x + row * L + t, L - t, v);
  }
}

template <typename T, typename I>
hipError_t start(const void* x, long rows, int L, long n, void* blob, void* out, hipStream_t st) {
  int8_t* q8 = static_cast<int8_t*>(blob);
  uint8_t* e8 = reinterpret_cast<uint8_t*>(blob) + ckpt8_exp_offset(rows, L);
  const dim3 grid((unsigned)std::min<long>((n + 255) / 256, 16384));
  if (out)
    hipLaunchKernelGGL((unpack_kernel<T, I>), grid, dim3(256), 0, st, q8, e8, (I)n, L,
                       static_cast<T*>(out));
  else
    hipLaunchKernelGGL((pack_kernel<T, I>), grid, dim3(256), 0, st, static_cast<const T*>(x), (I)n,
                       L, q8, e8);
  return hipGetLastError();
}

template <typename T>
hipError_t run(const void* x, long rows, int L, void* blob, void* out, hipStream_t st) {
  const long n = rows * (out ? (L + 7) / 8 : row_slots(L));
  // the loop's counter runs up to a grid past n
  return n < (1L << 31) ? start<T, uint32_t>(x, rows, L, n, blob, out, st)
                        : start<T, uint64_t>(x, rows, L, n, blob, out, st);
}

}  // namespace

hipError_t launch_ckpt8_pack(const void* x, long rows, int L, int dtype, void* blob,
                             hipStream_t st) {
  switch (dtype) {
    case 0: return run<float>(x, rows, L, blob, nullptr, st);
    case 1: return run<__bf16>(x, rows, L, blob, nullptr, st);
    default: return run<_Float16>(x, rows, L, blob, nullptr, st);
  }
}

hipError_t launch_ckpt8_unpack(const void* blob, long rows, int L, int dtype, void* x,
                               hipStream_t st) {
  void* b = const_cast<void*>(blob);
  switch (dtype) {
    case 0: return run<float>(nullptr, rows, L, b, x, st);
    case 1: return run<__bf16>(nullptr, rows, L, b, x, st);
    default: return run<_Float16>(nullptr, rows, L, b, x, st);
  }
}

}  // namespace dssm
