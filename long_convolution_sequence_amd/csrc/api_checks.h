// Argument checks shared by the host entry points of the calls that take
// activations of several types.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "../../include/dssm.h"
#include "dssm_internal.h"

namespace dssm {

constexpr int kMaxL = 1 << 24;
constexpr int kMaxH = 65535;
constexpr long kMaxRows = 1L << 24;   // workgroups of 256 lanes, four rows each at least

inline bool dtype_ok(int d) { return d == DSSM_F32 || d == DSSM_BF16 || d == DSSM_F16; }
inline size_t elem_size(int d) { return d == DSSM_F32 ? 4 : 2; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Dimensions and types common to the calls; *empty: no element at all.
inline int check_dims(const char* what, int B, int H, int L, int dtype, bool* empty) {
  if (B < 0 || H < 0 || L < 0)
    return fail(DSSM_ERR_INVALID_ARG, "%s: negative dimension (B=%d H=%d L=%d)", what, B, H, L);
  if (!dtype_ok(dtype))
    return fail(DSSM_ERR_INVALID_ARG, "%s: dtype must be DSSM_F32, DSSM_BF16 or DSSM_F16, got %d",
                what, dtype);
  if (H > kMaxH) return fail(DSSM_ERR_UNSUPPORTED, "%s: H=%d exceeds %d", what, H, kMaxH);
  if (L > kMaxL) return fail(DSSM_ERR_UNSUPPORTED, "%s: L=%d exceeds %d", what, L, kMaxL);
  // B H < 2^47 and L <= 2^24: the product cannot wrap
  if ((__int128)B * H * L > ((__int128)1 << 40))
    return fail(DSSM_ERR_UNSUPPORTED, "%s: B*H*L exceeds 2^40", what);
  *empty = B == 0 || H == 0 || L == 0;
  return DSSM_OK;
}

struct Named {
  const void* p;
  const char* name;
};

// Every pointer set and aligned to its element.
inline int check_ptrs(std::initializer_list<Named> list, size_t align) {
  for (const Named& n : list) {
    if (!n.p) return fail(DSSM_ERR_INVALID_ARG, "%s is NULL", n.name);
    if (!aligned(n.p, align))
      return fail(DSSM_ERR_INVALID_ARG, "%s is not aligned to %zu bytes", n.name, align);
  }
  return DSSM_OK;
}

inline int check_opt(const void* p, const char* name, size_t align) {
  if (p && !aligned(p, align))
    return fail(DSSM_ERR_INVALID_ARG, "%s is not aligned to %zu bytes", name, align);
  return DSSM_OK;
}

// No output is an input or another output.
inline int check_alias(std::initializer_list<Named> outs, std::initializer_list<Named> ins) {
  for (auto a = outs.begin(); a != outs.end(); ++a) {
    if (!a->p) continue;
    for (const Named& b : ins)
      if (a->p == b.p)
        return fail(DSSM_ERR_INVALID_ARG, "%s must not alias %s", a->name, b.name);
    for (auto b = outs.begin(); b != a; ++b)
      if (a->p == b->p)
        return fail(DSSM_ERR_INVALID_ARG, "%s must not alias %s", a->name, b->name);
  }
  return DSSM_OK;
}

inline int check_stride(long long stride, const char* name, int B, int H, int L) {
  if (B > 1 && stride < (long long)H * L)
    return fail(DSSM_ERR_INVALID_ARG, "%s=%lld is below H*L=%lld", name, stride,
                (long long)H * L);
  if (B > 1 && stride > (1LL << 40))
    return fail(DSSM_ERR_UNSUPPORTED, "%s=%lld exceeds 2^40", name, stride);
  return DSSM_OK;
}

inline int check_buffer(const void* p, const char* name) {
  if (!p) return fail(DSSM_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 256)) return fail(DSSM_ERR_INVALID_ARG, "%s must be 256-byte aligned", name);
  return DSSM_OK;
}

inline int check_space(const void* ws, size_t have, size_t need) {
  if (have < need)
    return fail(DSSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", have,
                need);
  return need ? check_buffer(ws, "workspace") : DSSM_OK;
}

// A launch that the launcher refuses to make: its grid has too many lanes.
inline int launch_check(hipError_t e, const char* what) {
  if (e == hipErrorInvalidConfiguration)
    return fail(DSSM_ERR_UNSUPPORTED, "%s: a grid of 2^32 lanes or more", what);
  return hip_check(e, what);
}

}  // namespace dssm
