// Host entry points of the short convolution and the selective scan: argument
// validation and launches on the caller's stream.
#include "../../include/dssm.h"
#include "api_checks.h"
#include "dssm_internal.h"

using namespace dssm;

namespace {

int check_shortconv(const dssm_shortconv_shape* s, bool* empty) {
  if (!s) return fail(DSSM_ERR_INVALID_ARG, "shape is NULL");
  if (int rc = check_dims("shortconv", s->B, s->H, s->L, s->dtype, empty)) return rc;
  if (s->K < 1) return fail(DSSM_ERR_INVALID_ARG, "shortconv: K=%d is below 1", s->K);
  if (s->K > kShortconvTaps)
    return fail(DSSM_ERR_UNSUPPORTED, "shortconv: K=%d exceeds %d", s->K, kShortconvTaps);
  if (s->act != DSSM_ACT_NONE && s->act != DSSM_ACT_SILU)
    return fail(DSSM_ERR_INVALID_ARG, "act must be DSSM_ACT_NONE or DSSM_ACT_SILU, got %d", s->act);
  if ((long)s->B * s->H > kMaxRows)
    return fail(DSSM_ERR_UNSUPPORTED, "shortconv: B*H=%ld exceeds 2^24", (long)s->B * s->H);
  return DSSM_OK;
}

// Inputs and parameters of either direction.
int check_shortconv_in(const void* u, long long stride_b, const float* w, const float* bias,
                       const dssm_shortconv_shape* s, const int* lens, const float* x0,
                       bool reads) {
  int rc;
  if ((rc = check_ptrs({{w, "w"}}, 4)) || (rc = check_opt(bias, "bias", 4)) ||
      (rc = check_opt(lens, "lens", 4)) || (rc = check_opt(x0, "x0", 4)))
    return rc;
  if (!reads) return DSSM_OK;
  if ((rc = check_ptrs({{u, "u"}}, elem_size(s->dtype)))) return rc;
  return check_stride(stride_b, "stride_b", s->B, s->H, s->L);
}

ShortconvCall shortconv_call(const void* u, long long stride_b, const float* w, const float* bias,
                             const dssm_shortconv_shape* s, const int* lens, const float* x0) {
  ShortconvCall c{};
  c.u = u;
  c.stride_b = stride_b;
  c.w = w;
  c.bias = bias;
  c.lens = lens;
  c.B = s->B;
  c.H = s->H;
  c.L = s->L;
  c.K = s->K;
  c.silu = s->act == DSSM_ACT_SILU;
  c.x0 = x0;
  return c;
}

int shortconv_run(bool step, const void* u, long long stride_b, const float* w, const float* bias,
                  const dssm_shortconv_shape* s, const int* lens, const float* x0, float* x_end,
                  void* y, void* stream) {
  bool empty = false;
  int rc = check_shortconv(s, &empty);
  if (rc) return rc;
  if (step && s->L != 1)
    return fail(DSSM_ERR_INVALID_ARG, "dssm_shortconv_step takes one time step (L must be 1, got %d)",
                s->L);
  if (s->B == 0 || s->H == 0) return ok();
  // with L = 0 only the state passes through
  if ((rc = check_shortconv_in(u, stride_b, w, bias, s, lens, x0, !empty)) ||
      (rc = check_opt(x_end, "x_end", 4)))
    return rc;
  if (!empty) {
    if ((rc = check_ptrs({{y, "y"}}, elem_size(s->dtype))) ||
        (rc = check_alias({{y, "y"}, {x_end, "x_end"}},
                          {{u, "u"}, {w, "w"}, {bias, "bias"}, {lens, "lens"}})))
      return rc;
    if (x0 && y == x0) return fail(DSSM_ERR_INVALID_ARG, "y must not alias x0");
  }
  ShortconvCall c = shortconv_call(u, stride_b, w, bias, s, lens, x0);
  c.xT = x_end;
  c.y = y;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if ((rc = launch_check(step ? launch_shortconv_step(c, s->dtype, st)
                              : launch_shortconv_forward(c, s->dtype, st),
                         "shortconv launch")))
    return rc;
  return ok();
}

int check_selective(const dssm_selective_shape* s, bool* empty) {
  if (!s) return fail(DSSM_ERR_INVALID_ARG, "shape is NULL");
  if (int rc = check_dims("selective", s->B, s->H, s->L, s->dtype, empty)) return rc;
  if (s->N < 1) return fail(DSSM_ERR_INVALID_ARG, "selective: N=%d is below 1", s->N);
  if (s->N > kSelectiveModes)
    return fail(DSSM_ERR_UNSUPPORTED, "selective: N=%d exceeds %d", s->N, kSelectiveModes);
  if (s->G < 1 || s->H % s->G)
    return fail(DSSM_ERR_INVALID_ARG, "selective: H=%d is not a multiple of G=%d", s->H, s->G);
  if ((long)s->B * s->H > kMaxRows)
    return fail(DSSM_ERR_UNSUPPORTED, "selective: B*H=%ld exceeds 2^24", (long)s->B * s->H);
  if ((__int128)s->B * s->H * s->N * ((s->L + 127) / 128) > ((__int128)1 << 36))
    return fail(DSSM_ERR_UNSUPPORTED, "selective: B*H*N*ceil(L/128) exceeds 2^36");
  // parts of 1024 steps of the modes' B and C gradients, numbered in 32 bits
  if ((__int128)s->B * s->G * s->N * ((s->L + 1023) / 1024) > ((__int128)1 << 29))
    return fail(DSSM_ERR_UNSUPPORTED, "selective: B*G*N*ceil(L/1024) exceeds 2^29");
  return DSSM_OK;
}

int check_selective_in(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                       bool reads) {
  if (!in) return fail(DSSM_ERR_INVALID_ARG, "inputs is NULL");
  const size_t e = elem_size(s->dtype);
  int rc;
  if ((rc = check_ptrs({{in->log_re, "log_re"}}, 4)) || (rc = check_opt(in->D, "D", 4)) ||
      (rc = check_opt(in->dt_bias, "dt_bias", 4)) || (rc = check_opt(in->lens, "lens", 4)))
    return rc;
  if (!reads) return DSSM_OK;
  if ((rc = check_ptrs({{in->u, "u"}, {in->delta, "delta"}, {in->Bm, "Bm"}, {in->Cm, "Cm"}}, e)) ||
      (rc = check_opt(in->z, "z", e)) ||
      (rc = check_stride(in->stride_u, "stride_u", s->B, s->H, s->L)) ||
      (rc = check_stride(in->stride_delta, "stride_delta", s->B, s->H, s->L)) ||
      (in->z && (rc = check_stride(in->stride_z, "stride_z", s->B, s->H, s->L))) ||
      (rc = check_stride(in->stride_B, "stride_B", s->B, s->G * s->N, s->L)) ||
      (rc = check_stride(in->stride_C, "stride_C", s->B, s->G * s->N, s->L)))
    return rc;
  return DSSM_OK;
}

SelectiveCall selective_call(const dssm_selective_inputs* in, const dssm_selective_shape* s) {
  SelectiveCall c{};
  c.u = in->u;
  c.delta = in->delta;
  c.z = in->z;
  c.Bm = in->Bm;
  c.Cm = in->Cm;
  c.stride_u = in->stride_u;
  c.stride_delta = in->stride_delta;
  c.stride_z = in->stride_z;
  c.stride_B = in->stride_B;
  c.stride_C = in->stride_C;
  c.log_re = in->log_re;
  c.D = in->D;
  c.dt_bias = in->dt_bias;
  c.lens = in->lens;
  c.B = s->B;
  c.H = s->H;
  c.G = s->G;
  c.N = s->N;
  c.L = s->L;
  return c;
}

// The checks of the forward calls (a sequence or one token) that both share.
int check_selective_forward(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                            const float* x0, const float* x_end, const void* y, bool reads) {
  int rc;
  if ((rc = check_selective_in(in, s, reads)) || (rc = check_opt(x0, "x0", 4)) ||
      (rc = check_opt(x_end, "x_end", 4)))
    return rc;
  if (!reads) return DSSM_OK;
  if ((rc = check_ptrs({{y, "y"}}, elem_size(s->dtype))) ||
      (rc = check_alias({{y, "y"}, {x_end, "x_end"}},
                        {{in->u, "u"}, {in->delta, "delta"}, {in->z, "z"}, {in->Bm, "Bm"},
                         {in->Cm, "Cm"}, {in->log_re, "log_re"}, {in->D, "D"},
                         {in->dt_bias, "dt_bias"}, {in->lens, "lens"}})))
    return rc;
  return x0 && y == x0 ? fail(DSSM_ERR_INVALID_ARG, "y must not alias x0") : DSSM_OK;
}

}  // namespace

extern "C" {

int dssm_shortconv_forward(const void* u, long long stride_b, const float* w, const float* bias,
                           const dssm_shortconv_shape* s, const int* lens, const float* x0,
                           float* x_end, void* y, void* stream) {
  return shortconv_run(false, u, stride_b, w, bias, s, lens, x0, x_end, y, stream);
}

int dssm_shortconv_step(const void* u, long long stride_b, const float* w, const float* bias,
                        const dssm_shortconv_shape* s, const int* lens, const float* x0,
                        float* x_end, void* y, void* stream) {
  return shortconv_run(true, u, stride_b, w, bias, s, lens, x0, x_end, y, stream);
}

int dssm_shortconv_workspace_size(const dssm_shortconv_shape* s, size_t* bytes) {
  if (!bytes) return fail(DSSM_ERR_INVALID_ARG, "bytes is NULL");
  bool empty = false;
  if (int rc = check_shortconv(s, &empty)) return rc;
  *bytes = s->B == 0 || s->H == 0 ? 0 : shortconv_workspace(s->B, s->H, s->K, s->L);
  return ok();
}

int dssm_shortconv_backward(const void* u, long long stride_b, const float* w, const float* bias,
                            const dssm_shortconv_shape* s, const int* lens, const float* x0,
                            const void* dy, const float* dx_end, const dssm_shortconv_grads* g,
                            void* ws, size_t ws_bytes, void* stream) {
  bool empty = false;
  int rc = check_shortconv(s, &empty);
  if (rc) return rc;
  if (s->H == 0) return ok();
  if (!g) return fail(DSSM_ERR_INVALID_ARG, "grads is NULL");
  if ((rc = check_shortconv_in(u, stride_b, w, bias, s, lens, x0, !empty)) ||
      (rc = check_opt(dx_end, "dx_end", 4)) || (rc = check_ptrs({{g->dw, "dw"}}, 4)) ||
      (rc = check_opt(g->dbias, "dbias", 4)) || (rc = check_opt(g->dx0, "dx0", 4)))
    return rc;
  const size_t e = elem_size(s->dtype);
  if (!empty && ((rc = check_ptrs({{dy, "dy"}, {g->du, "du"}}, e)) ||
                 (rc = check_stride(g->stride_b, "the gradient's stride_b", s->B, s->H, s->L))))
    return rc;
  const size_t need = s->B == 0 ? 0 : shortconv_workspace(s->B, s->H, s->K, s->L);
  if ((rc = check_space(ws, ws_bytes, need))) return rc;
  if ((rc = check_alias({{empty ? nullptr : g->du, "du"}, {g->dw, "dw"}, {g->dbias, "dbias"},
                         {g->dx0, "dx0"}, {need ? ws : nullptr, "workspace"}},
                        {{u, "u"}, {w, "w"}, {bias, "bias"}, {lens, "lens"}, {x0, "x0"}, {dy, "dy"},
                         {dx_end, "dx_end"}})))
    return rc;
  ShortconvCall c = shortconv_call(u, stride_b, w, bias, s, lens, x0);
  c.dy = dy;
  c.dx = dx_end;
  c.du = g->du;
  c.grad_stride_b = g->stride_b;
  c.dw = g->dw;
  c.dbias = g->dbias;
  c.dx0 = g->dx0;
  c.ws = ws;
  if ((rc = launch_check(launch_shortconv_backward(c, s->dtype, static_cast<hipStream_t>(stream)),
                         "shortconv backward launch")))
    return rc;
  return ok();
}

int dssm_selective_workspace_size(const dssm_selective_shape* s, int backward, size_t* bytes) {
  if (!bytes) return fail(DSSM_ERR_INVALID_ARG, "bytes is NULL");
  bool empty = false;
  if (int rc = check_selective(s, &empty)) return rc;
  *bytes = s->B == 0 || s->H == 0
               ? 0
               : selective_workspace(s->B, s->H, s->G, s->N, s->L, backward != 0);
  return ok();
}

int dssm_selective_ckpt_size(const dssm_selective_shape* s, size_t* bytes) {
  if (!bytes) return fail(DSSM_ERR_INVALID_ARG, "bytes is NULL");
  bool empty = false;
  if (int rc = check_selective(s, &empty)) return rc;
  *bytes = empty ? 0 : selective_ckpt(s->B, s->H, s->N, s->L);
  return ok();
}

int dssm_selective_forward(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                           const float* x0, float* x_end, void* y, void* ckpt, void* ws,
                           size_t ws_bytes, void* stream) {
  bool empty = false;
  int rc = check_selective(s, &empty);
  if (rc) return rc;
  if (s->B == 0 || s->H == 0) return ok();
  // with L = 0 only the state passes through
  if ((rc = check_selective_forward(in, s, x0, x_end, y, !empty))) return rc;
  if (empty) ckpt = nullptr;
  if (ckpt && (rc = check_buffer(ckpt, "ckpt"))) return rc;
  const size_t need = selective_workspace(s->B, s->H, s->G, s->N, s->L, false);
  if ((rc = check_space(ws, ws_bytes, need))) return rc;
  if (!empty && (rc = check_alias({{ckpt, "ckpt"}, {need ? ws : nullptr, "workspace"}},
                                  {{in->u, "u"}, {in->delta, "delta"}, {in->z, "z"},
                                   {in->Bm, "Bm"}, {in->Cm, "Cm"}, {in->log_re, "log_re"},
                                   {in->D, "D"}, {in->dt_bias, "dt_bias"}, {in->lens, "lens"},
                                   {x0, "x0"}, {x_end, "x_end"}, {y, "y"}})))
    return rc;
  SelectiveCall c = selective_call(in, s);
  c.x0 = x0;
  c.xT = x_end;
  c.y = y;
  c.ckpt = ckpt;
  c.ws = ws;
  if ((rc = launch_check(launch_selective_forward(c, s->dtype, static_cast<hipStream_t>(stream)),
                         "selective forward launch")))
    return rc;
  return ok();
}

int dssm_selective_step(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                        const float* x0, float* x_end, void* y, void* stream) {
  bool empty = false;
  int rc = check_selective(s, &empty);
  if (rc) return rc;
  if (s->L != 1)
    return fail(DSSM_ERR_INVALID_ARG,
                "dssm_selective_step takes one time step (L must be 1, got %d)", s->L);
  if (empty) return ok();
  if ((rc = check_selective_forward(in, s, x0, x_end, y, true))) return rc;
  SelectiveCall c = selective_call(in, s);
  c.x0 = x0;
  c.xT = x_end;
  c.y = y;
  if ((rc = launch_check(launch_selective_step(c, s->dtype, static_cast<hipStream_t>(stream)),
                         "selective step launch")))
    return rc;
  return ok();
}

int dssm_selective_backward(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                            const void* ckpt, const void* dy, const float* dx_end,
                            const dssm_selective_grads* g, void* ws, size_t ws_bytes,
                            void* stream) {
  bool empty = false;
  int rc = check_selective(s, &empty);
  if (rc) return rc;
  if (s->H == 0) return ok();
  if ((rc = check_selective_in(in, s, !empty))) return rc;
  if (!g) return fail(DSSM_ERR_INVALID_ARG, "grads is NULL");
  if ((rc = check_ptrs({{g->dlog_re, "dlog_re"}}, 4)) || (rc = check_opt(g->dx0, "dx0", 4)) ||
      (rc = check_opt(dx_end, "dx_end", 4)) ||
      (in->D && (rc = check_ptrs({{g->dD, "dD"}}, 4))) ||
      (in->dt_bias && (rc = check_ptrs({{g->ddt_bias, "ddt_bias"}}, 4))))
    return rc;
  if (!in->D && g->dD) return fail(DSSM_ERR_INVALID_ARG, "dD needs D");
  if (!in->dt_bias && g->ddt_bias) return fail(DSSM_ERR_INVALID_ARG, "ddt_bias needs dt_bias");
  const size_t e = elem_size(s->dtype);
  const void* dz = empty ? nullptr : g->dz;
  if (!empty) {
    const int H = s->H, GN = s->G * s->N;
    if ((rc = check_buffer(ckpt, "ckpt")) ||
        (rc = check_ptrs({{dy, "dy"}, {g->du, "du"}, {g->ddelta, "ddelta"}, {g->dB, "dB"},
                          {g->dC, "dC"}}, e)) ||
        (in->z && (rc = check_ptrs({{dz, "dz"}}, e))) ||
        (rc = check_stride(g->stride_u, "the gradient's stride_u", s->B, H, s->L)) ||
        (rc = check_stride(g->stride_delta, "the gradient's stride_delta", s->B, H, s->L)) ||
        (in->z && (rc = check_stride(g->stride_z, "the gradient's stride_z", s->B, H, s->L))) ||
        (rc = check_stride(g->stride_B, "the gradient's stride_B", s->B, GN, s->L)) ||
        (rc = check_stride(g->stride_C, "the gradient's stride_C", s->B, GN, s->L)))
      return rc;
    if (!in->z && dz) return fail(DSSM_ERR_INVALID_ARG, "dz needs z");
  }
  const size_t need = s->B == 0 ? 0 : selective_workspace(s->B, s->H, s->G, s->N, s->L, true);
  if ((rc = check_space(ws, ws_bytes, need))) return rc;
  const void* none = nullptr;
  if ((rc = check_alias(
           {{empty ? none : g->du, "du"}, {empty ? none : g->ddelta, "ddelta"}, {dz, "dz"},
            {empty ? none : g->dB, "dB"}, {empty ? none : g->dC, "dC"}, {g->dlog_re, "dlog_re"},
            {g->dD, "dD"}, {g->ddt_bias, "ddt_bias"}, {g->dx0, "dx0"},
            {need ? ws : none, "workspace"}},
           {{in->u, "u"}, {in->delta, "delta"}, {in->z, "z"}, {in->Bm, "Bm"}, {in->Cm, "Cm"},
            {in->log_re, "log_re"}, {in->D, "D"}, {in->dt_bias, "dt_bias"}, {in->lens, "lens"},
            {ckpt, "ckpt"}, {dy, "dy"}, {dx_end, "dx_end"}})))
    return rc;
  SelectiveCall c = selective_call(in, s);
  c.ckpt = const_cast<void*>(ckpt);
  c.dy = dy;
  c.dx = dx_end;
  c.du = g->du;
  c.ddelta = g->ddelta;
  c.dz = g->dz;
  c.dB = g->dB;
  c.dC = g->dC;
  c.stride_du = g->stride_u;
  c.stride_ddelta = g->stride_delta;
  c.stride_dz = g->stride_z;
  c.stride_dB = g->stride_B;
  c.stride_dC = g->stride_C;
  c.dlog_re = g->dlog_re;
  c.dD = g->dD;
  c.ddt_bias = g->ddt_bias;
  c.dx0 = g->dx0;
  c.ws = ws;
  if ((rc = launch_check(launch_selective_backward(c, s->dtype, static_cast<hipStream_t>(stream)),
                         "selective backward launch")))
    return rc;
  return ok();
}

}  // extern "C"
