// Host entry points of the gated recurrence, the 8-bit checkpoints and the
// residual norm: argument validation and launches on the caller's stream.
#include <cmath>
#include <cstdint>

#include "../../include/dssm.h"
#include "api_checks.h"
#include "dssm_internal.h"

using namespace dssm;

namespace {

constexpr long kMaxStrips = 1L << 21; // workgroups of up to 1024 lanes

int check_gated(const dssm_gated_shape* s, bool* empty) {
  if (!s) return fail(DSSM_ERR_INVALID_ARG, "shape is NULL");
  if (int rc = check_dims("gated", s->B, s->H, s->L, s->dtype, empty)) return rc;
  if ((long)s->B * s->H > kMaxRows)
    return fail(DSSM_ERR_UNSUPPORTED, "gated: B*H=%ld exceeds 2^24", (long)s->B * s->H);
  return DSSM_OK;
}

GatedCall gated_call(const dssm_gated_inputs* in, const dssm_gated_shape* s) {
  GatedCall c{};
  c.u = in->u;
  c.r = in->r;
  c.i = in->i;
  c.stride_b = in->stride_b;
  c.log_re = in->log_re;
  c.lens = in->lens;
  c.B = s->B;
  c.H = s->H;
  c.L = s->L;
  return c;
}

// The checks of the forward calls (a sequence or one token).
int check_forward(const dssm_gated_inputs* in, const dssm_gated_shape* s, const float* x0,
                  const float* x_end, const void* y, bool reads) {
  if (!in) return fail(DSSM_ERR_INVALID_ARG, "inputs is NULL");
  const size_t e = elem_size(s->dtype);
  int rc;
  if ((rc = check_opt(x0, "x0", 4)) || (rc = check_opt(x_end, "x_end", 4)) ||
      (rc = check_ptrs({{in->log_re, "log_re"}}, 4)) || (rc = check_opt(in->lens, "lens", 4)))
    return rc;
  if (!reads) return DSSM_OK;
  if ((rc = check_ptrs({{in->u, "u"}, {in->r, "r"}, {in->i, "i"}, {y, "y"}}, e)) ||
      (rc = check_stride(in->stride_b, "stride_b", s->B, s->H, s->L)))
    return rc;
  if ((rc = check_alias({{y, "y"}, {x_end, "x_end"}},
                        {{in->u, "u"}, {in->r, "r"}, {in->i, "i"}, {in->log_re, "log_re"}})))
    return rc;
  return x0 && y == x0 ? fail(DSSM_ERR_INVALID_ARG, "y must not alias x0") : DSSM_OK;
}

}  // namespace

extern "C" {

int dssm_gated_workspace_size(const dssm_gated_shape* s, size_t* bytes) {
  if (!bytes) return fail(DSSM_ERR_INVALID_ARG, "bytes is NULL");
  bool empty = false;
  if (int rc = check_gated(s, &empty)) return rc;
  *bytes = s->B == 0 || s->H == 0 ? 0 : gated_workspace(s->B, s->H, s->L);
  return ok();
}

static int check_kind(int kind, bool none) {
  if (kind == DSSM_CKPT_STATE || kind == DSSM_CKPT_INT8 || (none && kind == DSSM_CKPT_NONE))
    return DSSM_OK;
  return fail(DSSM_ERR_INVALID_ARG, "kind must be %sDSSM_CKPT_STATE or DSSM_CKPT_INT8, got %d",
              none ? "DSSM_CKPT_NONE, " : "", kind);
}

int dssm_gated_ckpt_size(const dssm_gated_shape* s, int kind, size_t* bytes) {
  if (!bytes) return fail(DSSM_ERR_INVALID_ARG, "bytes is NULL");
  bool empty = false;
  if (int rc = check_gated(s, &empty)) return rc;
  if (int rc = check_kind(kind, true)) return rc;
  *bytes = empty || kind == DSSM_CKPT_NONE
               ? 0
               : gated_ckpt_layout((long)s->B * s->H, s->L, kind).total;
  return ok();
}

int dssm_gated_forward(const dssm_gated_inputs* in, const dssm_gated_shape* s, const float* x0,
                       float* x_end, void* y, int kind, void* ckpt, void* ws, size_t ws_bytes,
                       void* stream) {
  bool empty = false;
  int rc = check_gated(s, &empty);
  if (rc) return rc;
  if ((rc = check_kind(kind, true))) return rc;
  if (s->B == 0 || s->H == 0) return ok();
  // with L = 0 only the state passes through
  if ((rc = check_forward(in, s, x0, x_end, y, !empty))) return rc;
  if (!empty && kind != DSSM_CKPT_NONE && (rc = check_buffer(ckpt, "ckpt"))) return rc;
  if ((rc = check_space(ws, ws_bytes, gated_workspace(s->B, s->H, s->L)))) return rc;
  if (!empty) {
    const void* kept = kind == DSSM_CKPT_NONE ? nullptr : ckpt;
    const std::initializer_list<Named> rest = {
        {in->u, "u"}, {in->r, "r"},       {in->i, "i"}, {in->log_re, "log_re"},
        {x0, "x0"},   {x_end, "x_end"}, {y, "y"},     {in->lens, "lens"}};
    if ((rc = check_alias({{kept, "ckpt"}, {ws, "workspace"}}, rest))) return rc;
  }
  GatedCall c = gated_call(in, s);
  c.x0 = x0;
  c.xT = x_end;
  c.y = y;
  c.kind = kind;
  c.ckpt = kind == DSSM_CKPT_NONE ? nullptr : ckpt;
  c.ws = ws;
  if ((rc = hip_check(launch_gated_forward(c, s->dtype, static_cast<hipStream_t>(stream)),
                      "gated forward launch")))
    return rc;
  return ok();
}

int dssm_gated_step(const dssm_gated_inputs* in, const dssm_gated_shape* s, const float* x0,
                    float* x_end, void* y, void* stream) {
  if (!s) return fail(DSSM_ERR_INVALID_ARG, "shape is NULL");
  bool empty = false;
  int rc = check_dims("gated step", s->B, s->H, s->L, s->dtype, &empty);
  if (rc) return rc;
  if (s->L != 1)
    return fail(DSSM_ERR_INVALID_ARG, "dssm_gated_step takes one time step (L must be 1, got %d)",
                s->L);
  if ((long)s->B * s->H > (long)INT32_MAX)
    return fail(DSSM_ERR_UNSUPPORTED, "gated step: B*H exceeds 2^31 - 1");
  if (empty) return ok();
  if ((rc = check_forward(in, s, x0, x_end, y, true))) return rc;
  GatedCall c = gated_call(in, s);
  c.x0 = x0;
  c.xT = x_end;
  c.y = y;
  if ((rc = hip_check(launch_gated_step(c, s->dtype, static_cast<hipStream_t>(stream)),
                      "gated step launch")))
    return rc;
  return ok();
}

int dssm_gated_backward(const dssm_gated_inputs* in, const dssm_gated_shape* s, int kind,
                        const void* ckpt, const void* dy, const float* dx_end,
                        const dssm_gated_grads* g, void* ws, size_t ws_bytes, void* stream) {
  bool empty = false;
  int rc = check_gated(s, &empty);
  if (rc) return rc;
  if ((rc = check_kind(kind, false))) return rc;
  if (s->H == 0) return ok();
  if (!in) return fail(DSSM_ERR_INVALID_ARG, "inputs is NULL");
  if (!g) return fail(DSSM_ERR_INVALID_ARG, "grads is NULL");
  const size_t e = elem_size(s->dtype);
  if ((rc = check_ptrs({{in->log_re, "log_re"}, {g->dlog_re, "dlog_re"}}, 4)) ||
      (rc = check_opt(g->dx0, "dx0", 4)) || (rc = check_opt(dx_end, "dx_end", 4)) ||
      (rc = check_opt(in->lens, "lens", 4)))
    return rc;
  const bool reads = kind == DSSM_CKPT_STATE;
  if (!empty) {
    if (reads && ((rc = check_ptrs({{in->u, "u"}, {in->r, "r"}, {in->i, "i"}}, e)) ||
                  (rc = check_stride(in->stride_b, "stride_b", s->B, s->H, s->L))))
      return rc;
    if ((rc = check_buffer(ckpt, "ckpt")) ||
        (rc = check_ptrs({{dy, "dy"}, {g->du, "du"}, {g->dr, "dr"}, {g->di, "di"}}, e)) ||
        (rc = check_stride(g->stride_b, "the gradients' stride_b", s->B, s->H, s->L)) ||
        (rc = check_alias({{g->du, "du"}, {g->dr, "dr"}, {g->di, "di"}, {g->dlog_re, "dlog_re"},
                           {g->dx0, "dx0"}},
                          {{dy, "dy"}, {ckpt, "ckpt"}, {in->log_re, "log_re"}, {dx_end, "dx_end"},
                           {reads ? in->u : dy, "u"}, {reads ? in->r : dy, "r"},
                           {reads ? in->i : dy, "i"}})))
      return rc;
  }
  if (s->B > 0 && (rc = check_space(ws, ws_bytes, gated_workspace(s->B, s->H, s->L)))) return rc;
  if (!empty &&
      (rc = check_alias({{ws, "workspace"}},
                        {{ckpt, "ckpt"}, {dy, "dy"}, {g->du, "du"}, {g->dr, "dr"}, {g->di, "di"},
                         {g->dlog_re, "dlog_re"}, {g->dx0, "dx0"}, {in->log_re, "log_re"},
                         {dx_end, "dx_end"}, {in->lens, "lens"}, {reads ? in->u : dy, "u"},
                         {reads ? in->r : dy, "r"}, {reads ? in->i : dy, "i"}})))
    return rc;
  GatedCall c = gated_call(in, s);
  c.kind = kind;
  c.ckpt = empty ? nullptr : const_cast<void*>(ckpt);
  c.dy = dy;
  c.dx = dx_end;
  c.du = g->du;
  c.dr = g->dr;
  c.di = g->di;
  c.grad_stride_b = g->stride_b;
  c.dlog_re = g->dlog_re;
  c.dx0 = g->dx0;
  c.ws = ws;
  if ((rc = hip_check(launch_gated_backward(c, s->dtype, static_cast<hipStream_t>(stream)),
                      "gated backward launch")))
    return rc;
  return ok();
}

static int check_ckpt8(long long rows, int L) {
  if (rows < 0 || L < 0)
    return fail(DSSM_ERR_INVALID_ARG, "negative dimension (rows=%lld L=%d)", rows, L);
  if (L > kMaxL) return fail(DSSM_ERR_UNSUPPORTED, "L=%d exceeds %d", L, kMaxL);
  if ((__int128)rows * (L > 0 ? L : 1) > ((__int128)1 << 40))
    return fail(DSSM_ERR_UNSUPPORTED, "rows*L exceeds 2^40");
  return DSSM_OK;
}

int dssm_ckpt8_size(long long rows, int L, size_t* bytes) {
  if (!bytes) return fail(DSSM_ERR_INVALID_ARG, "bytes is NULL");
  if (int rc = check_ckpt8(rows, L)) return rc;
  *bytes = rows == 0 || L == 0 ? 0 : ckpt8_bytes((long)rows, L);
  return ok();
}

static int ckpt8_run(bool pack, const void* from, long long rows, int L, int dtype, void* to,
                     void* stream) {
  int rc = check_ckpt8(rows, L);
  if (rc) return rc;
  if (!dtype_ok(dtype)) return fail(DSSM_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows == 0 || L == 0) return ok();
  const void* x = pack ? from : to;
  const void* blob = pack ? to : from;
  if ((rc = check_ptrs({{x, "x"}}, elem_size(dtype))) || (rc = check_buffer(blob, "blob")))
    return rc;
  if (x == blob) return fail(DSSM_ERR_INVALID_ARG, "x must not alias blob");
  hipStream_t st = static_cast<hipStream_t>(stream);
  if ((rc = hip_check(pack ? launch_ckpt8_pack(from, (long)rows, L, dtype, to, st)
                           : launch_ckpt8_unpack(from, (long)rows, L, dtype, to, st),
                      "ckpt8 launch")))
    return rc;
  return ok();
}

int dssm_ckpt8_pack(const void* x, long long rows, int L, int dtype, void* blob, void* stream) {
  return ckpt8_run(true, x, rows, L, dtype, blob, stream);
}

int dssm_ckpt8_unpack(const void* blob, long long rows, int L, int dtype, void* x, void* stream) {
  return ckpt8_run(false, blob, rows, L, dtype, x, stream);
}

static int check_resnorm(const dssm_resnorm_shape* s, bool* empty) {
  if (!s) return fail(DSSM_ERR_INVALID_ARG, "shape is NULL");
  if (int rc = check_dims("resnorm", s->B, s->H, s->L, s->dtype, empty)) return rc;
  if (s->norm != DSSM_NORM_RMS && s->norm != DSSM_NORM_LAYER)
    return fail(DSSM_ERR_INVALID_ARG, "norm must be DSSM_NORM_RMS or DSSM_NORM_LAYER, got %d",
                s->norm);
  if (!(s->eps >= 0.f) || std::isinf(s->eps))
    return fail(DSSM_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (s->H > kResnormMaxH)
    return fail(DSSM_ERR_UNSUPPORTED, "resnorm: H=%d exceeds %d", s->H, kResnormMaxH);
  if (s->L > kResnormMaxL)
    return fail(DSSM_ERR_UNSUPPORTED, "resnorm: L=%d exceeds %d", s->L, kResnormMaxL);
  // strips of eight steps at least
  if ((long)s->B * ((s->L + 7) / 8) > kMaxStrips)
    return fail(DSSM_ERR_UNSUPPORTED, "resnorm: B*ceil(L/8)=%ld exceeds 2^21",
                (long)s->B * ((s->L + 7) / 8));
  return DSSM_OK;
}

static ResnormCall resnorm_call(const void* x, const void* y, const void* g, long long stride_g,
                                const dssm_resnorm_params* p, const dssm_resnorm_shape* s,
                                const int* lens) {
  ResnormCall c{};
  c.x = x;
  c.y = y;
  c.g = y ? g : nullptr;
  c.stride_g = stride_g;
  c.w_post = p->w_post;
  c.scale = p->scale;
  c.w_pre = p->w_pre;
  c.lens = lens;
  c.B = s->B;
  c.H = s->H;
  c.L = s->L;
  c.layer = s->norm == DSSM_NORM_LAYER;
  c.eps = s->eps;
  return c;
}

// Inputs and parameters of either call: y's and g's parts only with y, n's
// weight only where n takes part.
static int check_resnorm_in(const void* x, const char* xname, const void* y, const void* g,
                            long long stride_g, const dssm_resnorm_params* p,
                            const dssm_resnorm_shape* s, const int* lens, bool with_n) {
  const size_t e = elem_size(s->dtype);
  int rc;
  if (!p) return fail(DSSM_ERR_INVALID_ARG, "params is NULL");
  if (!y && g) return fail(DSSM_ERR_INVALID_ARG, "a gate needs y");
  if ((rc = check_ptrs({{x, xname}}, e)) || (rc = check_opt(y, "y", e)) ||
      (rc = check_opt(g, "g", e)) || (rc = check_opt(lens, "lens", 4)))
    return rc;
  if (g && (rc = check_stride(stride_g, "stride_g", s->B, s->H, s->L))) return rc;
  if (y && (rc = check_ptrs({{p->w_post, "w_post"}, {p->scale, "scale"}}, 4))) return rc;
  if (with_n && (rc = check_ptrs({{p->w_pre, "w_pre"}}, 4))) return rc;
  return DSSM_OK;
}

int dssm_resnorm_forward(const void* x, const void* y, const void* g, long long stride_g,
                         const dssm_resnorm_params* p, const dssm_resnorm_shape* s,
                         const int* lens, void* o, void* n, float* stats, void* stream) {
  bool empty = false;
  int rc = check_resnorm(s, &empty);
  if (rc) return rc;
  if (empty) return ok();
  const size_t e = elem_size(s->dtype);
  if ((rc = check_resnorm_in(x, "x", y, g, stride_g, p, s, lens, n != nullptr))) return rc;
  if (y && (rc = check_ptrs({{o, "o"}}, e))) return rc;
  if (!y && o) return fail(DSSM_ERR_INVALID_ARG, "o needs y (without y the stream is x)");
  if (!y && (rc = check_ptrs({{n, "n"}}, e))) return rc;
  if ((rc = check_opt(n, "n", e)) || (rc = check_opt(stats, "stats", 4))) return rc;
  if ((rc = check_alias({{o, "o"}, {n, "n"}, {stats, "stats"}}, {{x, "x"}, {y, "y"}, {g, "g"}})))
    return rc;
  ResnormCall c = resnorm_call(x, y, g, stride_g, p, s, lens);
  c.o = o;
  c.n = n;
  c.stats = stats;
  if ((rc = hip_check(launch_resnorm_forward(c, s->dtype, static_cast<hipStream_t>(stream)),
                      "resnorm forward launch")))
    return rc;
  return ok();
}

int dssm_resnorm8_forward(const void* x, const void* y, const void* g, long long stride_g,
                          const dssm_resnorm_params* p, const dssm_resnorm_shape* s,
                          const int* lens, int form, void* o, void* q, float* qs, float* stats,
                          void* stream) {
  bool empty = false;
  int rc = check_resnorm(s, &empty);
  if (rc) return rc;
  if (form != DSSM_Q8_INT8 && form != DSSM_Q8_E4M3)
    return fail(DSSM_ERR_INVALID_ARG, "form must be DSSM_Q8_INT8 or DSSM_Q8_E4M3, got %d", form);
  if (empty) return ok();
  const size_t e = elem_size(s->dtype);
  if (!p) return fail(DSSM_ERR_INVALID_ARG, "params is NULL");
  if (y && !p->w_post && (g || p->scale))
    return fail(DSSM_ERR_INVALID_ARG, "a gate or a scale needs w_post");
  // without w_post y is only added: as a call without y, but for o
  const bool plain = y && !p->w_post;
  if ((rc = check_resnorm_in(x, "x", plain ? nullptr : y, g, stride_g, p, s, lens, true)) ||
      (rc = check_opt(y, "y", e)) || (y && (rc = check_ptrs({{o, "o"}}, e))))
    return rc;
  if (!y && o) return fail(DSSM_ERR_INVALID_ARG, "o needs y (without y the stream is x)");
  if ((rc = check_ptrs({{q, "q"}}, 1)) || (rc = check_ptrs({{qs, "qs"}}, 4)) ||
      (rc = check_opt(stats, "stats", 4)))
    return rc;
  if ((rc = check_alias({{o, "o"}, {q, "q"}, {qs, "qs"}, {stats, "stats"}},
                        {{x, "x"}, {y, "y"}, {g, "g"}, {p->w_post, "w_post"},
                         {p->scale, "scale"}, {p->w_pre, "w_pre"}, {lens, "lens"}})))
    return rc;
  ResnormCall c = resnorm_call(x, y, g, stride_g, p, s, lens);
  c.o = o;
  c.stats = stats;
  const Resnorm8Out out{form == DSSM_Q8_E4M3, q, qs};
  if ((rc = hip_check(launch_resnorm8(c, s->dtype, out, static_cast<hipStream_t>(stream)),
                      "resnorm8 forward launch")))
    return rc;
  return ok();
}

int dssm_resnorm_workspace_size(const dssm_resnorm_shape* s, size_t* bytes) {
  if (!bytes) return fail(DSSM_ERR_INVALID_ARG, "bytes is NULL");
  bool empty = false;
  if (int rc = check_resnorm(s, &empty)) return rc;
  *bytes = empty ? 0 : resnorm_workspace(s->B, s->H, s->L, s->dtype);
  return ok();
}

int dssm_resnorm_backward(const void* o, const void* y, const void* g, long long stride_g,
                          const float* stats, const dssm_resnorm_params* p,
                          const dssm_resnorm_shape* s, const int* lens, const void* d_o,
                          const void* d_n, const dssm_resnorm_grads* gr, void* ws,
                          size_t ws_bytes, void* stream) {
  bool empty = false;
  int rc = check_resnorm(s, &empty);
  if (rc) return rc;
  if (s->H == 0) return ok();
  if (!gr) return fail(DSSM_ERR_INVALID_ARG, "grads is NULL");
  if (empty) {  // no steps: the sums are zero, whichever of them there are
    if ((rc = check_opt(gr->dw_post, "dw_post", 4)) || (rc = check_opt(gr->dscale, "dscale", 4)) ||
        (rc = check_opt(gr->dw_pre, "dw_pre", 4)))
      return rc;
    ResnormCall c{};
    c.B = 0;
    c.H = s->H;
    c.dw_post = gr->dw_post;
    c.dscale = gr->dscale;
    c.dw_pre = gr->dw_pre;
    if ((rc = hip_check(launch_resnorm_backward(c, s->dtype, static_cast<hipStream_t>(stream)),
                        "resnorm backward launch")))
      return rc;
    return ok();
  }
  const size_t e = elem_size(s->dtype);
  if (!d_o && !d_n) return fail(DSSM_ERR_INVALID_ARG, "d_o and d_n are both NULL");
  if (!y && !d_n) return fail(DSSM_ERR_INVALID_ARG, "without y d_n is required");
  if ((rc = check_resnorm_in(o, "o", y, g, stride_g, p, s, lens, d_n != nullptr))) return rc;
  if ((rc = check_ptrs({{stats, "stats"}}, 4)) || (rc = check_opt(d_o, "d_o", e)) ||
      (rc = check_opt(d_n, "d_n", e)) || (rc = check_ptrs({{gr->dx, "dx"}}, e)) ||
      (rc = check_ptrs({{gr->dw_pre, "dw_pre"}}, 4)))
    return rc;
  if (y && ((rc = check_ptrs({{gr->dy, "dy"}}, e)) ||
            (rc = check_ptrs({{gr->dw_post, "dw_post"}, {gr->dscale, "dscale"}}, 4))))
    return rc;
  if (g && ((rc = check_ptrs({{gr->dg, "dg"}}, e)) ||
            (rc = check_stride(gr->stride_dg, "stride_dg", s->B, s->H, s->L))))
    return rc;
  const void* none = nullptr;
  if ((rc = check_alias({{gr->dx, "dx"}, {y ? gr->dy : none, "dy"}, {g ? gr->dg : none, "dg"},
                         {y ? gr->dw_post : none, "dw_post"}, {y ? gr->dscale : none, "dscale"},
                         {gr->dw_pre, "dw_pre"}},
                        {{o, "o"}, {y, "y"}, {g, "g"}, {d_o, "d_o"}, {d_n, "d_n"},
                         {stats, "stats"}})))
    return rc;
  if ((rc = check_space(ws, ws_bytes, resnorm_workspace(s->B, s->H, s->L, s->dtype)))) return rc;
  if ((rc = check_alias({{ws, "workspace"}},
                        {{o, "o"}, {y, "y"}, {g, "g"}, {d_o, "d_o"}, {d_n, "d_n"}, {stats, "stats"},
                         {gr->dx, "dx"}, {y ? gr->dy : none, "dy"}, {g ? gr->dg : none, "dg"},
                         {y ? gr->dw_post : none, "dw_post"}, {y ? gr->dscale : none, "dscale"},
                         {gr->dw_pre, "dw_pre"}})))
    return rc;
  ResnormCall c = resnorm_call(o, y, g, stride_g, p, s, lens);
  c.stats = const_cast<float*>(stats);
  c.d_o = d_o;
  c.d_n = d_n;
  c.dx = gr->dx;
  c.dy = y ? gr->dy : nullptr;
  c.dg = g ? gr->dg : nullptr;
  c.stride_dg = gr->stride_dg;
  c.dw_post = y ? gr->dw_post : nullptr;
  c.dscale = y ? gr->dscale : nullptr;
  c.dw_pre = gr->dw_pre;
  c.ws = ws;
  if ((rc = hip_check(launch_resnorm_backward(c, s->dtype, static_cast<hipStream_t>(stream)),
                      "resnorm backward launch")))
    return rc;
  return ok();
}

}  // extern "C"
