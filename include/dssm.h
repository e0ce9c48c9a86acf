/*
 * dssm.h -- C ABI of libdssm.so: the forward map of a bank of H independent
 * diagonal linear RNN / diagonal state-space channels on AMD MI355X (gfx950).
 *
 * The map (DLR = "Simplifying and Understanding State Space Models with
 * Diagonal Linear RNNs", section 2):
 *
 *   lambda[h,n] = exp(-log_re[h,n]^2 + i*log_im[h,n])        (parameterisation)
 *   K[h,j]      = sum_n W[h,n] * lambda[h,n]^j,  0 <= j < L    (kernel)
 *   y[b,h,k]    = sum_{j=0}^{k} Re(K[h,j]) u[b,h,k-j] + D[h] u[b,h,k]
 *
 * The real cast of the kernel is the DLR page's (section 2, first paragraph);
 * the D feed-through is the SSM layer of "The Annotated S4" (Part 1, "An SSM
 * neural network").  With bidirectional = 1 a second, independent DLR runs on
 * the time-reversed input and its reversed output is added (DLR page,
 * section 2, bidirectional paragraph):
 *
 *   y[b,h,k] += sum_{j=0}^{L-1-k} Re(K_b[h,j]) u[b,h,k+j] + D_b[h] u[b,h,k]
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Layouts are row-major, last index fastest.  ndir = 1 + bidirectional.
 * - Every array argument is a DEVICE pointer (memory of the current HIP
 *   device), float32, 16-byte aligned.  Complex values are interleaved
 *   (re, im) float32 pairs, i.e. torch.complex64 / view_as_real layout.
 * - `stream` is a hipStream_t (NULL = the legacy default stream).  Every call
 *   only enqueues kernels on `stream` and returns; it never synchronises.
 * - Ownership: the caller allocates and owns every buffer, including the
 *   workspace `ws` of at least the size reported by dssm_workspace_size().
 *   The library allocates no device memory and keeps no pointer after return
 *   (the one exception: the fixed per-device scratch array of
 *   dssm_forward_fft_noalloc, part of the library's device image).
 *   Outputs must not alias inputs.  The workspace may be reused by later calls
 *   on the same stream; concurrent calls need distinct workspaces.
 * - Errors: every call returns a dssm_status.  Arguments are validated on the
 *   host before anything is launched, so an error return means nothing was
 *   enqueued (except DSSM_ERR_HIP, reported by the launch itself).  No call
 *   aborts or throws.  dssm_last_error() gives a per-thread message.
 * - Thread safety: calls may be made from several threads; the only mutable
 *   library state is the per-thread last-error message and the per-device
 *   scratch address of dssm_forward_fft_noalloc (looked up once under a
 *   lock; see that call for the race between overlapping calls). 
 */
#ifndef DSSM_H
#define DSSM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DSSM_VERSION 10400 /* major*10000 + minor*100 + patch */

/* Status codes. */
typedef enum {
  DSSM_OK = 0,
  DSSM_ERR_INVALID_ARG = -1,  /* null pointer, bad dimension or flag, misaligned pointer */
  DSSM_ERR_UNSUPPORTED = -2,  /* valid but outside what this library computes */
  DSSM_ERR_WORKSPACE = -3,    /* ws_bytes smaller than dssm_workspace_size() */
  DSSM_ERR_HIP = -4           /* a HIP launch reported an error */
} dssm_status;

/* Operations, for dssm_workspace_size(). */
typedef enum {
  DSSM_OP_GEN = 0,     /* dssm_gen_kernel */
  DSSM_OP_FFT = 1,     /* dssm_forward_fft */
  DSSM_OP_SCAN = 2,    /* dssm_forward_scan */
  DSSM_OP_BWD = 3,     /* dssm_backward */
  DSSM_OP_S5_SCAN = 4,  /* dssm_s5_forward, method DSSM_S5_SCAN (shape N = state size P) */
  DSSM_OP_S5_FFT = 5,   /* dssm_s5_forward, method DSSM_S5_FFT (shape N = state size P) */
  DSSM_OP_S5_FUSED = 6  /* dssm_s5_forward, method DSSM_S5_FUSED (shape N = state size P) */
} dssm_op;

/* How dssm_s5_forward runs the state recurrence ("Simplified State Space
 * Layers for Sequence Modeling", section 2.3: the recurrent mode and the
 * convolution mode of a linear time-invariant system give the same map). */
typedef enum {
  DSSM_S5_SCAN = 0, /* the recurrence as a parallel scan over time */
  DSSM_S5_FFT = 1,  /* per state, the convolution with lambda_p^j by FFT */
  DSSM_S5_FUSED = 2 /* projections and recurrence in one pass over u (v, x on chip) */
} dssm_s5_method;

/* How the complex kernel K is cast to the real kernel the convolution applies
 * (DLR page, section 2 for the real cast; section 2.1 for DLR-prod). */
typedef enum {
  DSSM_CAST_RE = 0,    /* Re K_j */
  DSSM_CAST_RE_IM = 1  /* Re K_j * Im K_j (DLR-prod) */
} dssm_cast;

/* Shape of a DLR bank: batch B, channels H, modes N, length L. */
typedef struct {
  int B, H, N, L;
  int bidirectional; /* 0 or 1 */
} dssm_shape;

/* DLR parameters (device pointers, float32).
 *   log_re [ndir, H, N]      (log Lambda)_re
 *   log_im [ndir, H, N]      (log Lambda)_im
 *   W      [ndir, H, N, 2]   complex output weights w
 *   D      [ndir, H]         real feed-through
 * Direction 0 is left-to-right, direction 1 (if bidirectional) right-to-left. */
typedef struct {
  const float* log_re;
  const float* log_im;
  const float* W;
  const float* D;
} dssm_dlr_params;

/* Gradients of the DLR parameters (device pointers, float32, 16-byte
 * aligned), laid out as the parameters of dssm_dlr_params:
 *   dlog_re [ndir, H, N], dlog_im [ndir, H, N], dW [ndir, H, N, 2]
 *   (d f / d Re W, d f / d Im W), dD [ndir, H]. */
typedef struct {
  float* dlog_re;
  float* dlog_im;
  float* dW;
  float* dD;
} dssm_dlr_grads;

/* Library version (DSSM_VERSION of the build). */
int dssm_version(void);

/* Static text for a status code. */
const char* dssm_status_string(int status);

/* Detail of the last error returned on the calling thread ("" if none). */
const char* dssm_last_error(void);

/* Bytes of workspace needed by `op` for shape `s` (host only; launches
 * nothing).  Returns DSSM_ERR_INVALID_ARG / DSSM_ERR_UNSUPPORTED exactly
 * when the corresponding compute call would.  Limits common to the DLR calls:
 * 1 <= N <= 4096, H (1 + bidirectional) <= 65535, B H L <= 2^40 and
 * B H (1 + bidirectional) <= 2^31 - 1.  For DSSM_OP_S5_SCAN / _FFT / _FUSED
 * the shape is read as the S5 shape {B, H, P = N, L, bidirectional} and the
 * result is dssm_s5_workspace_size() of that method. */
int dssm_workspace_size(int op, const dssm_shape* s, size_t* bytes);

/* Kernel generation: K[d,h,j] = sum_n W[d,h,n] lambda[d,h,n]^j for 0 <= j < L
 * (DLR page, section 2: K = (<w, Lambda^k>)_{0<=k<L}).
 *   complex_out = 0: K is [ndir, H, L] float32 holding Re K.
 *   complex_out = 1: K is [ndir, H, L, 2] float32 holding K (re, im).
 * Powers are formed from lambda^r (r < 64) and anchors W lambda^(64q) that
 * are computed in float64 and rounded once to float32; the sum over modes is
 * a matrix-core contraction on split operands (fp16 hi + lo, three products,
 * float32 accumulation; the anchors scaled by a power of two first), ~22
 * significant bits per operand.  B and p->D are ignored (D may be NULL); the
 * workspace size is 0 (ws may be NULL).
 * Requires 1 <= N <= 4096, 1 <= L <= 2^24. */
int dssm_gen_kernel(const dssm_dlr_params* p, const dssm_shape* s, int complex_out,
                    float* K, void* ws, size_t ws_bytes, void* stream);

/* The real kernel a cast applies: K [ndir, H, L] float32 holding Re K_j
 * (cast = DSSM_CAST_RE, as dssm_gen_kernel with complex_out = 0) or
 * Re K_j * Im K_j (cast = DSSM_CAST_RE_IM, the DLR-prod kernel of the DLR page,
 * section 2.1), K as in dssm_gen_kernel.  Any other cast returns
 * DSSM_ERR_INVALID_ARG.  Other arguments and limits as dssm_gen_kernel. */
int dssm_gen_kernel_cast(const dssm_dlr_params* p, const dssm_shape* s, int cast, float* K,
                         void* ws, size_t ws_bytes, void* stream);

/* Layer forward by the convolution view: y [B, H, L] from u [B, H, L].
 * Generates Re K, takes its spectrum on a zero-padded circle of length 2M
 * (M = the smallest power of two >= max(L, 16)), and for each channel forms
 * y = first L samples of IFFT(FFT(pad(u)) * spectrum) + D u -- the Toeplitz
 * product computed as a circulant product of size 2M (DLR page, section 2;
 * "The Annotated S4", Part 1, "Training SSMs: the convolutional
 * representation").  For bidirectional = 1 the backward kernel enters as the
 * conjugate spectrum (a correlation) and D_f + D_b multiplies u.
 * Requires L <= 16384 (the FFT is staged in one compute unit's LDS); longer L
 * returns DSSM_ERR_UNSUPPORTED (use dssm_forward_scan). */
int dssm_forward_fft(const float* u, const dssm_dlr_params* p, const dssm_shape* s,
                     float* y, void* ws, size_t ws_bytes, void* stream);

/* dssm_forward_fft without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  The workspace of dssm_forward_fft (the
 * real kernel rows and the spectrum table) lives in a device array inside the
 * library, 64 MiB per device, held by each device from the library's first
 * call on it until the process ends; the call itself allocates and frees
 * nothing.  Shapes whose workspace, dssm_workspace_size(DSSM_OP_FFT, s), is
 * larger than 64 MiB return DSSM_ERR_UNSUPPORTED before anything is
 * enqueued (for example B=4, H=128, L=16384 needs 42 MB; H=256, L=16384 needs
 * 84 MB and is refused).  Every call on one device uses that device's one
 * array: calls that overlap in time on the same device (different streams,
 * or threads) race and give wrong results; serialise them.  Results are the
 * same as dssm_forward_fft's.  Other arguments, conventions and limits as
 * dssm_forward_fft. */
int dssm_forward_fft_noalloc(const float* u, const dssm_dlr_params* p, const dssm_shape* s,
                             float* y, void* stream);

/* dssm_forward_fft with the kernel cast `cast` in place of Re K: with
 * DSSM_CAST_RE_IM each direction's convolution applies Re K_j * Im K_j (the
 * DLR-prod layer of the DLR page, sections 2.1 and 3); DSSM_CAST_RE is
 * dssm_forward_fft.  Any other cast returns DSSM_ERR_INVALID_ARG.  The
 * workspace is dssm_workspace_size(DSSM_OP_FFT, s).  DLR-prod has no
 * recurrence entry point: as a recurrence it is a DLR of N^2 modes
 * lambda_n lambda_m. */
int dssm_forward_fft_cast(const float* u, const dssm_dlr_params* p, const dssm_shape* s,
                          int cast, float* y, void* ws, size_t ws_bytes, void* stream);

/* Gradients of the layer map (the map of dssm_forward_fft / dssm_forward_scan,
 * which is the same map) for the scalar f = sum(dy * y): the input gradient
 * du [B, H, L] and the parameter gradients g (DLR page, section 2: K_j =
 * sum_n W_n lambda_n^j, lambda = exp(-log_re^2 + i log_im), dK_j / dlambda =
 * j W lambda^(j-1)).  With the kernel cotangents
 *   G_f[h,j] = sum_{b,k} dy[b,h,k] u[b,h,k-j],  G_b[h,j] = sum_{b,k} dy[b,h,k] u[b,h,k+j]:
 *   du     = the transposed layer operator applied to dy (the convolution with
 *            the conjugate spectrum: correlation with Re K_f, convolution with
 *            Re K_b, plus (D_f + D_b) dy);
 *   dW     = sum_j G_j conj(lambda^j);   with Z = sum_j j G_j W lambda^j:
 *   dlog_re = -2 log_re Re Z,  dlog_im = -Im Z;   dD_d = sum_{b,k} dy u.
 * The cotangents are lagged correlations summed over the batch in the
 * frequency domain (one transform per pair (u_b, dy_b) and half of the 2L
 * circle, one inverse per channel and half, both directions from the same
 * inverse); the sums over j run on float32 matrix products over 64-tap
 * blocks combined with float64 powers lambda^(64 q).
 * u, dy, du: [B, H, L] float32, 16-byte aligned; du must not alias u or dy.
 * Workspace: dssm_workspace_size(DSSM_OP_BWD, s).  Requires L <= 16384 (as
 * dssm_forward_fft) and B H <= 2^26.  With B = 0 or L = 0 the parameter
 * gradients are set to zero (u, dy, du, ws unused); with H = 0 nothing is
 * done. */
int dssm_backward(const float* u, const float* dy, const dssm_dlr_params* p,
                  const dssm_shape* s, float* du, const dssm_dlr_grads* g, void* ws,
                  size_t ws_bytes, void* stream);

/* Layer forward by the recurrence view: x_k = lambda x_{k-1} + u_k (x_{-1} = 0,
 * every mode driven by u), y_k = Re(sum_n W_n x_{k,n}) + D u_k; the backward
 * direction runs over k = L-1 .. 0 and is added ("The Annotated S4", Part 1,
 * "Discrete-time SSM: the recurrent representation"; the diagonal parallel
 * scan of "Simplified State Space Layers for Sequence Modeling", section 2.2).
 * For N <= 64 (and B H <= 2^24) the map is computed by chunks of 64 steps:
 * within a chunk as dense contractions on the matrix cores (the Toeplitz
 * product of the taps plus the contribution of the carried state, on split
 * fp16 operands scaled by powers of two), across chunks by the state
 * recurrence; otherwise time is split into segments, one per lane, whose
 * carries are combined with powers of lambda computed in float64.  Accepts
 * any L >= 1. */
int dssm_forward_scan(const float* u, const dssm_dlr_params* p, const dssm_shape* s,
                      float* y, void* ws, size_t ws_bytes, void* stream);

/* Streaming (stateful) forward by the recurrence view, one direction: the
 * recurrence of dssm_forward_scan continued from a given state instead of
 * zero ("The Annotated S4", Part 1, "Discrete-time SSM: the recurrent
 * representation": the state carries everything the past contributes, so a
 * sequence processed in consecutive chunks gives the outputs of the whole):
 *   x_{-1} = x (on entry),  x_k = lambda x_{k-1} + u_k,
 *   y_k = Re(sum_n W_n x_{k,n}) + D u_k,  x = x_{L-1} (on exit).
 *   x [B, H, N] complex (float32 pairs), read and then overwritten in place;
 *   it must not alias u or y.  u, y [B, H, L] as for dssm_forward_scan.
 * Requires bidirectional = 0 (a right-to-left direction needs the future:
 * DSSM_ERR_UNSUPPORTED).  L = 0 leaves x unchanged.  Workspace: the size
 * dssm_workspace_size(DSSM_OP_SCAN, s) reports.  Chunks of a long sequence
 * agree with the unsplit call within float32 rounding (the segment carries
 * are combined in a different order). */
int dssm_forward_scan_state(const float* u, const dssm_dlr_params* p, const dssm_shape* s,
                            float* x, float* y, void* ws, size_t ws_bytes, void* stream);

/* One decode step for every (b, h), the recurrent view advanced by one token
 * (the constant work per generated token that the DLR page's PG-19
 * language-modelling paragraph contrasts with attention; "The Annotated S4",
 * Part 3, "Sampling and caching": the recurrent state is the cache):
 *   x <- lambda x + u_t,  y_t = Re(sum_n W_n x_n) + D u_t.
 *   u_t, y_t [B, H] float32; x [B, H, N] complex, updated in place (no alias).
 * s->L must be 1 and s->bidirectional 0.  lambda is formed in float64 and
 * rounded once to float32 per call; a run of k steps is the float32 chain of
 * k products, so its error grows with k like any float32 recurrence.  No
 * workspace.  Requires B H <= 262140 (one wave per (b, h), four per
 * workgroup, at most 65535 workgroups); larger B H returns
 * DSSM_ERR_UNSUPPORTED. */
int dssm_step(const float* u_t, const dssm_dlr_params* p, const dssm_shape* s, float* x,
              float* y_t, void* stream);

/* ------------------------------------------------------------------------
 * S5-style multi-input multi-output diagonal SSM ("Simplified State Space
 * Layers for Sequence Modeling", section 3): one diagonal state of size P
 * shared by all H inputs,
 *   v_k = Bbar u_k,  x_k = lambda * x_{k-1} + v_k  (x_{-1} = 0),
 *   y_k = Re(C x_k) + D * u_k,
 * with the discrete lambda and Bbar given directly (no discretisation is
 * applied) and no factor 2 on the real part.  Layouts:
 *   u, y   [B, H, L] float32
 *   lambda [P, 2]    complex
 *   Bbar   [P, H, 2] complex
 *   C      [H, P, 2] complex
 *   D      [H]       float32
 * The projections are dense contractions (over H, and over 2P) on the
 * matrix cores with split operands: each float32 operand is written as an
 * fp16 hi part plus an fp16 lo part after a power-of-two scale per row (or
 * per time step), and three fp16 products (hi.hi + hi.lo + lo.hi) are
 * accumulated in float32, about 22 significant bits per operand.  The
 * state recurrence runs by `method`:
 *   DSSM_S5_SCAN: v and x in the workspace, a segmented complex scan
 *     between the projections whose carries use powers of lambda computed in
 *     float64 (section 2.2, the parallel scan);
 *   DSSM_S5_FUSED: the same recurrence with v and x never written to memory:
 *     per 64-step tile of a batch row, v = Bbar u, the tile's recurrence and
 *     y = Re(C x) + D u in one kernel; the sequence of a row is cut into
 *     segments whose entering states come from a state-only pass (the state
 *     each segment leaves from zero), joined with powers of lambda in
 *     float64.  Requires P <= 128, H <= 256 and H L <= 2^29 (otherwise
 *     DSSM_ERR_UNSUPPORTED);
 *   DSSM_S5_FFT: per state p and batch row b, the causal convolution
 *     x_p = (lambda_p^j)_j * v_p (section 2.3, the convolution mode), by a
 *     complex FFT on a zero-padded circle of length 2M (M = the smallest
 *     power of two >= max(L, 16)); the spectrum of the powers,
 *     (1 - (lambda w^m)^M) / (1 - lambda w^m) with w = exp(-i pi / M), is
 *     evaluated in float64 and rounded once.  Requires L <= 16384 (longer L:
 *     DSSM_ERR_UNSUPPORTED); its workspace adds P x 2M complex values.
 * Any other method returns DSSM_ERR_INVALID_ARG.  bidirectional = 1 is
 * DSSM_ERR_UNSUPPORTED (the pages define no bidirectional S5).
 * Requires 1 <= P <= 4096, L <= 2^24, B <= 65535.
 * ------------------------------------------------------------------------ */
typedef struct {
  int B, H, P, L;
  int bidirectional; /* must be 0 */
} dssm_s5_shape;

typedef struct {
  const float* lambda;
  const float* Bbar;
  const float* C;
  const float* D;
} dssm_s5_params;

/* Bytes of workspace dssm_s5_forward needs with `method` (host only).
 * DSSM_S5_FUSED needs only the packed projections, the segment states and
 * powers of lambda; the other methods add v and x (2 x B P L complex
 * float32). */
int dssm_s5_workspace_size(const dssm_s5_shape* s, int method, size_t* bytes);

/* Bytes of workspace dssm_s5_forward_tv needs (host only): the packed
 * projections, v and x.  Errors as dssm_s5_workspace_size. */
int dssm_s5_tv_workspace_size(const dssm_s5_shape* s, size_t* bytes);

/* y [B, H, L] from u [B, H, L] by `method` (a dssm_s5_method); same
 * conventions as the DLR calls. */
int dssm_s5_forward(const float* u, const dssm_s5_params* p, const dssm_s5_shape* s, int method,
                    float* y, void* ws, size_t ws_bytes, void* stream);

/* S5 in continuous time with a step size that changes from step to step
 * ("Simplified State Space Layers for Sequence Modeling", section 3: a
 * diagonal continuous-time system with a learnable timescale per state,
 * discretised by zero-order hold; irregularly sampled sequences are handled
 * by supplying a different timescale to the discretisation at each step).
 * The timescale of state p at step k of batch row b is step[b, k] * delta[p];
 * with z = lambda_c[p] step[b, k] delta[p]:
 *   x_k = exp(z) x_{k-1} + (exp(z) - 1) / lambda_c[p] (Btilde u_k)_p,
 *   y_k = Re(C x_k) + D u_k,   x_{-1} = 0
 * ((exp(z) - 1) / lambda_c is step delta where lambda_c = 0).  Layouts:
 *   lambda_c [P, 2] complex (continuous-time), Btilde [P, H, 2] complex,
 *   C [H, P, 2] complex, D [H] float32, delta [P] float32,
 *   step [B, L] float32 (the caller's time increments over the nominal step;
 *   0 is allowed: the state is then carried over unchanged).
 * The projections are those of dssm_s5_forward (Btilde in place of Bbar);
 * the scan forms z in float64 and the discretised values in float32.  Same
 * shape limits and conventions as dssm_s5_forward, workspace
 * dssm_s5_tv_workspace_size; step must be 16-byte aligned. */
typedef struct {
  const float* lambda_c;
  const float* Btilde;
  const float* C;
  const float* D;
  const float* delta;
} dssm_s5_tv_params;

int dssm_s5_forward_tv(const float* u, const dssm_s5_tv_params* p, const dssm_s5_shape* s,
                       const float* step, float* y, void* ws, size_t ws_bytes, void* stream);

/* Timing variant of dssm_s5_forward (n_events = 8): start/stop pairs of the
 * four stages, in order: packing of Bbar and C, input projection, the state
 * recurrence (the scan kernel, or the spectrum and convolution kernels of
 * DSSM_S5_FFT), output projection (same event conventions as the DLR timing
 * variants).  For DSSM_S5_FUSED the last three pairs stamp the state-only
 * pass, the kernel that forms the powers of lambda, and the output pass
 * (which also joins the segment states); with one segment per row there is
 * no state-only pass and its pair is recorded back to back. */
int dssm_s5_forward_timed(const float* u, const dssm_s5_params* p, const dssm_s5_shape* s,
                          int method, float* y, void* ws, size_t ws_bytes, void* stream,
                          void* const* events, int n_events);

/* ------------------------------------------------------------------------
 * The gated recurrence and what stands around it in a block.  These calls take
 * activations of several types; their shapes follow the layer calls, time
 * fastest.  Conventions that differ from the calls above:
 * - `dtype` is the type of the activations (u, r, i, y, their gradients, ...);
 *   parameters, states and statistics are float32.  All arithmetic is in
 *   float32 (parameters' gradients are added up over batch and time in float32
 *   within a workgroup's share at most, in float64 from there) and every output
 *   is rounded once, to nearest even.
 * - Pointers need the alignment of their element type (workspaces and
 *   checkpoints 256 bytes).  No output, checkpoint or workspace may be another
 *   buffer of its call, except where stated (DSSM_ERR_INVALID_ARG).
 * - stride_b / stride_g / ...: elements between two batch rows, at least H L;
 *   the H L elements of a row are contiguous.  A joint projection's output
 *   [B, 3 H, L] is passed as three slices with stride_b = 3 H L.
 * - lens (may be NULL): [B] int32, the steps of each batch row that are live.
 *   Steps at or past lens[b] are not read; outputs there are 0, and the state
 *   is the one after step lens[b] - 1.  Values are clamped to 0 .. L.
 * ------------------------------------------------------------------------ */
typedef enum {
  DSSM_F32 = 0,  /* float32 */
  DSSM_BF16 = 1, /* bfloat16 */
  DSSM_F16 = 2   /* IEEE half */
} dssm_dtype;

/* What a forward pass keeps for the backward pass. */
typedef enum {
  DSSM_CKPT_NONE = 0,
  DSSM_CKPT_STATE = 1, /* the state entering every DSSM_GATED_CHUNK steps */
  DSSM_CKPT_INT8 = 2   /* these states, and u, r, i in 8 bits */
} dssm_ckpt_kind;

#define DSSM_GATED_CHUNK 512 /* steps between two kept states */
#define DSSM_CKPT8_GROUP 64  /* steps that share a power of two in 8 bits */

typedef struct {
  int B, H, L;
  int dtype; /* dssm_dtype */
} dssm_gated_shape;

/* Inputs of the gated recurrence:
 *   u, r, i [B, H, L] (stride_b between batch rows): input, recurrence gate and
 *   input gate (both before the sigmoid);  log_re [H] float32;  lens [B] or NULL. */
typedef struct {
  const void* u;
  const void* r;
  const void* i;
  long long stride_b;
  const float* log_re;
  const int* lens;
} dssm_gated_inputs;

/* Gradients: du, dr, di [B, H, L] (stride_b between batch rows), dlog_re [H]
 * float32, dx0 [B, H] float32 (may be NULL). */
typedef struct {
  void* du;
  void* dr;
  void* di;
  long long stride_b;
  float* dlog_re;
  float* dx0;
} dssm_gated_grads;

/* Bytes of workspace of dssm_gated_forward and dssm_gated_backward (host
 * only).  Requires H <= 65535, B H <= 2^24, L <= 2^24, B H L <= 2^40. */
int dssm_gated_workspace_size(const dssm_gated_shape* s, size_t* bytes);

/* Bytes of a checkpoint of `kind` (0 for DSSM_CKPT_NONE).  Layout, every part
 * padded to 256 bytes: the states [B, H, ceil(L / 512)] float32 entering the
 * chunks, then for DSSM_CKPT_INT8 u, r and i, each as dssm_ckpt8_pack writes
 * B H rows of L, but the gates' logits r and i only up to +-31.75 (infinities
 * and a mask's lowest value too: they would cost the rest of their group its
 * scale).  The sigmoid is 0 or 1 to 2^-45 there, but a step's drive goes with
 * sqrt(1 - a^2) ~ |log_re| sqrt(2 sigmoid(r)): from 8 bits a step that r alone
 * shuts is driven by up to 2^-22 |log_re| sigmoid(i) u, and its u, r and i have
 * the gradients of that, where the forward pass and DSSM_CKPT_STATE have 0
 * (shut by i too, the drive is below 2^-67 |log_re u|).  Steps that are not
 * live are 0. */
int dssm_gated_ckpt_size(const dssm_gated_shape* s, int kind, size_t* bytes);

/* The gated linear recurrence: for every (b, h) a real mode whose decay and
 * drive are gated at every step,
 *   a_t = exp(-log_re[h]^2 sigmoid(r_t)),
 *   x_t = a_t x_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) u_t,   y_t = x_t
 * (sigmoid(r) = 1 is the mode lambda = exp(-log_re^2) of the layer above; the
 * factor sqrt(1 - a^2) keeps the state's size whatever the decay).
 *   x0 [B, H] float32 (may be NULL: zero): the state before step 0;
 *   x_end [B, H] float32 (may be NULL): receives the state after the last live
 *   step; it may be x0 (streaming in place) -- otherwise x0 is not changed.
 * ckpt: dssm_gated_ckpt_size(kind) bytes for a backward pass (ignored for
 * DSSM_CKPT_NONE).  Where 1 - a^2 is below float32's normal range it counts as
 * 0.  Rows are walked by one or four waves; few long rows are split into
 * segments joined through the workspace. */
int dssm_gated_forward(const dssm_gated_inputs* in, const dssm_gated_shape* s, const float* x0,
                       float* x_end, void* y, int kind, void* ckpt, void* ws, size_t ws_bytes,
                       void* stream);

/* One token for every (b, h): u, r, i, y [B, H] (s->L must be 1; stride_b >= H),
 * states as above.  A stream with lens[b] <= 0 is idle: its state is kept and
 * its output is 0.  No workspace; B H <= 2^31 - 1. */
int dssm_gated_step(const dssm_gated_inputs* in, const dssm_gated_shape* s, const float* x0,
                    float* x_end, void* y, void* stream);

/* Gradients of f = sum(dy y) + sum(dx_end x_end).  kind and ckpt: what the
 * forward pass of the same inputs kept (DSSM_CKPT_STATE or _INT8), with the
 * same lens.  With DSSM_CKPT_STATE u, r and i are read again; with
 * DSSM_CKPT_INT8 they are not (in->u, r, i and in->stride_b are ignored): the
 * gradients are those of the map at the decoded u, r and i, with the state
 * taken up again from the kept state at every chunk.
 *   dy [B, H, L];  dx_end [B, H] float32 (may be NULL: zero).
 * dlog_re is summed over b and t in a fixed order (results repeat bit for bit);
 * with B = 0 or L = 0 it is zero. */
int dssm_gated_backward(const dssm_gated_inputs* in, const dssm_gated_shape* s, int kind,
                        const void* ckpt, const void* dy, const float* dx_end,
                        const dssm_gated_grads* g, void* ws, size_t ws_bytes, void* stream);

/* Activations in 8 bits.  x [rows, L] in groups of 64 steps (the last one
 * shorter): x ~ q 2^E, q whole with |q| <= 127, E the smallest exponent with
 * max |x| <= 127 2^E and not below -126; the one rounding is that of x 2^-E to
 * even (where that would pass the largest value of x's type, |q| is 63).  A
 * group that holds Inf or NaN stands for NaN.  Layout of `blob`
 * (256-byte aligned): int8 q [rows, L rounded up to 16], padded to 256 bytes,
 * then one byte E + 127 per group [rows, ceil(L / 64)] (255: NaN).
 * Requires 0 <= rows, 0 <= L <= 2^24, rows L <= 2^40. */
int dssm_ckpt8_size(long long rows, int L, size_t* bytes);
int dssm_ckpt8_pack(const void* x, long long rows, int L, int dtype, void* blob, void* stream);
int dssm_ckpt8_unpack(const void* blob, long long rows, int L, int dtype, void* x, void* stream);

/* The norms around a layer, joined with its gate, residual scale and sum.
 * Over the H channels of every (b, t):
 *   norm(a) = (a - mean) / sqrt(mean((a - mean)^2) + eps)  (mean 0 for
 *   DSSM_NORM_RMS),
 *   v = norm(y) w_post,  o = x + scale v silu(g),  n = norm(o) w_pre,
 * o the residual stream after the layer and n what the next layer reads (the
 * second norm is of the stream as it is stored, in `dtype`).  Both norms have a
 * weight and no bias, the layer norm too.  silu(g) = g sigmoid(g): 0 at the
 * type's lowest value, NaN at -infinity. */
typedef enum { DSSM_NORM_RMS = 0, DSSM_NORM_LAYER = 1 } dssm_norm;

typedef struct {
  int B, H, L;
  int dtype; /* dssm_dtype */
  int norm;  /* dssm_norm */
  float eps; /* >= 0; read by the forward call */
} dssm_resnorm_shape;

typedef struct {
  const float* w_post; /* [H]; unused without y */
  const float* scale;  /* [H]; unused without y */
  const float* w_pre;  /* [H]; unused without n */
} dssm_resnorm_params;

/* dx, dy, dg (stride_dg between batch rows) [B, H, L]; dw_post, dscale, dw_pre
 * [H] float32. */
typedef struct {
  void* dx;
  void* dy;
  void* dg;
  long long stride_dg;
  float* dw_post;
  float* dscale;
  float* dw_pre;
} dssm_resnorm_grads;

/* x [B, H, L];  y [B, H, L] or NULL: without y there is no sum, o must be NULL
 * and n = norm(x) w_pre;  g [B, H, L] (stride_g between batch rows) or NULL: no
 * gate (silu(g) replaced by 1);  o [B, H, L];  n [B, H, L], or NULL with y: the
 * stream only.  stats (may be NULL) receives what the backward pass needs:
 * float32 [2, B, L] (1 / sqrt of y, of o) for DSSM_NORM_RMS, [4, B, L] (mean and
 * 1 / sqrt of y, then of o) for DSSM_NORM_LAYER; rows of a norm that the call
 * does not form are not written.  Requires H <= 8192 (a workgroup holds the
 * channels of a few steps; larger H: DSSM_ERR_UNSUPPORTED), L <= 2^20
 * and B ceil(L / 8) <= 2^21.
 * A single token is L = 1. */
int dssm_resnorm_forward(const void* x, const void* y, const void* g, long long stride_g,
                         const dssm_resnorm_params* p, const dssm_resnorm_shape* s,
                         const int* lens, void* o, void* n, float* stats, void* stream);

/* Bytes of workspace of dssm_resnorm_backward. */
int dssm_resnorm_workspace_size(const dssm_resnorm_shape* s, size_t* bytes);

/* Gradients of f = sum(d_o o) + sum(d_n n) at the forward call's o (its x, in
 * the call without y) and stats, with the same y, g and lens.  d_o or d_n may
 * be NULL (zero; both: DSSM_ERR_INVALID_ARG); without y d_n is required and dx =
 * d_o + the norm's gradient, dy, dg, dw_post and dscale are not written and may
 * be NULL; without g dg is not; without d_n dw_pre is set to zero.  The
 * parameters' sums run in a fixed order; with B = 0 or L = 0 they are zero. */
int dssm_resnorm_backward(const void* o, const void* y, const void* g, long long stride_g,
                          const float* stats, const dssm_resnorm_params* p,
                          const dssm_resnorm_shape* s, const int* lens, const void* d_o,
                          const void* d_n, const dssm_resnorm_grads* gr, void* ws,
                          size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * A selective state space block: the short causal convolution, the scan whose
 * step sizes, drive and read-out come with every step, and the norm that feeds
 * the next product in 8 bits.  Conventions as for the gated recurrence (types,
 * strides, lens, aliases, sums in a fixed order).
 * ------------------------------------------------------------------------ */
typedef enum { DSSM_ACT_NONE = 0, DSSM_ACT_SILU = 1 } dssm_act;

typedef struct {
  int B, H, L;
  int K;     /* taps, 1 .. 8 */
  int dtype; /* dssm_dtype */
  int act;   /* dssm_act */
} dssm_shortconv_shape;

/* du [B, H, L] (stride_b between batch rows), dw [H, K], dbias [H], dx0
 * [B, H, K - 1] float32 (the last two may be NULL). */
typedef struct {
  void* du;
  long long stride_b;
  float* dw;
  float* dbias;
  float* dx0;
} dssm_shortconv_grads;

/* The short causal convolution of every channel,
 *   y_t = act(bias + sum_{k < K} w_k u_{t - (K - 1) + k}),
 * the steps before the first one coming from the state.
 *   u, y [B, H, L] (u: stride_b between batch rows);  w [H, K], bias [H] float32
 *   (bias may be NULL: zero);
 *   x0 [B, H, K - 1] float32 (may be NULL: zero): the K - 1 inputs before step
 *   0, the oldest first;  x_end [B, H, K - 1] (may be NULL) receives the last
 *   K - 1 up to the last live step (with fewer live steps, x0's last are kept
 *   ahead of them); it may be x0.
 * silu is 0 at the type's lowest value, NaN at -infinity.  Requires B H <= 2^24
 * and the limits of the gated recurrence; a sequence needs a lane per 8 steps, of
 * which a launch has fewer than 2^32. */
int dssm_shortconv_forward(const void* u, long long stride_b, const float* w, const float* bias,
                           const dssm_shortconv_shape* s, const int* lens, const float* x0,
                           float* x_end, void* y, void* stream);

/* One token for every (b, h): u, y [B, H] (s->L must be 1; stride_b >= H).  A
 * stream with lens[b] <= 0 is idle: its state is kept and its output is 0. */
int dssm_shortconv_step(const void* u, long long stride_b, const float* w, const float* bias,
                        const dssm_shortconv_shape* s, const int* lens, const float* x0,
                        float* x_end, void* y, void* stream);

/* Bytes of workspace of dssm_shortconv_backward (host only). */
int dssm_shortconv_workspace_size(const dssm_shortconv_shape* s, size_t* bytes);

/* Gradients of f = sum(dy y) + sum(dx_end x_end) for the forward call with the
 * same u, w, bias, lens and x0.  dy [B, H, L]; dx_end [B, H, K - 1] float32
 * (may be NULL: zero). */
int dssm_shortconv_backward(const void* u, long long stride_b, const float* w, const float* bias,
                            const dssm_shortconv_shape* s, const int* lens, const float* x0,
                            const void* dy, const float* dx_end, const dssm_shortconv_grads* g,
                            void* ws, size_t ws_bytes, void* stream);

#define DSSM_SELECTIVE_CHUNK 128 /* steps between two kept states */

typedef struct {
  int B, H, L;
  int N;     /* modes of a channel, 1 .. 128 */
  int G;     /* groups: channel h reads B and C of group h / (H / G); H % G = 0 */
  int dtype; /* dssm_dtype */
} dssm_selective_shape;

/* u, delta, z [B, H, L], Bm, Cm [B, G, N, L], each with its elements between two
 * batch rows (at least H L, G N L);  log_re [H, N], D [H], dt_bias [H] float32.
 * z, D and dt_bias may be NULL: no gate, no skip, no bias. */
typedef struct {
  const void* u;
  const void* delta;
  const void* z;
  const void* Bm;
  const void* Cm;
  long long stride_u, stride_delta, stride_z, stride_B, stride_C;
  const float* log_re;
  const float* D;
  const float* dt_bias;
  const int* lens; /* [B] or NULL */
} dssm_selective_inputs;

/* Gradients of the inputs, shaped and strided like them; dlog_re [H, N], dD,
 * ddt_bias [H], dx0 [B, H, N] float32.  dz goes with z, dD with D, ddt_bias with
 * dt_bias (NULL without them); dx0 may be NULL. */
typedef struct {
  void* du;
  void* ddelta;
  void* dz;
  void* dB;
  void* dC;
  long long stride_u, stride_delta, stride_z, stride_B, stride_C;
  float* dlog_re;
  float* dD;
  float* ddt_bias;
  float* dx0;
} dssm_selective_grads;

/* Bytes of workspace of dssm_selective_forward or (backward != 0)
 * dssm_selective_backward (host only): forward at most twice a checkpoint's, backward
 * at most 2 GiB (parts of dB and dC in float32, B G ceil(H / (16 G)) 2 N L of them where
 * that is less) and six times a checkpoint's.  Requires H <= 65535, B H <= 2^24, L <=
 * 2^24, B H L <= 2^40, B H N ceil(L / 128) <= 2^36, B G N ceil(L / 1024) <= 2^29;
 * the calls over sequences B G ceil(H / (16 G)) < 2^23 (16 channels of a group, or one,
 * to 512 lanes; 32 where L <= 64). */
int dssm_selective_workspace_size(const dssm_selective_shape* s, int backward, size_t* bytes);

/* Bytes of a checkpoint: the states [B, H, ceil(L / 128), N] float32 entering
 * the chunks (those of a row's dead chunks are not written), padded to 256. */
int dssm_selective_ckpt_size(const dssm_selective_shape* s, size_t* bytes);

/* The selective scan: for every (b, h) a bank of N real modes driven alike,
 *   dt_t = softplus(delta_t + dt_bias[h]),
 *   x_t = exp(-log_re[h]^2 dt_t) x_{t-1} + dt_t B_t u_t         (N values each),
 *   y_t = (sum_n C_t x_t + D[h] u_t) silu(z_t)
 * (a step of length 1 decays as the mode exp(-log_re^2) of the layer above;
 * delta = -infinity, with finite u_t and B_t, is a step that changes nothing; a step of
 * 2^127 without a drive is one that forgets all).
 *   x0 [B, H, N] float32 (may be NULL: zero): the state before step 0;
 *   x_end [B, H, N] float32 (may be NULL): receives the state after the last
 *   live step; it may be x0.
 * ckpt (may be NULL): dssm_selective_ckpt_size bytes, for a backward pass. */
int dssm_selective_forward(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                           const float* x0, float* x_end, void* y, void* ckpt, void* ws,
                           size_t ws_bytes, void* stream);

/* One token for every (b, h): u, delta, z, y [B, H], Bm, Cm [B, G, N] (s->L must
 * be 1; strides at least H, G N), states as above.  A stream with lens[b] <= 0
 * is idle: its state is kept and its output is 0.  No workspace. */
int dssm_selective_step(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                        const float* x0, float* x_end, void* y, void* stream);

/* Gradients of f = sum(dy y) + sum(dx_end x_end) for the forward call of the
 * same inputs that wrote ckpt.  dy [B, H, L]; dx_end [B, H, N] float32 (may be
 * NULL: zero). */
int dssm_selective_backward(const dssm_selective_inputs* in, const dssm_selective_shape* s,
                            const void* ckpt, const void* dy, const float* dx_end,
                            const dssm_selective_grads* g, void* ws, size_t ws_bytes,
                            void* stream);

/* The residual sum and norm of dssm_resnorm_forward with n in 8 bits, for the
 * product that reads it: per step a scale and whole numbers or e4m3 values,
 *   n_t = norm(o_t) w_pre,  qs_t = max_h |n_t| / M,  q_t = n_t / qs_t to nearest even,
 * M = 127 (DSSM_Q8_INT8) or 448 (DSSM_Q8_E4M3: 4 exponent bits, 3 of fraction, no
 * infinities).  n is not rounded in between.  A step that holds Inf or NaN has
 * qs NaN and q 0; one whose largest |(o - mean) w_pre| is below 2^-100, or that
 * is not live, has qs 0 and q 0.
 *   q [B, L, H], one byte each: channels fastest, unlike every other activation
 *   here (the operand of an 8-bit product reads along the summed axis);
 *   qs [B, L] float32;  the rest as dssm_resnorm_forward, and its limits.
 * Three forms: with y and w_post as there;  y without w_post: o = x + y (no norm
 * of y; scale and g must be NULL);  without y: n = norm(x) w_pre, o NULL.
 * stats (may be NULL): as there, for dssm_resnorm_backward, which takes the
 * rounding for the identity; for o = x + y call it without y: its dx is the
 * gradient of x and of y. */
typedef enum { DSSM_Q8_INT8 = 0, DSSM_Q8_E4M3 = 1 } dssm_q8_form;

int dssm_resnorm8_forward(const void* x, const void* y, const void* g, long long stride_g,
                          const dssm_resnorm_params* p, const dssm_resnorm_shape* s,
                          const int* lens, int form, void* o, void* q, float* qs, float* stats,
                          void* stream);

/* Timing variants: identical results to dssm_forward_fft / dssm_forward_scan;
 * the kernels of stage k are launched with hipExtLaunchKernel so that the GPU
 * itself stamps events[2k] when the stage's first kernel starts and
 * events[2k+1] when its last kernel ends (hipEventElapsedTime of a pair is
 * the stage's duration, without the dispatch gap before it).  A pair of NULL
 * handles leaves that stage untimed (plain launches: an event-stamped launch
 * costs more host time).  n_events = 4 for both:
 *   fft:  [0,1] parameters -> kernel spectrum (generator and spectrum
 *         kernels), [2,3] convolution.
 *   scan: [0,1] per-mode constants of the segmented scan (with the chunked
 *         matrix-core form, used for N <= 64, there is no such kernel and the
 *         pair is recorded back to back: a duration of ~0), [2,3] scan.
 * The events are owned by the caller and must have timing enabled; a NULL
 * array, a pair with one NULL handle, or a wrong n_events returns
 * DSSM_ERR_INVALID_ARG before anything is enqueued. */
int dssm_forward_fft_timed(const float* u, const dssm_dlr_params* p, const dssm_shape* s,
                           float* y, void* ws, size_t ws_bytes, void* stream,
                           void* const* events, int n_events);
int dssm_forward_scan_timed(const float* u, const dssm_dlr_params* p, const dssm_shape* s,
                            float* y, void* ws, size_t ws_bytes, void* stream,
                            void* const* events, int n_events);

#ifdef __cplusplus
}
#endif

#endif /* DSSM_H */
