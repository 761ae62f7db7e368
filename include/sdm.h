/*
 * sdm.h -- C ABI of the GB300 (sm_103a) Sparse Delta Memory forward step.
 *
 * The method (web pages, cited by title and section):
 *   [SDM notes]   "Sparse Delta Memory：中文精读笔记" (reading notes on
 *                 arXiv 2607.07386v1): 2.2 symbols, 2.3 product-key addressing,
 *                 2.4 Eq. (3)-(5) write / untouched slots / read, 2.5 Fig. 2.
 *   [FwPKM notes] Fast-weight Product Key Memory reading notes, 2.2: half-query
 *                 against sub-key tables; inverse-distance sub-score.
 *
 * One forward step per token t of every (b, h) chain:
 *   addressing  S_p[j] = <q_p, K_p[j]> (or -ln(eps + |q_p - K_p[j]|^2)), p = 1, 2;
 *               top-k of each half; best W (R) of the k*k sums S_1[a] + S_2[b];
 *               slot = a*s + b; weights = softmax over the selected sums.
 *   write       for i in I^w:  M~[i] = alpha_t M[i];
 *                              M[i]  = M~[i] + beta_t w_i (v_t - M~[i])   (Eq. (4))
 *               rows not in I^w are left bit-identical.
 *   read        y_t = sum_{i in I^r} q_i M[i], after the write.        (Eq. (5))
 *
 * Conventions for every entry point:
 *  - All tensor arguments are DEVICE pointers to dense row-major arrays that
 *    the caller allocates and owns; the library keeps no pointer after return.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Work is enqueued asynchronously; argument errors are returned before
 *    anything is enqueued.  Failures the device detects (an index out of
 *    range, a duplicate write slot, a wait that ran out) are recorded in a
 *    per-device status word that sdm_get_device_status() reads and clears.
 *  - Alignment: every tensor base must be 16-byte aligned.
 *  - A call with no work (B, H or T zero) enqueues nothing and returns
 *    SDM_OK after the shape check; its pointers are not looked at (empty
 *    tensors may pass NULL).
 *  - The library allocates no device memory (the status word is a static
 *    device variable; scratch is the caller's `workspace`).  There is no
 *    CPU fallback.
 *  - The device addresses of the library's static device arrays (the status
 *    word; the scratch of sdm_scan_noalloc) are looked up once per device and
 *    kept for the life of the process, and so are the two streams and the
 *    events sdm_forward uses for its overlapped windows (created on first
 *    use): do not go on using the library on a device after cudaDeviceReset
 *    (or any other teardown of its primary context), since those handles are
 *    then stale.
 */
#ifndef SDM_H
#define SDM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SDM_OK = 0,
  SDM_ERR_INVALID_ARG = 1,     /* null pointer, bad size, misaligned base       */
  SDM_ERR_UNSUPPORTED = 2,     /* valid but outside the limits listed below     */
  SDM_ERR_CUDA = 3,            /* a CUDA runtime call failed                    */
  SDM_ERR_TIMEOUT = 4,         /* device: a bounded wait ran out                */
  SDM_ERR_DEVICE_BOUNDS = 5,   /* device: a slot index outside [0, N)           */
  SDM_ERR_DUPLICATE_SLOT = 6   /* device: a slot repeated within one write set  */
} sdm_status;

/* SDM_E4M3 (8-bit float, 4 exponent bits, largest value 448) is an output
 * type of the residual norms only; every other argument takes the first two. */
typedef enum { SDM_F32 = 0, SDM_BF16 = 1, SDM_E4M3 = 2 } sdm_dtype;
typedef enum { SDM_SCORE_DOT = 0, SDM_SCORE_IDW = 1 } sdm_score_kind;
typedef enum { SDM_UPDATE_EQ4 = 0, SDM_UPDATE_SHARED_RESIDUAL = 1 } sdm_update_form;

typedef struct {
  int B, H, T;            /* batch, heads, tokens per chain                        */
  int n_sub;              /* s = sqrt(N) entries per sub-key table; N = s*s       */
  int d_h;                /* half-query / sub-key dimension                        */
  int d_v;                /* value width = row width of the table                 */
  int W, R;               /* write / read slots per token and head                */
  int k_w, k_r;           /* per-half top-k; 0 selects min(W, s) / min(R, s)      */
  sdm_dtype in_dtype;     /* dtype of q_w, q_r, K, v, alpha, beta                 */
  sdm_score_kind score;   /* sub-score kind                                        */
  float idw_eps;          /* eps of the inverse-distance score (1e-3 in [FwPKM])  */
  sdm_update_form update; /* SDM_UPDATE_EQ4: per-slot Eq. (4) [SDM notes 2.4].     */
                          /* SDM_UPDATE_SHARED_RESIDUAL: the residual shared by    */
                          /* the write set, read off Fig. 2 [SDM notes 2.5]:       */
                          /* M[i] = M~[i] + beta w_i (v - sum_j w_j M~[j]).        */
} sdm_shape;

/* Limits (anything else returns SDM_ERR_UNSUPPORTED):
 *   1 <= n_sub <= 512;  d_h in {16, 32, 64, 128, 256};  d_v a multiple of 16,
 *   16 <= d_v <= 2048;  1 <= W, R <= 64;  1 <= k <= min(64, n_sub) and
 *   W <= k_w^2, R <= k_r^2;  B*H*N*d_v < 2^40 elements;  B, H, T >= 0. */

/* Human-readable name of a status code (static string). */
const char* sdm_status_string(sdm_status st);

/* Sub-scores of one branch [SDM notes 2.3; FwPKM notes 2.2].
 *   q: [B,H,T,2,d_h] (in_dtype) half-queries of that branch;
 *   K: [H,2,s,d_h]   (in_dtype) the two sub-key tables of each head;
 *   S: [B,H,T,2,s]   float32 out: S[...,p,j] = <q_p, K_p[j]>, or
 *                    -ln(idw_eps + |q_p - K_p[j]|^2) when score = IDW.
 * Accumulation is fp32; used to compare addressing at the score level. */
sdm_status sdm_subscores(const sdm_shape* shape, const void* q, const void* K,
                         float* S, void* stream);

/* Product-key selection from given float32 sub-scores [SDM notes 2.3].
 *   sub_w, sub_r: [B,H,T,2,s] float32 sub-scores of the write / read branch;
 *   idx_w: [B,H,T,W] int32 out, wt_w: [B,H,T,W] float32 out;
 *   idx_r: [B,H,T,R] int32 out, wt_r: [B,H,T,R] float32 out.
 * Each half keeps its top k by (score desc, index asc); the k*k sums
 * fl32(S_1[a] + S_2[b]) are ranked by (sum desc, slot asc), slot = a*s + b;
 * the best W (R) are written in rank order, with the softmax of their sums.
 * Indices are exact: identical sub-scores give identical slots. */
sdm_status sdm_select(const sdm_shape* shape, const float* sub_w,
                      const float* sub_r, int32_t* idx_w, float* wt_w,
                      int32_t* idx_r, float* wt_r, void* stream);

/* Addressing: sdm_subscores + sdm_select for both branches, fused in one
 * kernel (the sub-scores never leave the chip).
 *   q_w, q_r: [B,H,T,2,d_h]; K: [H,2,s,d_h] (all in_dtype);
 *   outputs as in sdm_select. */
sdm_status sdm_address(const sdm_shape* shape, const void* q_w, const void* q_r,
                       const void* K, int32_t* idx_w, float* wt_w,
                       int32_t* idx_r, float* wt_r, void* stream);

/* Bytes of device workspace that sdm_scan / sdm_forward need for `shape`
 * (0 for an invalid shape).  The scan first resolves, for every row a step
 * touches, whether one of the few preceding steps still in flight wrote it
 * (a 16-bit code per token and row); the workspace holds those codes. */
size_t sdm_workspace_size(const sdm_shape* shape);

/* The write-then-read recurrence over t for every (b,h) chain
 * [SDM notes 2.4, Eq. (3)-(5)].
 *   idx_w/wt_w: [B,H,T,W] int32/float32; idx_r/wt_r: [B,H,T,R];
 *   alpha, beta: [B,H,T] (in_dtype); v: [B,H,T,d_v] (in_dtype);
 *   M: [B,H,N,d_v] float32, updated IN PLACE (the updated table is the result);
 *   y: [B,H,T,d_v] float32 out;
 *   workspace: device scratch of at least sdm_workspace_size(shape) bytes
 *   (ws_bytes), caller-owned, contents irrelevant on entry and on return.
 * shape->update selects the write: Eq. (4) per slot, or the shared residual
 * read off Fig. 2 (one prediction sum_j w_j M~[j] for the whole write set).
 * Write slots of one step must be distinct and all slots in [0, N); the
 * device checks both, skips the offending rows and records
 * SDM_ERR_DUPLICATE_SLOT / SDM_ERR_DEVICE_BOUNDS.  Calling this on
 * consecutive T-segments (the table carried in M) equals one call on the
 * concatenation.  M must not alias any other argument. */
sdm_status sdm_scan(const sdm_shape* shape, const int32_t* idx_w,
                    const float* wt_w, const int32_t* idx_r, const float* wt_r,
                    const void* alpha, const void* beta, const void* v,
                    float* M, float* y, void* workspace, size_t ws_bytes,
                    void* stream);

/* sdm_scan without a workspace, for callers that cannot allocate device
 * memory: e.g. a host framework that owns all device memory and only passes
 * in the tensors of a call, or a code path where a cudaMalloc (and the
 * device-wide synchronisation it may bring) is not allowed.  The paper has no
 * counterpart; this is an interface variant of sdm_scan, same arguments and
 * results minus `workspace`/`ws_bytes`.
 * Scratch: a fixed 8 MiB array of device memory in the library itself (every
 * GPU that loads the library holds it until the process exits).  Problems
 * needing more plan-code scratch than that, i.e.
 * B*H*T*round_up(W+R, 8)*2 bytes > 8 MiB (32768 token-heads at W = R = 64),
 * return SDM_ERR_UNSUPPORTED before anything is enqueued.
 * The first call on a device looks up the array's device address (with that
 * device current); make that first call before any stream capture.  All calls
 * share the one array: calls whose work overlaps on the GPU (other streams,
 * other threads) race and must be serialised by the caller.  Nothing in the
 * array needs clearing: every value a call reads, that call wrote first.
 * Calls no cudaMalloc, cudaFree or allocating library routine. */
sdm_status sdm_scan_noalloc(const sdm_shape* shape, const int32_t* idx_w,
                            const float* wt_w, const int32_t* idx_r,
                            const float* wt_r, const void* alpha, const void* beta,
                            const void* v, float* M, float* y, void* stream);

/* sdm_scan that also keeps an undo log [SDM notes 2.9, appendix A.3: the
 * forward pass writes the table in place and the backward pass brings back
 * earlier states by undoing the sparse writes, for O(T*W*d_v) extra memory].
 *   undo: [B,H,T,W,d_v] float32 out, caller-owned: undo[b,h,t,j,:] is the
 *         value row idx_w[b,h,t,j] held just before step t's write (an
 *         exact copy of the fp32 table row).
 * All other arguments, the workspace and the results as in sdm_scan. */
sdm_status sdm_scan_logged(const sdm_shape* shape, const int32_t* idx_w,
                           const float* wt_w, const int32_t* idx_r,
                           const float* wt_r, const void* alpha, const void* beta,
                           const void* v, float* M, float* y, float* undo,
                           void* workspace, size_t ws_bytes, void* stream);

/* Bytes of device workspace sdm_scan_undo needs: B*H*N*4 (one mark per
 * table row; 0 for an invalid shape). */
size_t sdm_undo_workspace_size(const sdm_shape* shape);

/* Undo a logged segment: M [B,H,N,d_v] float32, in place, goes back to the
 * table it was before the sdm_scan_logged call that produced `undo` for the
 * same idx_w [B,H,T,W] (shape->T = that segment's length).  Every row the
 * segment wrote gets the copy logged at its earliest write; other rows are
 * untouched.  The result is bit-exact.  Undoing segments in reverse order
 * walks a long sequence back chunk by chunk.
 *   workspace: at least sdm_undo_workspace_size(shape) bytes, caller-owned,
 *   contents irrelevant on entry and on return.
 * Slots outside [0, N) are skipped and recorded as SDM_ERR_DEVICE_BOUNDS. */
sdm_status sdm_scan_undo(const sdm_shape* shape, const int32_t* idx_w,
                         const float* undo, float* M, void* workspace,
                         size_t ws_bytes, void* stream);

/* Per-head RMS-Norm and element-wise output gate on the read result
 * [SDM notes 2.4, after Eq. (5); the head-mixing projection that follows is
 * not part of this library]:
 *   out[b,h,t,:] = y[b,h,t,:] / sqrt(mean_c y[b,h,t,c]^2 + eps)
 *                  * gamma[h,:] * g[b,h,t,:]
 *   y:     [B,H,T,d_v] float32 (the scan's output);
 *   g:     [B,H,T,d_v] output gate, in shape->in_dtype, applied as given;
 *   gamma: [H,d_v] float32 per-head scale, or NULL for ones;
 *   eps:   > 0;  out: [B,H,T,d_v] in out_dtype (SDM_BF16 or SDM_F32).
 * One pass over y, bandwidth-bound.  Shape fields other than B, H, T, d_v
 * and in_dtype only need to be valid. */
sdm_status sdm_rmsnorm_gate(const sdm_shape* shape, const float* y, const void* g,
                            const float* gamma, float eps, void* out,
                            sdm_dtype out_dtype, void* stream);

/* Optional epilogue of sdm_decode: the arguments of sdm_rmsnorm_gate. */
typedef struct {
  const void* g;         /* [B,H,T,d_v] output gate, in shape->in_dtype      */
  const float* gamma;    /* [H,d_v] per-head scale, or NULL for ones         */
  float eps;             /* > 0                                              */
  void* out;             /* [B,H,T,d_v] in out_dtype                         */
  sdm_dtype out_dtype;   /* SDM_BF16 or SDM_F32                              */
} sdm_epilogue;

/* The forward step fused into one launch for short sequences -- decode,
 * T = 1 per call [SDM notes 2.3-2.5; section 3 reports decode speed at the
 * shapes of 2.8: sqrt N = 240 / 480, d_v = 960 / 1920].  Same arguments and
 * results as sdm_forward (y, M in place, selections in idx_w/wt_w/idx_r/wt_r)
 * plus, when `epi` is non-NULL, the sdm_rmsnorm_gate epilogue on y written
 * to epi->out.  Each (b,h) chain runs its T steps in order on one CTA, or,
 * when there are too few chains to fill the GPU, on up to 8 CTAs that each
 * own a range of its columns (with the epilogue they form one thread-block
 * cluster for the row norm); the latency of a step is one chain's dependent
 * path; use sdm_forward for long T.  Needs no workspace.  Sub-scores are fp32 FFMA for both
 * input dtypes, so a selection can differ from one made on sdm_forward's
 * tensor-core scores only where two candidate sums are within fp32 rounding
 * of each other. */
sdm_status sdm_decode(const sdm_shape* shape, const void* q_w, const void* q_r,
                      const void* K, const void* alpha, const void* beta,
                      const void* v, float* M, float* y, int32_t* idx_w,
                      float* wt_w, int32_t* idx_r, float* wt_r,
                      const sdm_epilogue* epi, void* stream);

/* One full forward step: sdm_address then sdm_scan on `stream`.
 * Inputs as above; M updated in place, y written, and the selected indices
 * and weights returned in the caller's idx_w/wt_w/idx_r/wt_r buffers. */
/* Number of step windows sdm_forward cuts T into (1 = none; 0 for an
 * invalid shape): from T = 2048 on, T/512 windows (at most 32) where the
 * addressing runs on the tensor cores, else 4; every window but the last is
 * a whole number of 64-step blocks.  With more than one, the addressing of
 * window k+1 runs on a low-priority internal stream while window k is
 * scanned on a high-priority one, both joined back into the caller's
 * stream; results are bit-identical to sdm_address followed by sdm_scan.
 * Each window launches the addressing, plan and scan kernels once.  The
 * internal streams and events are created by the first windowed call on a
 * device: make that call outside a CUDA graph capture; later calls can be
 * captured (the fork and join are recorded with the caller's stream).  If
 * the streams cannot be created, sdm_forward runs unwindowed on the
 * caller's stream. */
int sdm_forward_windows(const sdm_shape* shape);

sdm_status sdm_forward(const sdm_shape* shape, const void* q_w, const void* q_r,
                       const void* K, const void* alpha, const void* beta,
                       const void* v, float* M, float* y, int32_t* idx_w,
                       float* wt_w, int32_t* idx_r, float* wt_r, void* workspace,
                       size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Gated delta recurrence: the dense counterpart of sdm_scan, one slot of
 * weight 1 per channel with the gates formed from their logits
 * [SDM notes 2.4: alpha = exp(-A softplus(z + b)), beta = sigmoid(z)].
 * For every sequence, row t and channel c:
 *   alpha = exp(-A[c] * softplus(za[t,c] + bias[c])),  beta = sigmoid(zb[t,c]);
 *   h~ = alpha h[t-1];  h[t] = h~ + beta (v[t,c] - h~);  y[t,c] = h[t].
 * The state h is float32 throughout; y is h rounded to the shape's dtype.
 *
 * Rows are packed: sequence s owns rows offsets[s] .. offsets[s+1]-1 of the
 * [rows, D] tensors.  `offsets` is a DEVICE array of n_seq + 1 int32, not
 * decreasing, within [0, rows]; NULL cuts the rows into n_seq equal parts.
 * A sequence may have no rows (its final state is its initial one).  Rows of
 * no sequence (before offsets[0], from offsets[n_seq] on) are neither read nor
 * written.  Offsets that break these rules are found on the device: nothing is
 * written and SDM_ERR_DEVICE_BOUNDS is recorded. */
typedef struct {
  int n_seq;              /* sequences, 0..65535                                 */
  int rows;               /* rows of the packed tensors                          */
  int D;                  /* channels, a multiple of 8, at most 65536            */
  int ld;                 /* elements between rows of za, zb, v (so that they can */
                          /* be column ranges of one wider projection); a        */
                          /* multiple of 8, at least D; 0 = D                    */
  int ld_grad;            /* the same of dza, dzb, dv; 0 = D                     */
  sdm_dtype dtype;        /* of za, zb, v, y, dy, dza, dzb, dv: SDM_F32/SDM_BF16 */
} sdm_recurrence;

/* Bytes of device workspace the forward / backward pass needs, and of the
 * `states` array that carries what the backward pass needs from the forward
 * one (0 for an invalid shape). */
size_t sdm_recurrence_workspace_size(const sdm_recurrence* shape);
size_t sdm_recurrence_states_size(const sdm_recurrence* shape);

/* Forward pass.
 *   za, zb, v: [rows, D] (rows ld apart); A, bias: [D] float32, NULL = ones /
 *   zeros, A not negative; offsets: see above, or NULL;
 *   h0: [n_seq, D] float32 initial states, or NULL for zeros;
 *   y:  [rows, D] out;  hT: [n_seq, D] float32 final states out, or NULL (may
 *   be h0 itself: states updated in place);
 *   states: NULL, or caller-owned scratch of sdm_recurrence_states_size bytes
 *   that sdm_recurrence_backward reads (contents private to the library);
 *   workspace: at least sdm_recurrence_workspace_size bytes, contents
 *   irrelevant on entry and on return; calls that may overlap on the GPU
 *   (other streams, captured graphs that run at the same time) need one each.
 * Apart from hT = h0, outputs must not overlap inputs or one another.  Results
 * are the same from run to run, bit for bit. */
sdm_status sdm_recurrence_forward(const sdm_recurrence* shape, const void* za, const void* zb,
                                  const void* v, const float* A, const float* bias,
                                  const int32_t* offsets, const float* h0, void* y, float* hT,
                                  float* states, void* workspace, size_t ws_bytes,
                                  void* stream);

/* Backward pass of sdm_recurrence_forward, for the same shape, inputs and
 * offsets and the `states` it wrote.
 *   dy: [rows, D] gradient of y;  dhT: [n_seq, D] float32 gradient of hT, or
 *   NULL for zeros;
 *   dza, dzb, dv: [rows, D] out (rows ld_grad apart);
 *   dA, dbias: [D] float32 out, sums over every row of every sequence, or
 *   NULL;  dh0: [n_seq, D] float32 out, or NULL (may be dhT itself).
 * Gradients are written, not added to what the arrays held.  Workspace,
 * overlap and repeatability as in the forward pass.  With n_seq = 0 only dA
 * and dbias are written (zeros). */
sdm_status sdm_recurrence_backward(const sdm_recurrence* shape, const void* za, const void* zb,
                                   const void* v, const float* A, const float* bias,
                                   const int32_t* offsets, const float* states, const void* dy,
                                   const float* dhT, void* dza, void* dzb, void* dv, float* dA,
                                   float* dbias, float* dh0, void* workspace, size_t ws_bytes,
                                   void* stream);

/* One token per sequence on a pool of states (decode): row i of the inputs
 * steps state row slots[i] in place and writes y row i.  Of the shape, rows
 * is the number of tokens; n_seq and ld_grad only need to be valid.
 *   state: [n_slots, D] float32, in place;  slots: [rows] int32, or NULL for
 *   row i = state row i (rows <= n_slots).  A negative slot is padding: that
 *   row of y and every state row stay as they are.  A slot >= n_slots
 *   (SDM_ERR_DEVICE_BOUNDS) or one that an earlier row already has
 *   (SDM_ERR_DUPLICATE_SLOT) is skipped in the same way and recorded.
 * Every slot is compared with all earlier ones, so that with slots the time has
 * a part that grows with the square of the rows (a quarter of the whole at 70000
 * rows of 1920 channels); rows is at most 4194304 then.
 * Needs no workspace.  y must not overlap an input. */
sdm_status sdm_recurrence_step(const sdm_recurrence* shape, const void* za, const void* zb,
                               const void* v, const float* A, const float* bias, float* state,
                               int n_slots, const int32_t* slots, void* y, void* stream);

/* ------------------------------------------------------------------------
 * Residual addition and RMS-Norm in front of a layer's projections (the norm
 * behind the read is sdm_rmsnorm_gate), optionally with the output in 8 bits:
 *   s = x + residual, rounded to the shape's dtype (s = x without a residual);
 *   n = s / sqrt(mean_c s_c^2 + eps) * gamma, from the rounded s, in float32;
 *   out = n in SDM_F32 or SDM_BF16; or, for SDM_E4M3, per row (group = 0) or
 *   per `group` channels: scale = max(max|n| / 448, 2^-126), float32, and
 *   out = n / scale rounded to nearest even, so that out * scale stands for n
 *   (both quotients are those of float32, themselves rounded to nearest).
 * A NaN in a row makes the row's outputs and scales NaN. */
typedef struct {
  int rows;               /* rows                                                */
  int D;                  /* channels, a multiple of 8, at most 16384            */
  sdm_dtype dtype;        /* of x, residual, s, dout, ds, dx: SDM_F32 / SDM_BF16 */
} sdm_norm;

/* Forward.
 *   x, residual: [rows, D]; residual may be NULL;  gamma: [D] float32 or NULL
 *   for ones;  eps: > 0;
 *   s: [rows, D] out, or NULL (may be x or residual itself: the residual
 *   stream updated in place);
 *   out: [rows, D] in out_dtype: SDM_F32, SDM_BF16 or SDM_E4M3;
 *   group: 0, 32, 64 or 128 (dividing D; 0 unless out_dtype is SDM_E4M3);
 *   scale: [rows] or [rows, D / group] float32 out, for SDM_E4M3 only.
 * out and scale must not overlap an input or s. */
sdm_status sdm_add_rmsnorm(const sdm_norm* shape, const void* x, const void* residual,
                           const float* gamma, float eps, void* s, void* out,
                           sdm_dtype out_dtype, int group, float* scale, void* stream);

/* Bytes of device workspace sdm_add_rmsnorm_backward needs (0 for an invalid
 * shape). */
size_t sdm_add_rmsnorm_workspace_size(const sdm_norm* shape);

/* Backward of the 16/32-bit forward from the s it wrote (x and residual have
 * the same gradient dx):
 *   w = dout gamma;  inv = 1 / sqrt(mean s^2 + eps);
 *   dx = ds + inv (w - s inv mean_c(w s inv));  dgamma = sum_rows dout s inv.
 *   dout: [rows, D] gradient of out, in the shape's dtype;  ds: [rows, D]
 *   gradient that reaches s from elsewhere, or NULL;  dx: [rows, D] out (may
 *   be dout or ds itself);  dgamma: [D] float32 out, written, or NULL;
 *   workspace: at least sdm_add_rmsnorm_workspace_size bytes if dgamma is
 *   given (else it may be NULL), one per overlapping call.
 * Results are the same from run to run, bit for bit. */
sdm_status sdm_add_rmsnorm_backward(const sdm_norm* shape, const void* s, const void* dout,
                                    const float* gamma, const void* ds, float eps, void* dx,
                                    float* dgamma, void* workspace, size_t ws_bytes,
                                    void* stream);

/* ------------------------------------------------------------------------
 * Residual addition and layer norm: sdm_add_rmsnorm with the mean taken off and
 * an offset added, everything else as there:
 *   s = x + residual, rounded to the shape's dtype;  c = s - mean_c s_c;
 *   n = c / sqrt(mean_c c_c^2 + eps) * gamma + beta, in float32;
 *   out = n, or in 8 bits with scales.
 * The mean is taken first and the squares are those of c.
 *   beta: [D] float32 or NULL for zeros. */
sdm_status sdm_add_layernorm(const sdm_norm* shape, const void* x, const void* residual,
                             const float* gamma, const float* beta, float eps, void* s, void* out,
                             sdm_dtype out_dtype, int group, float* scale, void* stream);

/* Bytes of device workspace sdm_add_layernorm_backward needs (0 for an invalid
 * shape). */
size_t sdm_add_layernorm_workspace_size(const sdm_norm* shape);

/* Backward of the 16/32-bit forward from the s it wrote, as
 * sdm_add_rmsnorm_backward:
 *   w = dout gamma;  inv = 1 / sqrt(mean c^2 + eps);
 *   dx = ds + inv (w - mean_c w - c inv mean_c(w c inv));
 *   dgamma = sum_rows dout c inv;  dbeta = sum_rows dout.
 *   dgamma, dbeta: [D] float32 out, written, or NULL; workspace: needed if one
 *   of them is given, one per overlapping call.
 * Results are the same from run to run, bit for bit. */
sdm_status sdm_add_layernorm_backward(const sdm_norm* shape, const void* s, const void* dout,
                                      const float* gamma, const void* ds, float eps, void* dx,
                                      float* dgamma, float* dbeta, void* workspace,
                                      size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Short causal convolution of every channel with its own taps, in front of a
 * recurrence.  For every sequence, row t and channel c:
 *   pre = bias[c] + sum_{k < taps} w[c, taps-1-k] x[t-k, c];
 *   y[t,c] = pre, or silu(pre) = pre / (1 + exp(-pre)),
 * in float32, rounded once.  Rows before a sequence are those of its start x0.
 * Packing, offsets, row strides and the treatment of bad offsets are those of
 * the recurrence above. */
typedef enum { SDM_ACT_NONE = 0, SDM_ACT_SILU = 1 } sdm_activation;

typedef struct {
  int n_seq;              /* sequences, 0..65535                                 */
  int rows;               /* rows of the packed tensors, at most 2^30            */
  int D;                  /* channels, a multiple of 8, at most 65536            */
  int taps;               /* 2, 3 or 4                                           */
  sdm_activation act;
  int ld;                 /* elements between rows of x; a multiple of 8, at     */
                          /* least D; 0 = D                                      */
  int ld_grad;            /* the same of dx; 0 = D                               */
  sdm_dtype dtype;        /* of x, y, x0, xT, state and their gradients:         */
                          /* SDM_F32 / SDM_BF16                                  */
} sdm_conv;

/* Forward pass.
 *   x: [rows, D] (rows ld apart);  w: [D, taps] float32, the last tap that of
 *   the row itself;  bias: [D] float32 or NULL for zeros;  offsets: as in
 *   sdm_recurrence_forward, or NULL;
 *   x0: [n_seq, taps-1, D] the rows in front of every sequence, oldest first,
 *   or NULL for zeros;
 *   y: [rows, D] out;  xT: [n_seq, taps-1, D] out, the last taps-1 rows of
 *   every sequence (of its start, where it is shorter), or NULL (may be x0
 *   itself: states updated in place).
 * Apart from xT = x0, outputs must not overlap inputs or one another. */
sdm_status sdm_short_conv_forward(const sdm_conv* shape, const void* x, const float* w,
                                  const float* bias, const int32_t* offsets, const void* x0,
                                  void* y, void* xT, void* stream);

/* Bytes of device workspace sdm_short_conv_backward needs (0 for an invalid
 * shape). */
size_t sdm_short_conv_workspace_size(const sdm_conv* shape);

/* Backward pass for the same shape and inputs.
 *   dy: [rows, D] gradient of y;  dxT: [n_seq, taps-1, D] gradient of xT, or
 *   NULL for zeros;
 *   dx: [rows, D] out (rows ld_grad apart);  dw: [D, taps], dbias: [D] float32
 *   out, sums over every row of every sequence, or NULL;  dx0: [n_seq, taps-1,
 *   D] out, or NULL;
 *   workspace: at least sdm_short_conv_workspace_size bytes if dw or dbias is
 *   given (else it may be NULL), one per overlapping call.
 * Gradients are written, not added to what the arrays held; outputs must not
 * overlap inputs or one another.  With n_seq = 0 only dw and dbias are written
 * (zeros).  Results are the same from run to run, bit for bit. */
sdm_status sdm_short_conv_backward(const sdm_conv* shape, const void* x, const float* w,
                                   const float* bias, const int32_t* offsets, const void* x0,
                                   const void* dy, const void* dxT, void* dx, float* dw,
                                   float* dbias, void* dx0, void* workspace, size_t ws_bytes,
                                   void* stream);

/* One token per sequence on a pool of windows (decode): row i of x goes
 * through the window slots[i], which loses its oldest row and gains x's.
 *   state: [n_slots, taps-1, D] in the shape's dtype, in place;  slots, n_slots
 *   and what is skipped and recorded: as in sdm_recurrence_step.
 * Needs no workspace.  y must not overlap an input. */
sdm_status sdm_short_conv_step(const sdm_conv* shape, const void* x, const float* w,
                               const float* bias, void* state, int n_slots, const int32_t* slots,
                               void* y, void* stream);

/* ------------------------------------------------------------------------
 * Selective state space scan: a diagonal recurrence with N states per channel
 * whose time step, input and output vectors depend on the token.  For every
 * sequence, row t, channel c of group g and state n:
 *   delta = softplus(dt[t,c] + bias[c]);
 *   h[c,n] = exp(-A[c,n] delta) h[c,n] + delta x[t,c] B[t,g,n];
 *   inner = sum_n C[t,g,n] h[c,n] + skip[c] x[t,c];
 *   y[t,c] = inner, or inner z / (1 + exp(-z)) with z = z[t,c].
 * Groups are of D / groups neighbouring channels.  The state h is float32
 * throughout; y is rounded once.  Packing, offsets and the treatment of bad
 * offsets are those of the recurrence above. */
typedef struct {
  int n_seq;              /* sequences, 0..65535                                 */
  int rows;               /* rows of the packed tensors, at most 2^30            */
  int D;                  /* channels, at most 65536                             */
  int N;                  /* states per channel: 8, 16, 32 or 64                 */
  int groups;             /* dividing D into multiples of 8 channels             */
  int ld;                 /* elements between rows of x and of dt; every stride  */
                          /* is a multiple of 8 and at least the row; 0 = dense  */
  int ld_z;               /* of z                                                */
  int ld_bc;              /* of B and of C (rows of groups * N)                  */
  int ld_grad;            /* of dx and of ddt                                    */
  int ld_z_grad;          /* of dz                                               */
  int ld_bc_grad;         /* of dB and of dC                                     */
  sdm_dtype dtype;        /* of x, dt, B, C, z, y, dy and the gradients of the   */
                          /* rows: SDM_F32 / SDM_BF16                            */
} sdm_selective;

/* Bytes of device workspace the forward and the backward pass need, and of the
 * `states` array that carries what the backward pass needs from the forward one
 * (a state every 16 rows; 0 for an invalid shape). */
size_t sdm_selective_scan_workspace_size(const sdm_selective* shape);
size_t sdm_selective_scan_backward_workspace_size(const sdm_selective* shape);
size_t sdm_selective_scan_states_size(const sdm_selective* shape);

/* Forward pass.
 *   x, dt: [rows, D];  A: [D, N] float32, not negative;  B, C: [rows, groups,
 *   N];  skip, bias: [D] float32 or NULL for zeros;  z: [rows, D] or NULL for
 *   no gate;  offsets: as in sdm_recurrence_forward, or NULL;
 *   h0: [n_seq, D, N] float32 initial states, or NULL for zeros;
 *   y: [rows, D] out;  hT: [n_seq, D, N] float32 final states out, or NULL (may
 *   be h0 itself: states updated in place);
 *   states: NULL, or caller-owned scratch of sdm_selective_scan_states_size
 *   bytes that sdm_selective_scan_backward reads;
 *   workspace: at least sdm_selective_scan_workspace_size bytes, contents
 *   irrelevant on entry and on return; calls that may overlap on the GPU (other
 *   streams, captured graphs that run at the same time) need one each.
 * Apart from hT = h0, outputs must not overlap inputs or one another.  Results
 * are the same from run to run, bit for bit. */
sdm_status sdm_selective_scan_forward(const sdm_selective* shape, const void* x, const void* dt,
                                      const float* A, const void* B, const void* C,
                                      const float* skip, const float* bias, const void* z,
                                      const int32_t* offsets, const float* h0, void* y, float* hT,
                                      float* states, void* workspace, size_t ws_bytes,
                                      void* stream);

/* Backward pass for the same shape, inputs and offsets and the `states` that
 * the forward pass wrote.
 *   dy: [rows, D] gradient of y;  dhT: [n_seq, D, N] float32 gradient of hT, or
 *   NULL for zeros;
 *   dx, ddt: [rows, D], dB, dC: [rows, groups, N], dz: [rows, D] (with z only)
 *   out;  dA: [D, N], dskip, dbias: [D] float32 out, sums over every row of
 *   every sequence, or NULL;  dh0: [n_seq, D, N] float32 out, or NULL (may be
 *   dhT itself);
 *   workspace: at least sdm_selective_scan_backward_workspace_size bytes.
 * Gradients are written, not added to what the arrays held.  Overlap and
 * repeatability as in the forward pass.  With n_seq = 0 only dA, dskip and
 * dbias are written (zeros). */
sdm_status sdm_selective_scan_backward(const sdm_selective* shape, const void* x, const void* dt,
                                       const float* A, const void* B, const void* C,
                                       const float* skip, const float* bias, const void* z,
                                       const int32_t* offsets, const float* states,
                                       const void* dy, const float* dhT, void* dx, void* ddt,
                                       float* dA, void* dB, void* dC, float* dskip, float* dbias,
                                       void* dz, float* dh0, void* workspace, size_t ws_bytes,
                                       void* stream);

/* One token per sequence on a pool of states (decode): row i of the inputs
 * steps state slots[i] in place and writes y row i.
 *   state: [n_slots, D, N] float32, in place;  slots, n_slots and what is
 *   skipped and recorded: as in sdm_recurrence_step.
 * Needs no workspace.  y must not overlap an input. */
sdm_status sdm_selective_scan_step(const sdm_selective* shape, const void* x, const void* dt,
                                   const float* A, const void* B, const void* C,
                                   const float* skip, const float* bias, const void* z,
                                   float* state, int n_slots, const int32_t* slots, void* y,
                                   void* stream);

/* Synchronizes `stream`, then returns and clears the device status word of
 * the current device (SDM_OK if no device-side failure was recorded). */
sdm_status sdm_get_device_status(void* stream);

/* Scan launch tuning for the calling process (0 = automatic):
 *   depth      steps whose rows are in flight per chain slice, 1..16;
 *   col_slice  columns of d_v per CTA, 16, 32 or 64 (must divide d_v).
 * Results do not depend on these; only speed does. */
sdm_status sdm_set_scan_tuning(int depth, int col_slice);

/* How long a block of sdm_recurrence_forward or _backward waits for what other
 * blocks publish, for the calling process's calls from now on: microseconds,
 * 0..1e7; -1 = the default, 4e6.  A wait that runs out ends the call's kernels,
 * which record SDM_ERR_TIMEOUT; the call's outputs are void then, and the next
 * call is as good as any.  With 0 a wait that is not over at the first look runs
 * out, which shows this on a real device. */
sdm_status sdm_set_recurrence_wait(long long limit_us);

/* Self-test of the bounded device wait: launches one CTA that waits on a
 * barrier no thread ever completes, with a limit of `timeout_ns`
 * nanoseconds (1e6..1e10), then records SDM_ERR_TIMEOUT and returns.
 * Shows on a real device that a wait that runs out ends the kernel cleanly. */
sdm_status sdm_selftest_wait_timeout(long long timeout_ns, void* stream);

/* Measurement reference, not part of the method: the scan's row traffic
 * ([SDM notes] 2.4: per step of every (chain, column slice) unit, the W + R
 * rows it touches are fetched and the W written rows stored back) with no
 * arithmetic and no dependency between steps.  For each of chains x
 * (d_v / col_slice) units and each of T steps, `loads` row pieces of
 * col_slice floats are copied from rows drawn uniformly from the unit's chain
 * in `src` into shared memory, and the first `stores` of them are written to
 * other uniformly drawn rows of the same chain and columns in `dst`; draws
 * are a fixed hash of (seed, unit, step, position).  Bytes moved:
 * chains * d_v * T * (loads + stores) * 4.  A timed call gives the rate HBM
 * sustains for the scan's access pattern.
 *   src, dst   device [chains, rows, d_v] float32 (may be the same array; the
 *              contents of dst afterwards are unspecified); 16-byte aligned.
 *   col_slice  16, 32 or 64, dividing d_v;  1 <= loads <= 128;
 *   0 <= stores <= loads;  1 <= rows < 2^32.
 * Argument errors return SDM_ERR_INVALID_ARG before anything is enqueued. */
sdm_status sdm_measure_row_traffic(const float* src, float* dst, long long chains,
                                   long long rows, int d_v, int col_slice, int T, int loads,
                                   int stores, unsigned seed, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SDM_H */
