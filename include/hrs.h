/*
 * hrs.h - hybrid recurrent state: verify-span checkpoints, greedy acceptance
 * and on-device rollback for Gated DeltaNet (GDN) layers, on AMD MI355X
 * (gfx950).
 *
 * The library implements the data-parallel hot path of verifying a
 * speculative-decoding draft block through the recurrent layers of a hybrid
 * Qwen3.5/3.6-style target:
 *
 *   conv1d_verify_span  causal depthwise conv over the span, conv state
 *                       captured after every position
 *   gdn_verify_span     gated delta rule over the span (chain or draft tree),
 *                       F32 state checkpoint after every position
 *   accept_greedy       target argmax per position and the longest matching
 *                       prefix / root path
 *   rollback_restore    restore the accepted checkpoint of every layer on the
 *                       device, index read on the device, no replay
 *   ring_set_2d / ring_get_2d
 *                       batched feature-ring row copies with wraparound
 *
 * and, beside them: gdn_verify_span_from, conv1d_verify_span_nocapture and
 * conv_state_advance (zero-copy rollback), gdn_layer_verify_span (one layer
 * fused into one kernel) and gdn_span_chunked (long spans in chunks).
 *
 * For the same target's full-attention layers, and for targets that sample:
 *
 *   qk_norm_rope        RMS norm of every query and key head and the position
 *                       rotation, in one pass
 *   attn_verify_span    attention of the span (chain or draft tree) over a
 *                       paged cache and the span's own root paths
 *   attn_verify_shared  the same for requests that share a prefix, which is read
 *                       once for all of them
 *   kv_cache_append     the accepted path's keys and values into the cache
 *                       pages of every layer, indices read on the device
 *   accept_sample       verification of the drafts against the target's
 *                       probabilities from given random numbers
 *   accept_sample_filtered
 *                       the same after top-k, top-p and min-p
 *   accept_hold         requests that cannot go on (pages full or missing, no
 *                       valid temperature) taken out before the commit;
 *                       accept_hold_behind: of requests that share a prefix
 *   kv_pages_reserve / kv_pages_reserve_step / kv_pages_release
 *                       page tables that grow from a free list and shrink back
 *                       into it, and the slots of new positions
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - Memory: every device buffer is allocated and owned by the caller. The
 *    library allocates and frees nothing and keeps no pointer after a call
 *    returns. Host arrays (parent, runs) are read during the call only.
 *  - Streams: every device call is asynchronous on `stream` (a hipStream_t
 *    passed as void*; NULL means the null stream). Nothing synchronises.
 *  - Layout: dense, row-major, dims as written. Multi-layer buffers carry a
 *    leading [L] dim; per-layer calls take pointers into one layer.
 *  - Alignment: device pointers must be 16-byte aligned.
 *  - Errors: a negative return means nothing was launched (fail closed),
 *    except HRS_EDEVICE, which reports that the launch itself failed.
 *    Every argument check runs on the host before any HIP call, so the
 *    checks also work on a machine without a GPU.
 *  - Thread safety: the library holds no mutable global state shared
 *    between threads; each thread keeps a record of its last HIP error (see
 *    hrs_last_hip_error) and a cache of the device attributes its launches
 *    need (compute units, LDS per block), keyed by the current device.
 *  - Determinism: results are bit-identical from run to run, and the
 *    arithmetic of one position does not depend on the span length or on the
 *    tree topology (attn_verify_span: bit-identical from run to run of the
 *    same call, and whatever the keys and values that a query does not count
 *    hold; where a context is split among blocks depends on every length in
 *    the batch, and inside a block on T * Hq / Hkv, so the same request in
 *    another batch or a longer span agrees to rounding only).
 *
 * Sources (the pages this path comes from):
 *  [P1] lucebox PR #533, "feat: DFlash support for tensor-parallel Qwen3.6
 *       targets": Changes, Verification, Sustained performance.
 *  [P2] openinfer PR #626, "feat(qwen35): add opt-in DFlash speculative
 *       decoding": Summary, What Changed, Future Work.
 *  [P3] lucebox PR #506, "perf(dflash): split-chain fast rollback with F32
 *       SSM checkpoints (+29% decode)": Summary, Memory trade-off, Safety
 *       boundary, Verification.
 *  [GDN] Yang, Kautz, Hatamizadeh, "Gated Delta Networks: Improving Mamba2
 *       with Delta Rule", ICLR 2025: the gated delta rule.
 */
#ifndef HRS_H
#define HRS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HRS_ABI_VERSION 1

/* Largest span (root + drafts) a call accepts. */
#define HRS_MAX_POS 64

typedef enum {
  HRS_OK = 0,
  HRS_EINVAL = -1,       /* bad size, NULL pointer or dtype combination  */
  HRS_EGEOMETRY = -2,    /* draft geometry rejected by the guard          */
  HRS_EALIGN = -3,       /* device pointer not 16-byte aligned            */
  HRS_EDEVICE = -4,      /* the HIP launch failed                         */
  HRS_EUNSUPPORTED = -5  /* valid request outside the built kernel set    */
} hrs_status;

/* HRS_F8E4M3 (OCP e4m3, no infinities, largest 448) is a cache type only. */
typedef enum { HRS_F32 = 0, HRS_BF16 = 1, HRS_F8E4M3 = 2 } hrs_dtype;

typedef enum { HRS_CHAIN = 0, HRS_TREE = 1 } hrs_topology;

/* Verdicts of the geometry guard (see hrs_validate_tree). */
typedef enum {
  HRS_GEOM_OK = 0,
  HRS_GEOM_NULL = 1,       /* no parent array where one is required        */
  HRS_GEOM_TRUNCATED = 2,  /* n_pos outside [1, HRS_MAX_POS]               */
  HRS_GEOM_ROOT = 3,       /* parent[0] != -1, or a second root            */
  HRS_GEOM_RANGE = 4,      /* parent[i] < -1 or parent[i] >= n_pos         */
  HRS_GEOM_FORWARD = 5,    /* i <= parent[i] (self, cyclic, forward)       */
  HRS_GEOM_NOT_CHAIN = 6   /* chain required but parent[i] != i - 1        */
} hrs_geometry_class;

/*
 * hrs_validate_tree - the fail-closed geometry guard ([P3] Safety boundary:
 * sibling, malformed-root, skipped-parent, cyclic/forward-parent,
 * out-of-range, truncated and null geometry are rejected before execution).
 *
 * parent: host array of n_pos entries; position 0 is the committed root
 *         (parent -1) and every other position names an earlier position.
 * require_chain: nonzero = only the root-inclusive pure chain
 *         (parent[i] == i - 1) is accepted, as on [P3]; zero = any tree in
 *         topological order (draft trees, [P1] Verification: DDTree).
 * geometry_class: optional out (may be NULL), one hrs_geometry_class; the
 *         lowest-index offending position decides.
 * Returns HRS_OK or HRS_EGEOMETRY. Host only; touches no device.
 */
int hrs_validate_tree(const int32_t* parent, int32_t n_pos, int32_t require_chain,
                      int32_t* geometry_class);

/* ------------------------------------------------------------------------ */
/* GDN verify span                                                          */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t n_req;      /* R  requests in the batch                          */
  int32_t n_pos;      /* T  span positions: committed root + K drafts      */
  int32_t n_kheads;   /* Hk key heads                                      */
  int32_t n_vheads;   /* Hv value heads; Hv % Hk == 0                      */
  int32_t d_k;        /* key dim: 64 or 128                                */
  int32_t d_v;        /* value dim: multiple of 16, at most 256            */
  hrs_dtype in_dtype; /* dtype of q, k, v, a, b                            */
  float q_scale;      /* q is multiplied by this after widening (1.0 = none) */
  hrs_topology topo;  /* HRS_CHAIN or HRS_TREE                             */
  const int32_t* parent; /* host [n_req][n_pos] when topo == HRS_TREE, else
                            ignored (may be NULL)                          */
} hrs_gdn_desc;

/*
 * gdn_verify_span - the gated delta rule ([GDN]) over a verify span, with an
 * F32 state checkpoint after every position ([P3] Summary: F32 SSM
 * checkpoints captured during verify for rollback without replay; [P3]
 * Verification: the GDN op writes every intermediate state to a persist
 * buffer).
 *
 * Per request r, value head h (key head g = h / (Hv/Hk)), position t whose
 * parent is p (chain: p = t - 1), with P = state[r][h] when p == -1 else
 * ckpt[r][p][h]:
 *     u        = P k_t[g]
 *     S_t      = a_t[h] P + b_t[h] (v_t[h] - a_t[h] u) k_t[g]^T
 *                (= a P (I - b k k^T) + b v k^T)
 *     ckpt[r][t][h] = S_t            (float32)
 *     out[r][t][h]  = S_t (q_scale q_t[g])
 * S is d_v rows (value dims) by d_k columns (key dims). The math is float32
 * with bf16 inputs widened exactly.
 *
 * Layouts:  q, k  [R][T][Hk][d_k]      in_dtype
 *           v     [R][T][Hv][d_v]      in_dtype
 *           a, b  [R][T][Hv]           in_dtype (decay and write strength)
 *           state [R][Hv][d_v][d_k]    float32
 *           ckpt  [R][T][Hv][d_v][d_k] float32
 *           out   [R][T][Hv][d_v]      float32
 * ckpt != NULL: state is read only; every position is captured.
 * ckpt == NULL: no capture ([P3] review: rollback storage only when
 *           explicitly requested); chain only; the state after the last
 *           position is written back to `state` (plain decode when T == 1).
 * Tree geometry is checked with hrs_validate_tree(require_chain = 0) for
 * every request before anything is launched. Errors: HRS_EINVAL,
 * HRS_EALIGN, HRS_EGEOMETRY, HRS_EUNSUPPORTED (d_k/d_v outside the built
 * set), HRS_EDEVICE.
 */
int gdn_verify_span(const hrs_gdn_desc* desc, const void* q, const void* k,
                    const void* v, const void* a, const void* b, float* state,
                    float* ckpt, float* out, void* stream);

/* Where a span's initial state comes from when it is not `state`. */
typedef struct {
  const float* ckpt;    /* device: the previous span's checkpoints of this layer,
                           [R][n_pos][Hv][d_v][d_k] float32 */
  const int32_t* node;  /* device [R]: the accepted position of that span
                           (accept_node of accept_greedy) */
  int32_t n_pos;        /* positions of the previous span, in [1, HRS_MAX_POS] */
} hrs_span_source;

/*
 * gdn_verify_span_from - zero-copy rollback: gdn_verify_span whose initial
 * state for request r is src->ckpt[r][src->node[r]], read in place on the
 * device, instead of `state`. Rolling back to the accepted checkpoint then
 * costs nothing: no copy into `state` happens at all ([P3] Summary restores
 * the accepted F32 checkpoint; this reads it where it already is). Capture is
 * required (ckpt != NULL) and ckpt must not overlap src->ckpt, so callers
 * alternate two checkpoint buffers between consecutive spans. A request whose
 * node is outside [0, src->n_pos) writes no checkpoint or output; status
 * (optional device int32, may be NULL) receives the number of such requests.
 * The canonical state can be materialised any time with rollback_restore.
 * Arithmetic, layouts and other errors as gdn_verify_span.
 */
int gdn_verify_span_from(const hrs_gdn_desc* desc, const hrs_span_source* src, const void* q,
                         const void* k, const void* v, const void* a, const void* b, float* ckpt,
                         float* out, int32_t* status, void* stream);

/*
 * gdn_verify_span_timed - gdn_verify_span whose kernel dispatch also records
 * two caller-created hipEvent_t (from the same HIP runtime as `stream`):
 * `start_event` as the kernel starts and `stop_event` as it ends. The events
 * travel inside the dispatch, so no extra command sits between kernels and
 * the interval is the kernel's own execution. Either event may be NULL.
 * Measurement support; arguments, results and errors as gdn_verify_span.
 */
int gdn_verify_span_timed(const hrs_gdn_desc* desc, const void* q, const void* k,
                          const void* v, const void* a, const void* b, float* state,
                          float* ckpt, float* out, void* stream, void* start_event,
                          void* stop_event);

/* Longest span gdn_span_chunked accepts. */
#define HRS_MAX_CHUNKED_POS (1 << 20)

typedef struct {
  hrs_gdn_desc gdn;     /* shapes, input dtype, q_scale; topo must be HRS_CHAIN */
  int32_t log_gates;    /* nonzero: `a` holds log decays g_t = log a_t (<= 0),
                           so a_t = exp(g_t); zero: `a` holds a_t itself */
  hrs_dtype out_dtype;  /* dtype of `out`: HRS_F32, or HRS_BF16 (each output
                           rounded to the nearest bf16, ties to even) */
} hrs_chunked_desc;

/* Bytes of device workspace gdn_span_chunked needs for this descriptor:
 * n_req x n_vheads x min(ceil(n_pos / 64), 32) x 20,992 (one record of T,
 * P T and the decays per request, value head and chunk of a 32-chunk
 * segment; 21.5 MB for one request of 32 heads at any length from 2,048
 * positions). 0 for a NULL descriptor or sizes out of range. */
size_t gdn_span_chunked_workspace_bytes(const hrs_chunked_desc* desc);

/*
 * gdn_span_chunked - the gated delta rule of gdn_verify_span over a long
 * chain span (prefill length, up to HRS_MAX_CHUNKED_POS positions), computed
 * by chunks of 64 positions in the chunkwise form of the delta rule ([GDN]:
 * the hardware-efficient chunkwise algorithm with the WY/UT representation).
 * Inside a chunk starting from state S_0 the written values
 *     w_t = b_t (v_t - a_t S_{t-1} k_t)
 * solve the unit lower-triangular system
 *     w_t + sum_{j<t} b_t G[t][j] (k_t . k_j) w_j = b_t (v_t - g_t S_0 k_t),
 * G[t][j] = a_{j+1}...a_t, g_t = a_0...a_t (products inside the chunk, so
 * zero or tiny decays are exact), i.e. W = T Y with T the inverse of the
 * system's matrix; then S_t = a_t S_{t-1} + w_t k_t^T and o_t = S_t
 * (q_scale q_t) as in gdn_verify_span. Same mathematics, different rounding
 * order: results agree with gdn_verify_span to f32 rounding, not bit for bit.
 *
 * Arguments, layouts and capture as gdn_verify_span, chain only
 * (desc->gdn.topo must be HRS_CHAIN; parent is ignored), with two variants:
 * log-space gates and bf16 outputs (`out` [R][T][Hv][d_v] in out_dtype).
 * ckpt != NULL writes every position's state and leaves `state` unchanged;
 * ckpt == NULL updates `state` in place to the state after the last
 * position. workspace: caller-owned device memory of at least
 * gdn_span_chunked_workspace_bytes(desc) bytes, 16-byte aligned, contents
 * ignored and overwritten (the per-chunk T, P T and decays; spans longer
 * than 32 chunks reuse it segment by segment, two launches per segment).
 * Errors: HRS_EINVAL (sizes, NULL pointers or workspace, a workspace smaller
 * than required, n_pos outside [1, HRS_MAX_CHUNKED_POS], out_dtype),
 * HRS_EALIGN, HRS_EUNSUPPORTED (tree topology; d_k or d_v other than 128),
 * HRS_EDEVICE.
 */
int gdn_span_chunked(const hrs_chunked_desc* desc, const void* q, const void* k, const void* v,
                     const void* a, const void* b, float* state, float* ckpt, void* out,
                     void* workspace, size_t workspace_bytes, void* stream);

typedef struct {
  hrs_gdn_desc gdn;    /* shapes, dtype, q_scale and topology of the span */
  int32_t conv_width;  /* W of the conv; 4 is built                        */
  int32_t silu;        /* nonzero: SiLU after the conv (the layer's order)  */
  float l2_eps;        /* added to |q|^2 and |k|^2 before the square root   */
} hrs_gdn_layer_desc;

/*
 * gdn_layer_verify_span - one GDN layer's verify span in the layer's own
 * order, in one kernel: the causal depthwise conv of the projected channels
 * (as conv1d_verify_span, optional SiLU), split into q, k and v heads, q and
 * k scaled to unit L2 norm per head, then the gated delta rule with a
 * checkpoint after every position (as gdn_verify_span). The conv and
 * recurrent states are the layer's hybrid state ([P2] What Changed); the
 * recurrence and checkpoints are those of gdn_verify_span ([GDN]; [P3]
 * Summary). The conv output never leaves the chip.
 *
 * Per request r and position t with conv output y_t (float32, C channels,
 * C = 2 Hk d_k + Hv d_v, channel order [q heads | k heads | v heads]):
 *     q_t[g] = y_t[g d_k .. ) / sqrt(|.|^2 + l2_eps)
 *     k_t[g] = y_t[Hk d_k + g d_k .. ) / sqrt(|.|^2 + l2_eps)
 *     v_t[h] = y_t[2 Hk d_k + h d_v .. )
 * then ckpt and out exactly as gdn_verify_span with q_scale applied to the
 * normalised q.
 *
 * Layouts:  x          [R][T][C]        gdn.in_dtype
 *           conv_w     [C][W]           gdn.in_dtype; w[c][W-1] multiplies x_t
 *           conv_state [R][W-1][C]      gdn.in_dtype, read only
 *           a, b       [R][T][Hv]       gdn.in_dtype
 *           state      [R][Hv][d_v][d_k] float32, read only
 *           ckpt, out  as gdn_verify_span (ckpt is required)
 * Exactly one of `state` and `src` gives the initial state; with `src` the
 * span starts in place from the previous span's accepted checkpoint as in
 * gdn_verify_span_from (status, optional, counts requests whose node is out
 * of range; they write nothing). The conv state after the accepted position
 * comes from conv_state_advance. Errors: HRS_EINVAL, HRS_EALIGN,
 * HRS_EGEOMETRY, HRS_EUNSUPPORTED (W != 4, d_k/d_v outside the built set),
 * HRS_EDEVICE.
 */
int gdn_layer_verify_span(const hrs_gdn_layer_desc* desc, const void* x, const void* conv_w,
                          const void* conv_state, const void* a, const void* b,
                          const float* state, const hrs_span_source* src, float* ckpt,
                          float* out, int32_t* status, void* stream);

/* ------------------------------------------------------------------------ */
/* Causal depthwise conv1d over the span                                    */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t n_req;     /* R                                                  */
  int32_t n_pos;     /* T                                                  */
  int32_t channels;  /* C, multiple of 8                                   */
  int32_t width;     /* W, conv width; 4 is built                          */
  hrs_dtype dtype;   /* dtype of x, w and the conv state                   */
  int32_t silu;      /* nonzero: y = z / (1 + exp(-z)) after the conv (to  */
                     /* a few ulp: hardware exp2 and reciprocal)           */
  hrs_topology topo;
  const int32_t* parent; /* host [n_req][n_pos] when topo == HRS_TREE      */
} hrs_conv_desc;

/*
 * conv1d_verify_span - causal depthwise conv over the span with the conv
 * state captured after every position ([P2] What Changed: the hybrid state
 * includes the conv state; [P1] Changes: conv state restored on device).
 *
 * For position t with parent p, the window is the parent's conv state
 * (conv_state for the root) followed by x_t, oldest first:
 *     y[r][t][c]        = sum_m w[c][m] window[m][c]     (float32 math)
 *     conv_ckpt[r][t]   = window[1..W-1]                 (exact copies)
 * w[c][W-1] multiplies the current input. No bias.
 *
 * Layouts:  x          [R][T][C]        dtype
 *           w          [C][W]           dtype
 *           conv_state [R][W-1][C]      dtype, oldest row first
 *           conv_ckpt  [R][T][W-1][C]   dtype
 *           y          [R][T][C]        float32
 * conv_ckpt == NULL: no capture, chain only; conv_state is advanced in
 * place to the state after the last position.
 * Errors: HRS_EINVAL, HRS_EALIGN, HRS_EGEOMETRY, HRS_EUNSUPPORTED (W != 4),
 * HRS_EDEVICE.
 */
int conv1d_verify_span(const hrs_conv_desc* desc, const void* x, const void* w,
                       void* conv_state, void* conv_ckpt, float* y, void* stream);

/*
 * conv1d_verify_span_nocapture - conv1d_verify_span that writes only y (chain
 * or tree); conv_state is read only and no per-position conv state is
 * written. With conv_state_advance below this replaces the [T][W-1][C] conv
 * checkpoint: the conv state after any position is the last W-1 entries of
 * [conv_state rows, x along that position's root path], so it can be rebuilt
 * from inputs the caller already holds.
 */
int conv1d_verify_span_nocapture(const hrs_conv_desc* desc, const void* x, const void* w,
                                 const void* conv_state, float* y, void* stream);

typedef struct {
  int32_t n_layers;  /* L */
  int32_t n_req;     /* R */
  int32_t n_pos;     /* T of the span just verified */
  int32_t channels;  /* C, multiple of 8 */
  int32_t width;     /* W; 4 is built */
  hrs_dtype dtype;   /* dtype of x and the conv state */
} hrs_conv_advance_desc;

/*
 * conv_state_advance - conv-state rollback without checkpoints: for every
 * layer l and request r, with n = accept_len[r] + 1 positions on the accepted
 * path path[r][0..n-1] (from accept_greedy),
 *     conv_state[l][r] = last W-1 rows of [conv_state[l][r], x[l][r][path[0]], ...,
 *                                          x[l][r][path[n-1]]]
 * in one launch, reading the index data on the device ([P1] Changes: conv
 * state restored on device). Bit-exact copies of input rows.
 * Layouts: x [L][R][T][C], conv_state [L][R][W-1][C] (dtype); path [R][T],
 * accept_len [R] int32 device. A request whose accept_len is outside [0, T)
 * or whose path holds an index outside [0, T) is left untouched; status
 * (optional device int32) receives the number of such requests.
 * Errors: HRS_EINVAL, HRS_EALIGN, HRS_EUNSUPPORTED (W != 4), HRS_EDEVICE.
 */
int conv_state_advance(const hrs_conv_advance_desc* desc, const void* x, void* conv_state,
                       const int32_t* path, const int32_t* accept_len, int32_t* status,
                       void* stream);

/* ------------------------------------------------------------------------ */
/* Greedy acceptance                                                        */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t n_req;   /* R                                                    */
  int32_t n_pos;   /* T (rows of logits per request)                       */
  int32_t vocab;   /* V, multiple of 8                                     */
  hrs_dtype logit_dtype;
  hrs_topology topo;
  const int32_t* parent; /* host [n_req][n_pos] when topo == HRS_TREE      */
} hrs_accept_desc;

/* Bytes of device workspace accept_greedy needs for this descriptor
 * (0 if the descriptor is invalid). */
size_t accept_greedy_workspace_bytes(const hrs_accept_desc* desc);

/*
 * accept_greedy - greedy verification of one draft block per request
 * ([P2] Summary: greedy request whose output matches plain greedy decoding;
 * [P1] Verification: chain speculative generation and DDTree).
 *
 *  argmax[r][t]  = index of the largest logit of row (r, t); ties go to the
 *                  lowest index; NaN never wins; an all-NaN row gives 0.
 *  A position t >= 1 is matched when its parent is matched and
 *  tokens[r][t] == argmax[r][parent[t]]; the root (t = 0, the committed
 *  token) is always matched.
 *  accept_node[r] = the deepest matched position (lowest index on ties)
 *  accept_len[r]  = its depth = number of accepted drafts
 *  path[r][0..accept_len] = root .. accept_node, then -1 up to T
 *  bonus[r]       = argmax[r][accept_node], the next step's root token
 *
 * Layouts: logits [R][T][V] logit_dtype; tokens [R][T] int32; outputs int32
 * device arrays argmax [R][T], accept_node [R], accept_len [R],
 * path [R][T], bonus [R]. workspace: device scratch of at least
 * accept_greedy_workspace_bytes(desc) bytes, 16-byte aligned, contents
 * ignored on entry. Size limits: n_req * n_pos <= 65535 * 64 and
 * n_req * n_pos * ceil(V / 16384) <= 2^24 (else HRS_EINVAL). Errors:
 * HRS_EINVAL, HRS_EALIGN, HRS_EGEOMETRY, HRS_EDEVICE.
 */
int accept_greedy(const hrs_accept_desc* desc, const void* logits, const int32_t* tokens,
                  int32_t* argmax, int32_t* accept_node, int32_t* accept_len,
                  int32_t* path, int32_t* bonus, void* workspace,
                  size_t workspace_bytes, void* stream);

/* Largest workspace accept_greedy_noalloc can use: 1 MiB, the pass-1 keys of
 * up to 131,072 (row, 16384-logit chunk) pairs (e.g. 272 rows of 151,936
 * logits need 21,760 bytes). */
#define HRS_ACCEPT_NOALLOC_MAX_BYTES (1u << 20)

/*
 * accept_greedy_noalloc - accept_greedy for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation): the pass-1 keys live in a fixed device array of
 * HRS_ACCEPT_NOALLOC_MAX_BYTES inside the library instead of a caller's
 * workspace. The call itself allocates nothing. The array exists once per GPU
 * and stays for the life of the process; its device address is looked up on
 * the first call on each GPU (with that GPU current). Nothing in it needs to
 * start at zero: every key a call reads is written by the same call.
 * Calls that overlap in time on one GPU (different streams, or host threads
 * sharing a GPU) share the array and race; serialise them.
 * Arguments, results and errors as accept_greedy without the workspace,
 * plus HRS_EINVAL when accept_greedy_workspace_bytes(desc) exceeds
 * HRS_ACCEPT_NOALLOC_MAX_BYTES.
 */
int accept_greedy_noalloc(const hrs_accept_desc* desc, const void* logits, const int32_t* tokens,
                          int32_t* argmax, int32_t* accept_node, int32_t* accept_len, int32_t* path,
                          int32_t* bonus, void* stream);

/* ------------------------------------------------------------------------ */
/* On-device rollback                                                       */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t n_layers;      /* L                                              */
  int32_t n_req;         /* R                                              */
  int32_t n_pos;         /* T                                              */
  int32_t n_vheads;      /* Hv                                             */
  int32_t d_k, d_v;
  int32_t conv_channels; /* C (0 with NULL conv buffers: no conv restore)  */
  int32_t conv_width;    /* W                                              */
  hrs_dtype conv_dtype;
} hrs_rollback_desc;

/*
 * rollback_restore - fast rollback: for every layer l and request r,
 *     state[l][r]      = ckpt[l][r][accept_node[r]]
 *     conv_state[l][r] = conv_ckpt[l][r][accept_node[r]]
 * in one launch, with the accepted index read from device memory, so no host
 * round trip sits between acceptance and restore ([P1] Changes: restore
 * split SSM and convolution state on device, synchronize once; [P3]
 * Summary: restore the accepted checkpoint without replay).
 *
 * Layouts:  ckpt       [L][R][T][Hv][d_v][d_k] float32
 *           state      [L][R][Hv][d_v][d_k]    float32
 *           conv_ckpt  [L][R][T][W-1][C]       conv_dtype (may be NULL)
 *           conv_state [L][R][W-1][C]          conv_dtype (NULL with conv_ckpt)
 *           accept_node [R] int32, device
 *           status     one int32, device: written by the launch with the
 *                      number of requests whose accept_node is outside
 *                      [0, T); those requests are left untouched.
 * Errors: HRS_EINVAL (also L * R > 65535, or one (layer, request) state or
 * conv state of 2 GiB or more), HRS_EALIGN, HRS_EDEVICE.
 */
int rollback_restore(const hrs_rollback_desc* desc, const float* ckpt, float* state,
                     const void* conv_ckpt, void* conv_state,
                     const int32_t* accept_node, int32_t* status, void* stream);

/* ------------------------------------------------------------------------ */
/* Feature ring                                                             */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t ring_id;    /* which ring                                        */
  int32_t start_pos;  /* first slot, in [0, n_slots)                       */
  int32_t n_rows;     /* rows in the run, in [0, n_slots]                  */
  int32_t packed_row; /* first row in the packed buffer                    */
} hrs_ring_run;

typedef struct {
  int32_t n_rings;       /* rings (one per request)                        */
  int32_t n_slots;       /* S slots per ring                               */
  int32_t width;         /* D elements per row; D * elem_size % 16 == 0   */
  hrs_dtype dtype;
  int32_t n_packed_rows; /* rows in the packed buffer                      */
  int32_t n_runs;
  const hrs_ring_run* runs; /* host [n_runs]                               */
} hrs_ring_desc;

/*
 * ring_set_2d / ring_get_2d - batched feature-ring synchronisation: a run
 * of n rows starting at slot p occupies slots (p + i) mod S; a wrapping run
 * is split into two non-wrapping runs and every run of the call is copied by
 * one launch ([P1] Changes: one get_2d and one set_2d per non-wrapping run
 * instead of two transfers and a sync per token).
 *
 *   set: ring[id][(p + i) mod S][:] = packed[row + i][:]
 *   get: packed[row + i][:]         = ring[id][(p + i) mod S][:]
 * Layouts: ring [n_rings][S][D], packed [n_packed_rows][D], both dtype.
 * Destinations of one call must not overlap (set: ring slots; get: packed
 * rows), so the result never depends on copy order. Errors: HRS_EINVAL,
 * HRS_EALIGN, HRS_EDEVICE.
 */
int ring_set_2d(const hrs_ring_desc* desc, void* ring, const void* packed, void* stream);
int ring_get_2d(const hrs_ring_desc* desc, const void* ring, void* packed, void* stream);

/* ------------------------------------------------------------------------ */
/* Full-attention layers of the span                                        */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t n_req;      /* R                                                 */
  int32_t n_pos;      /* T: chain up to HRS_MAX_CHUNKED_POS, tree up to
                         HRS_MAX_POS                                       */
  int32_t n_heads;    /* Hq query heads                                    */
  int32_t n_kvheads;  /* Hkv key heads                                     */
  int32_t d;          /* head dim: multiple of 16, at most 256             */
  int32_t rot;        /* rotated elements of a head: multiple of 16, at
                         most d; 0 = no rotation                           */
  hrs_dtype dtype;    /* dtype of q, k, the weights and the outputs        */
  int64_t q_stride;   /* elements from one position's heads to the next    */
  int64_t k_stride;   /* position's, in q and in k (R and T collapse):
                         multiples of 8, at least heads * d; 0 = dense     */
  float eps;          /* added to the mean square                          */
  float weight_offset;/* added to every weight (1.0 for zero-centred ones) */
  int32_t interleaved;/* zero: element i turns with i + rot/2; nonzero: 2i
                         with 2i + 1                                       */
  hrs_topology topo;
  const int32_t* parent; /* host [n_req][n_pos] when topo == HRS_TREE      */
} hrs_qk_desc;

/*
 * qk_norm_rope - RMS norm over each query and key head and the rotation by
 * position, in one pass ([P2] file table: batched Q/K norm and RoPE). Per
 * request r, position t and head, with x the head's d elements:
 *     n[i] = x[i] / sqrt(mean(x^2) + eps) * (weight_offset + w[i])
 *     angle_i = (seq_len[r] + depth(t)) * freq[i],          i < rot / 2
 *     (n[a], n[b]) -> (n[a] cos - n[b] sin, n[b] cos + n[a] sin)
 * for the pair (a, b) of angle i; elements from rot on are not turned.
 * depth(t) is t in a chain and the length of t's root path in a tree. The
 * angle is formed and reduced to a turn in 64 bits, so far positions are
 * exact; the rest is float32, rounded once. q_weight or k_weight NULL: that
 * side is rotated without a norm.
 *
 * Layouts:  q [R][T][Hq][d], k [R][T][Hkv][d]   dtype, strided as above
 *           q_weight, k_weight [d]              dtype (or NULL)
 *           freq    [rot/2] float64             radians per position
 *           seq_len [R] int32, device           tokens before the root
 *           q_out [R][T][Hq][d], k_out [R][T][Hkv][d]  dtype, dense
 * q_out may be q itself, and k_out k, where that side is dense; any other
 * overlap of an output with a buffer of the call is not allowed. Errors:
 * HRS_EINVAL (also R * T > 2^24), HRS_EALIGN, HRS_EGEOMETRY, HRS_EUNSUPPORTED
 * (d, rot), HRS_EDEVICE.
 */
int qk_norm_rope(const hrs_qk_desc* desc, const void* q, const void* k, const void* q_weight,
                 const void* k_weight, const double* freq, const int32_t* seq_len, void* q_out,
                 void* k_out, void* stream);

/* A paged key/value cache. One layer's keys (and, in a buffer of its own, its
 * values) are [n_pages][Hkv][page_size][d]; slot j of request r is row
 * j % page_size of page page_table[r][j / page_size]. A table entry outside
 * [0, n_pages) stands for a page that is not there: its slots take no part in
 * attention and are not written. */
typedef struct {
  int32_t n_pages;
  int32_t page_size;  /* slots per page: a power of two from 16 to 1024    */
  int32_t table_len;  /* entries per request in the page table             */
  hrs_dtype dtype;    /* HRS_BF16 or HRS_F8E4M3 beside bf16 spans, HRS_F32
                         beside f32 spans                                  */
} hrs_cache_desc;

typedef struct {
  int32_t n_req;      /* R                                                 */
  int32_t n_pos;      /* T in [1, HRS_MAX_POS]; 1 = plain decoding         */
  int32_t n_heads;    /* Hq query heads; Hq % Hkv == 0                     */
  int32_t n_kvheads;  /* Hkv key/value heads                               */
  int32_t d;          /* head dim: 64, 128 or 256                          */
  hrs_dtype dtype;    /* dtype of q, k, v and out: HRS_F32 or HRS_BF16     */
  int64_t q_stride;   /* elements from one position's heads to the next    */
  int64_t k_stride;   /* position's (R and T collapse): multiples of 8, at */
  int64_t v_stride;   /* least heads * d; 0 = dense                        */
  float scale;        /* of the scores (1 / sqrt(d) as a rule)             */
  int32_t window;     /* a position sees the last `window` positions, its
                         own among them; 0 = all                           */
  hrs_cache_desc cache;
  hrs_topology topo;
  const int32_t* parent; /* host [n_req][n_pos] when topo == HRS_TREE      */
} hrs_attn_desc;

/* Bytes of device workspace attn_verify_span needs for these sizes (0 for a
 * NULL descriptor or sizes out of range). It does not depend on lengths. */
size_t attn_verify_span_workspace_bytes(const hrs_attn_desc* desc);

/*
 * attn_verify_span - attention of a verify span over a paged cache: the
 * full-attention layers' counterpart of gdn_verify_span ([P2] file table:
 * causal-window attention over pages; [P1] Verification: DDTree). Query
 * (r, t, h), key/value head g = h / (Hq/Hkv), n = seq_len[r]:
 *     out = sum_j w_j v_j,  w = softmax over j of scale (q . k_j)
 * over the context slots j in [0, n) of request r, read from the cache, and
 * the span positions on t's root path (t among them), read from k and v, the
 * span's own rows, which need not be in the cache. With a window W only slots
 * j > n + depth(t) - W and path positions s with depth(t) - depth(s) < W
 * count. Cached e4m3 values stand for k_scale[g], v_scale[g] times themselves
 * (NULL: 1); span rows are taken as they are. What does not count has no
 * influence, whatever it holds (infinities and NaN included). Every position
 * counts itself, so no query is without a score; where all of them are -inf
 * the result is NaN, as the formula's. Sums and softmax statistics are
 * float32. For the product with bf16 values a weight keeps 16 bits, beside
 * e4m3 values it is rounded to float16 (11 bits, and 2^-32 of the row's
 * largest weight at least).
 *
 * Layouts:  q [R][T][Hq][d], k, v [R][T][Hkv][d]  dtype, strided as above
 *           k_cache, v_cache [n_pages][Hkv][page_size][d]  cache.dtype
 *           page_table [R][table_len] int32, seq_len [R] int32, device
 *           k_scale, v_scale [Hkv] float32, device (e4m3 caches only;
 *           4-byte aligned, so rows of an [L][Hkv] array will do)
 *           out [R][T][Hq][d] dtype, dense
 *           workspace: device scratch of at least
 *           attn_verify_span_workspace_bytes(desc) bytes, contents ignored
 * out, status and workspace must not overlap each other or any input. A
 * request whose seq_len is outside [0, table_len * page_size] keeps its rows
 * of out as they were; status (optional device int32) receives the
 * number of such requests. Calls that may run at the same time need
 * workspaces of their own. Errors: HRS_EINVAL (sizes, dtype combination,
 * R > 4096, Hkv > 1024, Hq / Hkv > 64; also where one request's longest table
 * has more than about 2^31 tiles over all heads, or the cache more than 2^32
 * groups of 16 rows), HRS_EALIGN, HRS_EGEOMETRY, HRS_EUNSUPPORTED (d),
 * HRS_EDEVICE.
 */
int attn_verify_span(const hrs_attn_desc* desc, const void* q, const void* k, const void* v,
                     const void* k_cache, const void* v_cache, const int32_t* page_table,
                     const int32_t* seq_len, const float* k_scale, const float* v_scale, void* out,
                     int32_t* status, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace attn_verify_shared needs for these sizes (0 for a
 * NULL descriptor or sizes out of range). It does not depend on lengths, nor on
 * the cache. About twice the bytes of R * T * Hq results in float32 (up to five
 * times those where hundreds of rows a key head leave the card's last round of
 * blocks less than full), and those of the parts of up to 512 blocks. */
size_t attn_verify_shared_workspace_bytes(const hrs_attn_desc* desc);

/*
 * attn_verify_shared - attn_verify_span of requests that share a prefix, whose
 * keys and values are read once for all of them: the rows of all requests are
 * one operand of its products. Slots j < P = prefix_len[0] of every request are
 * those of prefix_table (row j % page_size of page prefix_table[j /
 * page_size]), the others those of the request's own table, at the same place
 * as ever (a request's own entries are not read where all of their slots are
 * below P). seq_len counts both: a request with seq_len[r] < P counts the first
 * seq_len[r] slots of the prefix. Otherwise arguments, layouts, masks, results
 * and refusals are those of attn_verify_span, up to rounding.
 *
 * What is computed for all requests at once are the slots that every one of
 * them counts at every position: from the latest window's start to the shortest
 * context's end within the prefix, in whole groups of 128. What is behind that
 * each request reads for itself, so one short or empty request costs all of
 * them (16 chains of 17 behind 26,758 slots: 246 us, one of them with 13,000
 * slots 345, with none 427). Batches of up to 256
 * requests are one unit (trees: fewer where their positions fill the launch's
 * arguments), larger ones several. In a unit with more than 256 rows (positions
 * times query heads) of a key head, a bf16 span's weights over those slots are
 * rounded once, to bf16 (beside e4m3 values to float16), and it is the rounded
 * weights that are summed.
 *
 * prefix_table [prefix_pages] int32, prefix_len [1] int32, device;
 * prefix_pages >= 1. A prefix_len outside [0, prefix_pages * page_size] refuses
 * all requests (status: R). prefix_table may be part of page_table. workspace:
 * at least attn_verify_shared_workspace_bytes(desc) bytes. Errors as
 * attn_verify_span.
 */
int attn_verify_shared(const hrs_attn_desc* desc, int32_t prefix_pages, const void* q, const void* k,
                       const void* v, const void* k_cache, const void* v_cache,
                       const int32_t* prefix_table, const int32_t* prefix_len,
                       const int32_t* page_table, const int32_t* seq_len, const float* k_scale,
                       const float* v_scale, void* out, int32_t* status, void* workspace,
                       size_t workspace_bytes, void* stream);

typedef struct {
  int32_t n_layers;   /* L                                                 */
  int32_t n_req;      /* R                                                 */
  int32_t n_pos;      /* T of the span; up to HRS_MAX_POS with a path, up to
                         HRS_MAX_CHUNKED_POS without                       */
  int32_t n_kvheads;  /* Hkv                                               */
  int32_t d;          /* head dim: multiple of 16, at most 256             */
  hrs_dtype dtype;    /* dtype of k and v                                  */
  int64_t k_stride;   /* elements from one position's heads to the next    */
  int64_t v_stride;   /* position's (L, R and T collapse): multiples of 8,
                         at least Hkv * d; 0 = dense                       */
  hrs_cache_desc cache;
} hrs_append_desc;

/*
 * kv_cache_append - the accepted rows of a span into the cache pages of every
 * layer, in one launch, with the accepted path read from device memory: the
 * full-attention layers' counterpart of conv_state_advance. For every layer
 * l, request r and i in [0, accept_len[r]], j = seq_len[r] + i:
 *     cache[l][page_table[r][j / page_size]][h][j % page_size]
 *         = span[l][r][path[r][i]][h]                (keys and values)
 *     seq_len_out[r] = seq_len[r] + accept_len[r] + 1
 * path NULL: the identity (chains, prefill). Same dtype: exact copies. e4m3
 * caches: divided by k_scale[l][h], v_scale[l][h] (NULL: 1), limited to
 * +-448 and rounded to the nearest e4m3, ties to even; NaN stays NaN.
 *
 * Layouts:  k, v [L][R][T][Hkv][d] dtype, strided as above
 *           k_cache, v_cache [L][n_pages][Hkv][page_size][d] cache.dtype
 *           page_table [R][table_len], seq_len [R], accept_len [R],
 *           path [R][T] (or NULL) int32, device
 *           k_scale, v_scale [L][Hkv] float32, device (e4m3 caches only;
 *           4-byte aligned)
 *           seq_len_out [R] int32, device: seq_len itself, a buffer apart
 *           from every other one, or NULL
 * The caches and status must not overlap any other buffer of the call.
 * A request is left untouched (seq_len_out[r] = seq_len[r]) and counted in
 * status (optional device int32) when accept_len is outside [0, T), seq_len
 * is negative, seq_len + accept_len + 1 > table_len * page_size, or one of
 * its path entries is outside [0, T). Rows whose page is not there are not
 * written. Two requests of one call must not write the same slot. Errors:
 * HRS_EINVAL (sizes, dtype combination, L or R > 65535, R * T > 2^24),
 * HRS_EALIGN, HRS_EUNSUPPORTED (d), HRS_EDEVICE.
 */
int kv_cache_append(const hrs_append_desc* desc, const void* k, const void* v, void* k_cache,
                    void* v_cache, const int32_t* page_table, const int32_t* seq_len,
                    const int32_t* accept_len, const int32_t* path, const float* k_scale,
                    const float* v_scale, int32_t* seq_len_out, int32_t* status, void* stream);

/* ------------------------------------------------------------------------ */
/* Acceptance by sampling                                                   */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t n_req;   /* R                                                    */
  int32_t n_pos;   /* T (rows of logits per request)                       */
  int32_t vocab;   /* V, multiple of 8                                     */
  hrs_dtype logit_dtype;
  hrs_dtype draft_dtype; /* dtype of draft_probs (ignored without them)    */
  hrs_topology topo;
  const int32_t* parent; /* host [n_req][n_pos] when topo == HRS_TREE      */
} hrs_sample_desc;

/* Bytes of device workspace accept_sample needs for this descriptor
 * (0 if the descriptor is invalid). */
size_t accept_sample_workspace_bytes(const hrs_sample_desc* desc);

/*
 * accept_sample - verification of one draft block per request against the
 * target's probabilities, from given random numbers: the kept tokens and the
 * next one are distributed as if drawn from the target itself. It stands
 * beside accept_greedy for requests that sample. With p_t the softmax of
 * logits[r][t] / temperature[r], x_t = tokens[r][t], u_t = uniforms[r][t]:
 *
 *  With draft_probs (chain only; row t is the distribution q_t that x_{t+1}
 *  was drawn from): starting at the root, t = 1, 2, ... is accepted while
 *      u_t q_{t-1}(x_t) < p_{t-1}(x_t);
 *  at the first position that is not, the rest is max(p_{t-1} - q_{t-1}, 0).
 *  Without draft_probs (chain or tree; drafts were picked, not drawn): at a
 *  node n the rest starts as p_n; n's children are tried in index order, and
 *  child t is accepted, and the walk goes on from it, when
 *      u_t (1 - sum of p_n over the tokens already rejected at n) < p_n(x_t);
 *  a token that is not accepted is taken out of the rest (a second child
 *  with the same token is never accepted).
 *  accept_node, accept_len, path: the last accepted position, its depth and
 *  root path (then -1), as accept_greedy.
 *  bonus[r] = the first v in index order with a positive weight and
 *      weight(0) + ... + weight(v) > u_0 (total weight)
 *  where weight is the rest at accept_node (p itself where every draft of the
 *  chain was accepted, where the node has no children, or where the rest is
 *  zero everywhere); the last v with a positive weight if there is none.
 *  token_prob[r][t] = p_{parent(t)}(x_t), float32; 1 for the root.
 *
 * Random numbers are meant to be in [0, 1) and independent. A NaN logit has
 * probability zero; +inf logits share the whole probability; a row without
 * any finite or +inf logit has p = 0 everywhere and bonus 0. Temperature 0 is
 * the limit (the largest logits share the probability); NULL means 1. A
 * token outside [0, V) has probability zero. A request whose temperature is
 * negative or NaN keeps its outputs as they were; status (optional device
 * int32) receives the number of such requests. Probabilities are float32
 * with 64-bit sums; the bonus draw (weights, total and cumulative sums) is in
 * 64 bits, where the border of a long float32 sum would decide.
 *
 * Layouts:  logits [R][T][V] logit_dtype; tokens [R][T] int32;
 *           uniforms [R][T] float32; draft_probs [R][T][V] draft_dtype or
 *           NULL; temperature [R] float32 or NULL; token_prob [R][T] float32;
 *           accept_node, accept_len, bonus [R], path [R][T] int32; all
 *           device. workspace: device scratch of at least
 *           accept_sample_workspace_bytes(desc) bytes, contents ignored.
 * Outputs and workspace must not overlap each other or any input.
 * Size limits as accept_greedy, R <= 65535 and V <= 2^30. Errors: HRS_EINVAL,
 * HRS_EALIGN, HRS_EGEOMETRY, HRS_EUNSUPPORTED (draft_probs with a tree),
 * HRS_EDEVICE.
 */
int accept_sample(const hrs_sample_desc* desc, const void* logits, const int32_t* tokens,
                  const float* uniforms, const void* draft_probs, const float* temperature,
                  float* token_prob, int32_t* accept_node, int32_t* accept_len, int32_t* path,
                  int32_t* bonus, int32_t* status, void* workspace, size_t workspace_bytes,
                  void* stream);

/* Bytes of device workspace accept_sample_filtered needs for this descriptor
 * (0 if the descriptor is invalid): about 2 KiB for every 8192 logits and
 * 8 KiB a row. */
size_t accept_sample_filtered_workspace_bytes(const hrs_sample_desc* desc);

/*
 * accept_sample_filtered - accept_sample for requests that sample from the
 * target's probabilities after top-k, top-p and min-p. The tokens of row
 * (r, t) stand in the order of their logits, largest first, equal ones by
 * index, NaN left out; w_i = e^((z_i - z_0) / temperature[r]) is the weight of
 * the i-th. The first n = min(n_k, n_p, n_m) of them stay:
 *     n_k = top_k[r] (all where it is outside [1, V], or without top_k)
 *     n_p = the smallest n with w_0 + ... + w_{n-1} >= top_p[r] (w_0 + ... +
 *           w_{n_k - 1}), at least 1 (all from top_p[r] = 1 on, for NaN, or
 *           without top_p)
 *     n_m = how many have w_i >= min(min_p[r], 1) (all up to min_p[r] = 0,
 *           for NaN, or without min_p)
 * and p_t is their weights divided by their sum, zero elsewhere. Everything
 * else as accept_sample, whose results it gives without limits; n_pos = 1 is
 * plain sampling (bonus). Weights below e^-48 of the largest count as none.
 * Borders are decided on 64-bit sums of weights in 64 bits where a row is
 * settled by its largest few hundred logits or a bf16 row by how often each
 * value is there; the total that a top-p without a top-k is a share of, where
 * such a row has weights behind those, is good to 18 units of 2^-24, and so is
 * the sum of a row without limits. Other rows' weights are good to 3 units, and
 * their sum, of whole numbers, to V 2^-51 more. The draw is in 64 bits.
 *
 * Layouts: as accept_sample; top_k [R] int32, top_p, min_p [R] float32, device,
 *          each or NULL; workspace of at least
 *          accept_sample_filtered_workspace_bytes(desc) bytes.
 * Overlaps, refused requests (by their temperature), status, size limits and
 * errors as accept_sample.
 */
int accept_sample_filtered(const hrs_sample_desc* desc, const void* logits, const int32_t* tokens,
                           const float* uniforms, const void* draft_probs, const float* temperature,
                           const int32_t* top_k, const float* top_p, const float* min_p,
                           float* token_prob, int32_t* accept_node, int32_t* accept_len,
                           int32_t* path, int32_t* bonus, int32_t* status, void* workspace,
                           size_t workspace_bytes, void* stream);

typedef struct {
  int32_t n_req;     /* R                                                  */
  int32_t n_pos;     /* T of the span, in [1, HRS_MAX_POS]                 */
  int32_t n_pages;   /* pages, slots of a page and entries of a request's  */
  int32_t page_size; /* table, as hrs_cache_desc                           */
  int32_t table_len;
} hrs_hold_desc;

/*
 * accept_hold - takes the requests that cannot go on out of an acceptance,
 * between accept_greedy or accept_sample and the entry points that commit it
 * ([P3] Safety boundary: rejected before execution). A request goes on if
 * held[r] is 0, its temperature is not negative or NaN, accept_len[r] and
 * accept_node[r] are in [0, T), path[r][0..accept_len[r]] too, and slots
 * seq_len[r] .. seq_len[r] + accept_len[r] lie inside its page table, in
 * pages that are there. Then last_node[r] = accept_node[r]. Otherwise
 *     accept_node[r] = accept_len[r] = bonus[r] = -1,  path[r][:] = -1
 * and, where held[r] was 0, held[r] = 1 and held_node[r] = last_node[r].
 * rollback_restore, conv_state_advance, kv_cache_append and the next
 * gdn_verify_span_from or gdn_layer_verify_span all leave a request with
 * such indices as it is, so none of its state moves, in this step or later
 * ones, until the caller clears held[r]. Its recurrent state then still is in
 * the checkpoint buffer that this step's spans started from, at held_node[r].
 *
 * Layouts:  page_table [R][table_len], seq_len [R] int32, temperature [R]
 *           float32 or NULL (1); accept_node, accept_len, bonus, held,
 *           last_node [R] and path [R][T] int32, read and written; held_node
 *           [R] int32 or NULL (spans that started from `state`); all device.
 *           No two of them overlap.
 * Errors: HRS_EINVAL (R > 65535; sizes as hrs_cache_desc), HRS_EALIGN,
 * HRS_EDEVICE.
 */
int accept_hold(const hrs_hold_desc* desc, const int32_t* page_table, const int32_t* seq_len,
                const float* temperature, int32_t* accept_node, int32_t* accept_len, int32_t* path,
                int32_t* bonus, int32_t* held, int32_t* last_node, int32_t* held_node, void* stream);

/*
 * accept_hold_behind - accept_hold of requests behind a prefix that all of them
 * read: a request whose seq_len[r] is below prefix_len is held too, since its
 * rows would go into the prefix's pages, or into slots that are read there.
 * Errors as accept_hold; HRS_EINVAL also for prefix_len < 0.
 */
int accept_hold_behind(const hrs_hold_desc* desc, int32_t prefix_len, const int32_t* page_table,
                       const int32_t* seq_len, const float* temperature, int32_t* accept_node,
                       int32_t* accept_len, int32_t* path, int32_t* bonus, int32_t* held,
                       int32_t* last_node, int32_t* held_node, void* stream);

/* ------------------------------------------------------------------------ */
/* Page lists                                                               */
/* ------------------------------------------------------------------------ */

typedef struct {
  int32_t n_req;     /* R in [1, 4096]                                     */
  int32_t n_pos;     /* new positions of a request at most, in
                        [1, HRS_MAX_CHUNKED_POS] (release: ignored but for
                        that range)                                        */
  int32_t n_pages;   /* pages, slots of a page and entries of a request's  */
  int32_t page_size; /* table, as hrs_cache_desc                           */
  int32_t table_len;
  int32_t n_prefix;  /* leading entries of every table that hold the pages
                        of a prefix shared by all requests; 0 = none. Whole
                        pages of it: new positions are written behind them */
} hrs_pages_desc;

/* Bytes of device workspace the two calls need for this descriptor (0 if it
 * is invalid). */
size_t kv_pages_workspace_bytes(const hrs_pages_desc* desc);

/*
 * kv_pages_reserve - pages for the new positions of every request, from a
 * free list on the device, and their slots ([P2] What Changed: the hybrid
 * state includes the KV cache; [P1] Changes: nothing through the host). The
 * list is a stack free_pages[0 .. n_free). With S = page_size,
 * m = n_new[r] (NULL: n_pos), request r needs
 *     need_r = max(0, ceil((seq_len[r] + m) / S) - max(n_held[r], n_prefix))
 * pages beyond those it holds (table entries [0, n_held[r])) and the prefix's.
 * It is served where need_0 + ... + need_r <= n_free: in request order until
 * the list is used up. Requests that need nothing are always served. The
 * pages of all served requests are the last ones of the list, in request
 * order, each request's in the order of its entries. Then
 *     page_table[r][n_held[r] .. n_prefix) = prefix_table[same]
 *     page_table[r][max(n_held[r], n_prefix) + i] = its i-th page
 *     n_held[r] = max(n_held[r], n_prefix) + (its pages), n_free -= all pages
 *     slot_map[r][t] = page * S + j % S of j = seq_len[r] + t, t < m, in
 *         entry j / S of the table as it is then; -1 where that entry is not
 *         held or names no page, and for t >= m
 * A request that is not served gets no page (the prefix's excepted). One
 * whose seq_len is negative, n_new outside [0, n_pos], n_held outside
 * [0, table_len] or that would need more than table_len entries is left as it
 * is, with a slot map of -1. status (optional device int32) receives the
 * number of both. n_free outside [0, n_pages] counts as the nearest of these.
 *
 * Layouts: seq_len, n_new, n_held [R], prefix_table [n_prefix] (NULL with
 *          n_prefix 0), page_table [R][table_len], free_pages [n_pages],
 *          n_free [1] int32; slot_map [R][n_pos] int64 or NULL; all device.
 *          workspace: device scratch of at least kv_pages_workspace_bytes(desc)
 *          bytes, contents ignored.
 * page_table, n_held, n_free, slot_map, status and workspace overlap nothing
 * else of the call. Errors: HRS_EINVAL, HRS_EALIGN, HRS_EDEVICE.
 */
int kv_pages_reserve(const hrs_pages_desc* desc, const int32_t* seq_len, const int32_t* n_new,
                     const int32_t* prefix_table, int32_t* page_table, int32_t* n_held,
                     const int32_t* free_pages, int32_t* n_free, int64_t* slot_map, int32_t* status,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * kv_pages_reserve_step - kv_pages_reserve for the spans of a verify step, of
 * which a part is accepted: positions behind the last slot of a request's table
 * are left out (m is at most table_len * S - seq_len[r]; -1 in the slot map)
 * where kv_pages_reserve refuses the request, and a request with
 * skip[r] != 0 (accept_hold's held; [R] int32, device, or NULL) takes nothing
 * and is left as it is, with a slot map of -1 and without being counted in
 * status: what it would take is for those behind it. Layouts, overlaps and
 * errors as kv_pages_reserve.
 */
int kv_pages_reserve_step(const hrs_pages_desc* desc, const int32_t* seq_len, const int32_t* n_new,
                          const int32_t* skip, const int32_t* prefix_table, int32_t* page_table,
                          int32_t* n_held, const int32_t* free_pages, int32_t* n_free,
                          int64_t* slot_map, int32_t* status, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * kv_pages_release - the counterpart: every request keeps the pages of its
 * first keep_len[r] slots (0: a request that has ended) and the prefix's.
 * Entries [max(ceil(keep_len[r] / S), n_prefix), n_held[r]) go back on top of
 * the list, in request order and the order of the entries, and become -1;
 * n_held[r] becomes their start. Entries that name no page are dropped, and so
 * is what the list has no place for. What kv_pages_reserve gave, given back by
 * the next call, restores list and tables. The same page must not be in two
 * tables behind the prefix. A request whose keep_len is negative or n_held
 * outside [0, table_len] is left as it is; status (optional device int32)
 * receives their number. Layouts, overlaps and errors as kv_pages_reserve
 * (free_pages is written).
 */
int kv_pages_release(const hrs_pages_desc* desc, const int32_t* keep_len, int32_t* page_table,
                     int32_t* n_held, int32_t* free_pages, int32_t* n_free, int32_t* status,
                     void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Misc                                                                     */
/* ------------------------------------------------------------------------ */

/* Static description of a status code; never NULL. */
const char* hrs_strerror(int status);

/* HRS_ABI_VERSION of the built library. */
int hrs_abi_version(void);

/* hipError_t of the last launch an entry point made on the calling thread
 * (0 = success): the detail behind HRS_EDEVICE. Per-thread. */
int hrs_last_hip_error(void);

/* hipGetErrorString() of hrs_last_hip_error(); never NULL. */
const char* hrs_last_hip_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* HRS_H */
