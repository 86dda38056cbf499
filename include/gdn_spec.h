/*
 * gdn_spec.h -- C ABI of libgdnspec: ReplaySSM ring spec-verify for one
 * Gated DeltaNet (GDN) linear-attention layer, and its KDA variant (one gate
 * per key channel), on a single GB300 GPU (sm_103a).
 *
 * Sources (web pages, cited by title and section):
 *   [blog]    "PR #28695 详解：GDN ReplaySSM Ring Spec-Verify" (yuyanqi.com)
 *   [pr28695] prhub summary of sglang PR #28695 "[GDN] Support ReplaySSM Ring
 *             Spec-Verify"
 *   [pr33102] prhub report of sglang PR #33102 "fused replayssm ring write into
 *             flashinfer gdn mtp verify kernel"
 *   [pr36821] prhub summary of sglang PR #36821 (fused KDA verify with the
 *             ReplaySSM ring write)
 *
 * The layer keeps, per cache slot (one slot per request):
 *   - a frozen fp32 checkpoint state S0                  [num_slots, HV, V, K]
 *   - a ring of L raw records of committed and draft tokens:
 *       rawv [num_slots, HV, L, V], rawk [num_slots, H, L, K] (I/O dtype,
 *       bitwise copies of the inputs, k before its L2 norm), g and beta fp32
 *       ([blog] appendix A.1; [pr36821] ring layout; [pr33102] test anchor 2)
 *   - three cursors shared by all layers of the model ([blog] §4.1, §10.2):
 *       write_pos  committed-but-unfolded records in the ring,
 *       cache_base ring position of the oldest of them,
 *       is_flush   set by commit when the next window might not fit.
 * Record o (0 <= o < write_pos) sits at ring position (cache_base + o) & (L-1);
 * the draft window of a verify is written at (cache_base + write_pos + s) &
 * (L-1), s < T ([blog] §10.1).
 *
 * The recurrence (decay, then delta against the decayed state; [blog] §12.1):
 *   g = -exp(A_log) * softplus(a + dt_bias), beta = sigmoid(b)
 *   k^ = k / sqrt(|k|^2 + l2_eps), q^ likewise
 *   S_t = exp(g_t) S_{t-1} (I - beta_t k^_t k^_t^T) + beta_t v_t k^_t^T
 *         (KDA: S_{t-1} diag(exp(g_t)) in place of exp(g_t) S_{t-1})
 *   o_t = scale * S_t q^_t
 *
 * Calls and their order per decode step: gdn_spec_verify once per layer
 * inside the forward; after sampling, gdn_spec_commit once; then
 * gdn_spec_fold once over all layers (it does work only for slots whose
 * is_flush was set).  gdn_spec_reset at the prefill -> decode handoff.
 *
 * Conventions for every call:
 *   - All tensor pointers are caller-owned DEVICE memory of the current CUDA
 *     device; the library never allocates, frees or copies them, and keeps no
 *     pointer after the call returns.  Descriptor structs are read on the
 *     host during the call only.
 *   - Tensors are dense, row-major in the shapes given, base addresses 16-byte
 *     aligned.
 *   - Calls are asynchronous and ordered on `stream` (a cudaStream_t, passed
 *     as void*; NULL is the legacy default stream).  They do not synchronise
 *     and do not allocate, so they can be captured into a CUDA graph, except
 *     gdn_spec_read_status, which synchronises.
 *   - Slots named in one call must be distinct; `slot_idx[b] < 0` marks a
 *     padding row, which reads and writes nothing (verify writes zeros to
 *     its output rows).
 *   - Return value: 0 on success, a negative GDN_SPEC_E* code for an error
 *     the host can see (nothing is launched then).  Conditions only the
 *     device can see never trap: the kernel ORs a GDN_SPEC_ST_* bit into
 *     *status, skips the row, and verify writes zeros to its outputs.
 */
#ifndef GDN_SPEC_H
#define GDN_SPEC_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_SPEC_ABI_VERSION 6   /* 2: adds gdn_spec_prefill and the snapshot comparison calls;
                                    3: adds gdn_spec_verify_d, gdn_spec_set_wait_limit, commit's
                                       cursor check and the poisoning of rows a fold or prefill
                                       could not finish;
                                    4: adds gdn_spec_prefill_path, the chunk-parallel prefill and
                                       the tensor-core KDA verify ("tc_kda");
                                    5: adds the softmax-attention layers' step: gdn_spec_tree_attn,
                                       gdn_spec_rope and gdn_spec_rope_append, and the paged cache
                                       gdn_spec_kv_*;
                                    6: adds prompts through the softmax-attention layers:
                                       gdn_spec_prompt_attn, gdn_spec_norm_rope, its gradient and
                                       gdn_spec_norm_rope_append */

/* host-side error codes (return values) */
#define GDN_SPEC_OK            0
#define GDN_SPEC_EINVAL       -1   /* null pointer, bad size, L not a power of two or L < 2T, H does not divide HV */
#define GDN_SPEC_EDTYPE       -2   /* unknown io_dtype or gate_kind */
#define GDN_SPEC_EALIGN       -3   /* a base pointer not 16-byte aligned, or K / V not a multiple of 8 */
#define GDN_SPEC_ECUDA        -4   /* a CUDA call or launch failed */
#define GDN_SPEC_EUNSUPPORTED -5   /* shape outside what the kernels handle (see gdn_spec_verify) */

/* device-side status bits, ORed into cursors->status */
#define GDN_SPEC_ST_ACCEPT_RANGE   1u  /* commit: accept_len < 0 or > T                  */
#define GDN_SPEC_ST_SLOT_OOR       2u  /* slot_idx[b] >= num_slots                        */
#define GDN_SPEC_ST_RING_OVERFLOW  4u  /* verify: write_pos + T > L (a fold was skipped)  */
#define GDN_SPEC_ST_CURSOR_CORRUPT 8u  /* write_pos < 0, write_pos > L or cache_base outside [0, L) */
#define GDN_SPEC_ST_TIMEOUT       16u  /* a bounded device wait ran out: that call's outputs are invalid.
                                              verify: the CTA that saw it drains its copies and stops, so
                                              rows it had not reached keep whatever `out` held and their
                                              window records may be missing from the ring (do not commit
                                              that step).  fold / prefill: every row with an unfinished
                                              item is poisoned (write_pos = -1, so later calls report
                                              CURSOR_CORRUPT for it); its checkpoint may be partly folded
                                              or partly prefilled, so the slot must be rebuilt:
                                              gdn_spec_reset, then gdn_spec_prefill. */
#define GDN_SPEC_ST_UNFOLDED      32u  /* prefill: continuing from a checkpoint whose ring is not folded */
#define GDN_SPEC_ST_NO_PAGES      64u  /* kv_reserve, kv_fork: not enough free pages or table columns for
                                              the row; other calls: the slot's pages do not hold its tokens */
#define GDN_SPEC_ST_PAGE_OOR     128u  /* a page table entry in use is outside [0, num_pages): the row's
                                              outputs are not valid */
#define GDN_SPEC_ST_SLOT_BUSY    256u  /* kv_fork: the destination slot holds tokens or pages */

#define GDN_SPEC_GATE_SCALAR  0    /* GDN: one gate per (token, v-head)            */
#define GDN_SPEC_GATE_PER_KEY 1    /* KDA: one gate per (token, v-head, key channel) */

#define GDN_SPEC_DTYPE_BF16 0
#define GDN_SPEC_DTYPE_FP32 1

/* One GDN layer: dimensions, numerics and its per-slot state. */
typedef struct {
    int32_t H;          /* q/k heads                                               */
    int32_t HV;         /* v heads; H divides HV; v-head hv uses q/k head hv / (HV/H) */
    int32_t K;          /* key dim: 32, 64 or 128                                  */
    int32_t V;          /* value dim (multiple of 8)                               */
    int32_t T;          /* draft window (tokens per row per verify), 1..16         */
    int32_t L;          /* ring length: a power of two, >= 2T ([pr28695] config check) */
    int32_t num_slots;  /* slots in the pool                                       */
    int32_t gate_kind;  /* GDN_SPEC_GATE_SCALAR or GDN_SPEC_GATE_PER_KEY           */
    int32_t io_dtype;   /* dtype of q, k, v, a, b, out, rawv, rawk                 */
    float   scale;      /* output scale (1.0 unless the model scales q)            */
    float   l2_eps;     /* epsilon inside the square root of the q/k L2 norm (1e-6) */
    float  *checkpoint; /* fp32 [num_slots, HV, V, K]                              */
    void   *rawv;       /* io_dtype [num_slots, HV, L, V]                          */
    void   *rawk;       /* io_dtype [num_slots, H, L, K]                           */
    float  *ring_g;     /* fp32 [num_slots, HV, L] (GATE_PER_KEY: [num_slots, HV, L, K]) */
    float  *ring_beta;  /* fp32 [num_slots, HV, L]                                 */
} gdn_spec_layer;

/* Per-slot cursors, shared by every layer of the model, and the status word. */
typedef struct {
    int32_t  num_slots;
    int32_t *write_pos;   /* [num_slots] */
    int32_t *cache_base;  /* [num_slots] */
    int32_t *is_flush;    /* [num_slots] */
    uint32_t *status;     /* [1], device status bits; cleared only by gdn_spec_read_status */
} gdn_spec_cursors;

/*
 * gdn_spec_verify -- output of the whole draft window of every batch row,
 * from the frozen checkpoint plus the ring history, without materialising
 * any per-draft state ([blog] §1.1, §4.1, §5.1; [pr28695] implementation
 * item 3).  Also writes the window's raw records into the ring at
 * (cache_base + write_pos + s) & (L-1) as a side channel: rawv/rawk are
 * bitwise copies of v/k, g/beta the fp32 gate values the kernel computed;
 * the output does not depend on whether the ring positions held anything
 * before ([pr33102] test anchors 1-2; [pr36821] ring write placement).
 * Checkpoint and cursors are only read.
 *
 *   slot_idx  int32 [B]            slot of each row; < 0 marks a padding row
 *   q, k      io_dtype [B, T, H, K]
 *   v         io_dtype [B, T, HV, V]
 *   a         io_dtype [B, T, HV]   (GATE_PER_KEY: [B, T, HV, K])
 *   b         io_dtype [B, T, HV]
 *   A_log     fp32 [HV]
 *   dt_bias   fp32 [HV]             (GATE_PER_KEY: [HV, K])
 *   out       io_dtype [B, T, HV, V]  (written)
 *
 * Device status: SLOT_OOR, CURSOR_CORRUPT, RING_OVERFLOW (the row is skipped
 * and its outputs are zero).  Supported shapes: K in {32, 64, 128}; L <= 128
 * (GATE_SCALAR) or L <= 64 (GATE_PER_KEY); T <= 16; otherwise
 * GDN_SPEC_EUNSUPPORTED.
 */
int gdn_spec_verify(const gdn_spec_layer *layer, const gdn_spec_cursors *cursors,
                    const int32_t *slot_idx, int32_t B,
                    const void *q, const void *k, const void *v, const void *a,
                    const void *b, const float *A_log, const float *dt_bias, void *out,
                    void *stream);

/*
 * gdn_spec_verify_d -- comparison variant of gdn_spec_verify for a ring that
 * also caches every token's corrected delta d_t = beta_t (v_t - S_t^- k^_t)
 * (S_t^- the state after token t's decay): the first design of [blog] §12.1
 * and appendix A.1.  With the history's d cached the verify solves only the
 * window's T x T system; with T = 1 (plain decode) no system at all ([blog]
 * §12.2, §12.9, Part A).  Outputs as gdn_spec_verify; writes the window's raw
 * records into the ring and the window's d into `dring` at the same positions
 * (cache_base + write_pos + s) & (L-1).  The checkpoint and cursors are only
 * read; commit, fold (which replays the raw records, so the cached d never
 * reach the checkpoint) and reset are the ring path's.  A layer that uses it
 * must use it for every verify since its last prefill or reset, so that
 * every committed record's d is in the d ring.
 *   dring  fp32 [num_slots, HV, L, V]   (caller-owned device memory)
 *   other arguments as gdn_spec_verify.
 * Supported shapes: bf16 I/O, GATE_SCALAR, K = 128, V a multiple of 128,
 * L <= 64, T <= 8; otherwise GDN_SPEC_EUNSUPPORTED.
 */
int gdn_spec_verify_d(const gdn_spec_layer *layer, float *dring, const gdn_spec_cursors *cursors,
                      const int32_t *slot_idx, int32_t B, const void *q, const void *k,
                      const void *v, const void *a, const void *b, const float *A_log,
                      const float *dt_bias, void *out, void *stream);

/*
 * gdn_spec_commit -- after sampling: for each row with a slot,
 *   write_pos += accept_len[b];  is_flush = (write_pos + 2T > L)
 * ([blog] §4.2, §8.1-8.2: the early-flush margin keeps one more window in the
 * ring).  Rejected drafts cost nothing: their records stay past write_pos and
 * are overwritten by the next verify ([blog] §4.2-4.3).
 *   accept_len  int32 [B], device; 0 <= accept_len <= T (it counts the bonus
 *               token); outside that the row is skipped with ACCEPT_RANGE.
 * A row whose cursors are out of range (write_pos outside [0, L], cache_base
 * outside [0, L)) is skipped with CURSOR_CORRUPT and left as it is.
 */
int gdn_spec_commit(const gdn_spec_cursors *cursors, int32_t T, int32_t L,
                    const int32_t *slot_idx, int32_t B, const int32_t *accept_len,
                    void *stream);

/*
 * gdn_spec_fold -- exact fold ([pr28695] implementation item 3; [blog] §12.7):
 * for every row whose slot has is_flush set, replay its write_pos committed
 * raw records into the checkpoint of every one of the n_layers layers with the
 * recurrence itself (token by token, fp32), then set
 *   cache_base = (cache_base + write_pos) & (L-1), write_pos = 0, is_flush = 0.
 * Rows without is_flush are left alone, so calling it every step is cheap and
 * calling it twice is harmless.  All layers must have the same dimensions,
 * gate kind and io dtype.  `layers` is a host array of n_layers descriptors.
 */
int gdn_spec_fold(const gdn_spec_layer *layers, int32_t n_layers,
                  const gdn_spec_cursors *cursors, const int32_t *slot_idx, int32_t B,
                  void *stream);

/*
 * gdn_spec_reset -- prefill -> decode handoff ([blog] appendix A.2): for each
 * row with a slot, write_pos = cache_base = 0 and is_flush = 0.  The caller
 * has written that slot's checkpoint.
 */
int gdn_spec_reset(const gdn_spec_cursors *cursors, const int32_t *slot_idx, int32_t B,
                   void *stream);

/*
 * gdn_spec_prefill -- prefill of each row's N prompt tokens into its slot
 * (the step before decode; the reset of the prefill -> decode handoff,
 * [blog] appendix A.2, is part of it): for every v-head the recurrence runs
 * over the tokens from a zero state (from_zero != 0) or from the slot's
 * checkpoint (from_zero == 0, which gives chunked prefill across calls);
 * every token's output is written, the final state becomes the slot's
 * checkpoint, and the slot's cursors are reset (write_pos = cache_base =
 * is_flush = 0).  The ring is not written.  Two kernels (gdn_spec_prefill_path
 * names the one a layer uses): "chunk" -- scalar gate, bf16 I/O, K = 128 and V
 * a multiple of 128 -- the chunk-parallel UT form on the tensor cores, 64
 * tokens per step ([blog] appendix B.1 names chunk_gated_delta_rule as the
 * prefill authority; tf32 operands, the state update split into tf32 high and
 * low parts); "sequential" -- every other shape, token by token in fp32 as
 * the fold does.
 *   q, k      io_dtype [B, N, H, K]
 *   v         io_dtype [B, N, HV, V]
 *   a         io_dtype [B, N, HV]   (GATE_PER_KEY: [B, N, HV, K])
 *   b         io_dtype [B, N, HV]
 *   A_log     fp32 [HV];  dt_bias fp32 [HV] (GATE_PER_KEY: [HV, K])
 *   out       io_dtype [B, N, HV, V]  (written)
 * N >= 0 (N = 0 only zeroes the checkpoints when from_zero, and resets).
 * Device status: SLOT_OOR, CURSOR_CORRUPT, and UNFOLDED when from_zero == 0
 * and the slot's write_pos is not 0 (committed records not yet folded: fold
 * them first); such a row is skipped (its checkpoint and cursors untouched,
 * its outputs zero).
 */
int gdn_spec_prefill(const gdn_spec_layer *layer, const gdn_spec_cursors *cursors,
                     const int32_t *slot_idx, int32_t B, int32_t N,
                     const void *q, const void *k, const void *v, const void *a,
                     const void *b, const float *A_log, const float *dt_bias, void *out,
                     int32_t from_zero, void *stream);

/*
 * Comparison variant, not part of the ring path: the per-draft snapshot
 * design that the ReplaySSM ring replaces ([blog] §0-§1: the intermediate_ssm
 * buffer, one full state per draft position), kept so that its cost can be
 * measured beside the ring on the same machine.
 *
 * gdn_spec_snapshot_verify -- for every row and v-head, from the slot's
 * checkpoint, advance through the T window tokens, write every position's
 * output and store the full state after every position:
 *   snap      fp32 [B, T, HV, V, K]  (written; caller-owned; T V K 4 bytes
 *             per (row, v-head): 256 KiB at the Qwen3-Next shape and T = 4)
 *   q, k, v, a, b, A_log, dt_bias, out: as gdn_spec_verify.
 * The checkpoint is only read; cursors and ring are not used (the status
 * word records SLOT_OOR).
 *
 * gdn_spec_snapshot_commit -- checkpoint[slot_idx[b]] = snap[b, accept_len[b]
 * - 1] for 1 <= accept_len <= T (0 keeps the state; outside [0, T]:
 * ACCEPT_RANGE); accept_len int32 [B], device.
 */
int gdn_spec_snapshot_verify(const gdn_spec_layer *layer, const gdn_spec_cursors *cursors,
                             const int32_t *slot_idx, int32_t B,
                             const void *q, const void *k, const void *v, const void *a,
                             const void *b, const float *A_log, const float *dt_bias, void *out,
                             float *snap, void *stream);
int gdn_spec_snapshot_commit(const gdn_spec_layer *layer, const gdn_spec_cursors *cursors,
                             const int32_t *slot_idx, int32_t B, const int32_t *accept_len,
                             const float *snap, void *stream);

/*
 * gdn_spec_set_wait_limit -- diagnostic: the number of polls after which the
 * first wait on each asynchronous data copy gives up (verify's checkpoint
 * tile on the tensor-core path, the fold's ring records, prefill's prompt
 * chunks).  A wait that gives up sets GDN_SPEC_ST_TIMEOUT; the copy is then
 * drained with the default limit before its buffer is reused, so a small
 * limit exercises the timeout path without leaving anything in flight.
 * Applies to calls made (or graphs captured) afterwards, in every thread of
 * the process.  0xFFFFFFFF restores the default (2^20 polls of at most about
 * 256 ns each: 0.3 s at most).
 * Returns the previous limit.  Not for production use.
 */
uint32_t gdn_spec_set_wait_limit(uint32_t polls);

/*
 * gdn_spec_read_status -- copy the device status word to *host_out after
 * synchronising `stream`; clears it on the device when `clear` is non-zero.
 * Not for use inside a captured graph.
 */
int gdn_spec_read_status(const gdn_spec_cursors *cursors, uint32_t *host_out, int32_t clear,
                         void *stream);

/* Text for a GDN_SPEC_E* code. */
const char *gdn_spec_strerror(int code);

/* GDN_SPEC_ABI_VERSION of the loaded library. */
int gdn_spec_abi_version(void);

/* Name of the verify kernel gdn_spec_verify would launch for this layer
 * ("tc" = TMA + tcgen05 path for the scalar gate, "tc_kda" = TMA + tcgen05
 * path for the per-key gate, "generic" = CUDA-core path), or NULL if the
 * layer is invalid.  Host only; launches nothing. */
const char *gdn_spec_verify_path(const gdn_spec_layer *layer);

/* Name of the prefill kernel gdn_spec_prefill would launch for this layer
 * ("chunk" = chunk-parallel tensor-core path, "sequential" = token-by-token
 * CUDA-core path), or NULL if the layer is invalid.  Host only; launches
 * nothing. */
const char *gdn_spec_prefill_path(const gdn_spec_layer *layer);

/* ======================================================================
 * The softmax-attention layers of a hybrid model: a speculative step over a
 * paged key/value cache.  Per layer: gdn_spec_rope_append (rotary positions,
 * the window's keys and values written behind the committed tokens), then
 * gdn_spec_tree_attn (the window's attention; a window is a tree of drafted
 * tokens).  Per step, over all layers: gdn_spec_kv_commit (the accepted path
 * moves together behind the committed tokens) and gdn_spec_kv_reserve (pages
 * for the next window).  gdn_spec_kv_fork and gdn_spec_kv_free start and end
 * a sequence that shares another one's pages.
 * ====================================================================== */

/*
 * The cache of all softmax-attention layers.  Slot s holds length[s] committed
 * tokens; token i of slot s is row i % P of page page_table[s][i / P], in every
 * layer.  The drafted tokens of a step follow the committed ones (position
 * length[s] + node) in the same pages.  A page may be held by several slots
 * (ref counts them); only full pages are ever shared, so no shared page is
 * written.  Page p is free exactly when ref[p] == 0 and bit p % 32 of
 * free_bits[p / 32] is set.  num_pages * P and max_pages * P are below 2^31, and
 * n_layers * HKV is at most 2^20 (GDN_SPEC_EUNSUPPORTED otherwise, as for the
 * limits that the calls name).
 */
typedef struct {
    int32_t n_layers;     /* softmax-attention layers                                   */
    int32_t num_pages;    /* pages in the pool                                          */
    int32_t HKV;          /* key/value heads                                            */
    int32_t P;            /* tokens per page: 16, 32, 64, 128 or 256                    */
    int32_t D;            /* head dim: a multiple of 8, at most 256                     */
    int32_t io_dtype;     /* dtype of k, v and of the calls' q, k, v, out               */
    int32_t num_slots;    /* slots in the pool                                          */
    int32_t max_pages;    /* columns of page_table: pages a slot can hold               */
    void *k, *v;          /* io_dtype [n_layers, num_pages, HKV, P, D]                  */
    int32_t *page_table;  /* [num_slots, max_pages], -1 where there is no page          */
    int32_t *n_pages;     /* [num_slots] pages held                                     */
    int32_t *length;      /* [num_slots] committed tokens                               */
    int32_t *ref;         /* [num_pages] slots that hold the page                       */
    uint32_t *free_bits;  /* [ceil(num_pages / 32)]                                     */
    uint32_t *status;     /* [1], device status bits (GDN_SPEC_ST_*); may be the word of
                             a gdn_spec_cursors                                         */
} gdn_spec_kv_cache;

/* gdn_spec_kv_init -- every slot empty, every page free.  k and v are not touched. */
int gdn_spec_kv_init(const gdn_spec_kv_cache *cache, void *stream);

/*
 * gdn_spec_kv_reserve -- pages for up to T more tokens: row b's slot gets the
 * pages it lacks to hold length + n tokens, n = n_tokens[b] (NULL: T).  The free
 * pages of lowest number are handed out in row order, so the tables depend only
 * on the calls made.  Row b is served when it lacks none or when the pages that
 * rows 0..b lack together are free (rows that are refused for another reason
 * lack none); otherwise it keeps what it has and NO_PAGES is set.  B <= 8192, and
 * B * max_pages is below 2^31.
 *   n_tokens  int32 [B], device, 0 <= n_tokens <= T, or NULL
 *   done      int32 [B], device (written): 1 where the row is served, else 0
 * Device status: SLOT_OOR, ACCEPT_RANGE (n_tokens), CURSOR_CORRUPT, NO_PAGES.
 */
int gdn_spec_kv_reserve(const gdn_spec_kv_cache *cache, const int32_t *slot_idx, int32_t B, int32_t T,
                        const int32_t *n_tokens, int32_t *done, void *stream);

/*
 * gdn_spec_kv_fork -- slot dst_idx[b] becomes a copy of slot src_idx[b]: the
 * full pages of its committed tokens are shared (ref + 1), the committed rows of
 * a last, partly filled page are copied to a page of its own in every layer
 * (pages that the source holds past them are not taken over).  A
 * destination must be empty (SLOT_BUSY otherwise), and no destination may be
 * named twice or be a source; a source may be named often.  Rows are served as
 * by gdn_spec_kv_reserve.  A negative index on either side is a padding row.
 * B <= 8192.
 *   done      int32 [B], device (written)
 * Device status: SLOT_OOR, CURSOR_CORRUPT, SLOT_BUSY, NO_PAGES, PAGE_OOR (a page of the
 * source's committed tokens is not one of the pool); such a row gives done = 0, and its
 * destination stays empty.
 */
int gdn_spec_kv_fork(const gdn_spec_kv_cache *cache, const int32_t *src_idx, const int32_t *dst_idx,
                     int32_t B, int32_t *done, void *stream);

/*
 * gdn_spec_kv_commit -- after sampling: the accepted drafts of every row move
 * together, row i of the window's committed tokens taken from drafted node
 * path[b][i] (i < accept_len[b]), in every layer, in place; then
 * length += accept_len.  Pages are kept for the next window.  With a path,
 * T <= 1024.
 *   path        int32 [B, T], device: strictly ascending nodes in [0, T) (a
 *               parent is numbered before its children), or NULL: nodes 0, 1, ...
 *   accept_len  int32 [B], device, 0 <= accept_len <= T
 * Device status: ACCEPT_RANGE (accept_len, or a path that does not ascend in
 * [0, T)), SLOT_OOR, CURSOR_CORRUPT, NO_PAGES, PAGE_OOR; such a row is left as
 * it is.
 */
int gdn_spec_kv_commit(const gdn_spec_kv_cache *cache, const int32_t *slot_idx, int32_t B, int32_t T,
                       const int32_t *path, const int32_t *accept_len, void *stream);

/* gdn_spec_kv_free -- each row's slot becomes empty; a page that no slot holds any more is free.
 * Device status: SLOT_OOR, CURSOR_CORRUPT (counts out of range: the row is left as it is; a page that
 * nobody holds: it stays as it is), PAGE_OOR (an entry that is no page is dropped). */
int gdn_spec_kv_free(const gdn_spec_kv_cache *cache, const int32_t *slot_idx, int32_t B, void *stream);

/* gdn_spec_kv_read_status -- as gdn_spec_read_status, for a cache's status word. */
int gdn_spec_kv_read_status(const gdn_spec_kv_cache *cache, uint32_t *host_out, int32_t clear,
                            void *stream);

/* pairs of a rotated vector: (x[i], x[i + rot/2]) or (x[2i], x[2i + 1]) */
#define GDN_SPEC_ROPE_HALF        0
#define GDN_SPEC_ROPE_INTERLEAVED 1

/* how the frequencies f_i = base^(-2i/rot) are scaled for contexts longer than trained on */
#define GDN_SPEC_ROPE_NONE   0
#define GDN_SPEC_ROPE_LINEAR 1  /* f_i / factor                                              */
#define GDN_SPEC_ROPE_NTK    2  /* base * factor^(rot / (rot - 2)) in place of base          */
#define GDN_SPEC_ROPE_YARN   3  /* f_i / factor and f_i mixed by a ramp over i between the pairs
                                   that turn `low` (floor) and `high` (ceil) times in `original`
                                   positions (low is the larger number: the faster pair); cos and
                                   sin times 0.1 ln(factor) + 1                              */
#define GDN_SPEC_ROPE_BANDS  4  /* f_i / factor and f_i mixed by (turns - low) / (high - low)
                                   clamped to [0, 1], turns = original f_i / (2 pi)          */

typedef struct {
    int32_t kind;      /* GDN_SPEC_ROPE_NONE ...                  */
    int32_t reserved;  /* 0                                       */
    double factor;     /* >= 1                                    */
    double original;   /* positions trained on (YARN, BANDS)      */
    double low, high;  /* YARN: fast, slow (32, 1); BANDS: 1, 4   */
} gdn_spec_rope_scaling;

/* A rotary plan, filled once by gdn_spec_rope_init or gdn_spec_rope_init_freqs (host only) and then
 * passed to the calls, which copy it into their launch. */
typedef struct {
    int32_t D;           /* head dim: a multiple of 8, at most 256                  */
    int32_t rot;         /* leading dims that are rotated: even, 2 .. D             */
    int32_t layout;      /* GDN_SPEC_ROPE_HALF or GDN_SPEC_ROPE_INTERLEAVED         */
    float   mscale;      /* factor on cos and sin                                   */
    uint64_t freq[128];  /* turns per position of pair i, as a fraction of 2^64     */
} gdn_spec_rope_plan;

/* gdn_spec_rope_init -- frequencies from a base and a scaling (NULL: none). */
int gdn_spec_rope_init(gdn_spec_rope_plan *plan, int32_t D, int32_t rot, int32_t layout, double base,
                       const gdn_spec_rope_scaling *scaling);

/* gdn_spec_rope_init_freqs -- frequencies given in radians per position, rot / 2 of them (host). */
int gdn_spec_rope_init_freqs(gdn_spec_rope_plan *plan, int32_t D, int32_t rot, int32_t layout,
                             const double *freqs, double mscale);

/*
 * gdn_spec_rope -- out = R x: pair i of every head of token n turned by the
 * angle pos[n] f_i and multiplied by mscale, the other dims copied.  transpose
 * != 0 gives R^T x, the gradient of x from that of out.  The angle is taken
 * modulo a turn in 64-bit fixed point, so it does not lose precision at long
 * positions; the products are fp32 and rounded once.
 *   pos   int32 [N], device
 *   x     io_dtype [N, heads, D]: token n at x + n * x_stride elements, its heads dense
 *   out   io_dtype [N, heads, D]: token stride out_stride; may be x itself with the same stride
 * Strides are multiples of 8 elements, at least heads * D, which is at most 2^22.
 */
int gdn_spec_rope(const gdn_spec_rope_plan *plan, int32_t N, int32_t heads, int32_t io_dtype,
                  const int32_t *pos, const void *x, int64_t x_stride, void *out, int64_t out_stride,
                  int32_t transpose, void *stream);

/*
 * gdn_spec_rope_append -- a window's rotary positions and its append to one
 * layer of the cache: q_out = R q; R k and v are written behind the committed
 * tokens of row b's slot, token t at length + t, t < n_tokens[b] (NULL: T).
 * length is not changed (gdn_spec_kv_commit moves it; for a prompt, with
 * path = NULL and accept_len = n_tokens).  The pages must have been reserved.
 *   q      io_dtype [B, T, HQ, D], k, v io_dtype [B, T, HKV, D]: token (b, t) at
 *          (b * T + t) * {q,k,v}_stride elements, its heads dense, so the three can be
 *          slices of one projection's output.  Strides are multiples of 8 elements.
 *   pos    int32 [B, T], device; NULL: length + t (a chain)
 *   q_out  io_dtype [B, T, HQ, D], dense (written; zeros for padding rows and t >= n_tokens)
 * T >= 1, any length; B * T is below 2^31 and (HQ + 2 HKV) * D at most 2^22.
 * Device status: SLOT_OOR, ACCEPT_RANGE (n_tokens), CURSOR_CORRUPT, NO_PAGES: such a
 * row writes zeros to q_out only.  PAGE_OOR: the tokens whose place in the page table is
 * no page write zeros to q_out only; the row's other tokens are served (with the entry
 * mended, the same call serves the whole row).
 */
int gdn_spec_rope_append(const gdn_spec_rope_plan *plan, const gdn_spec_kv_cache *cache, int32_t layer,
                         const int32_t *slot_idx, int32_t B, int32_t T, const int32_t *n_tokens,
                         const int32_t *pos, int32_t HQ, const void *q, int64_t q_stride, const void *k,
                         int64_t k_stride, const void *v, int64_t v_stride, void *q_out, void *stream);

/*
 * gdn_spec_tree_attn -- softmax attention of a window of drafted tokens over
 * one layer of the cache.  Node t of row b attends to the length committed
 * tokens of its slot and, of the window's tokens (cache positions length + n,
 * n < tree_len[b]), to those whose bit n is set in tree_mask[b][t]:
 *   out = sum_j p_j v_j,  p = softmax_j(scale <q, k_j>)
 * A node that attends to nothing, a node t >= tree_len[b] and a padding row give
 * zeros (lse: -inf).  What is masked has no effect, whatever its bits.
 *   q          io_dtype [B, T, HQ, D]; HKV divides HQ, head h reads kv head h / (HQ / HKV)
 *   tree_mask  uint64 [B, T], device; NULL: a chain (node t attends to nodes 0..t)
 *   tree_len   int32 [B], device, 0 <= tree_len <= T; NULL: T
 *   scale      > 0, and scale * log2(e) a finite fp32 number
 *   out        io_dtype [B, T, HQ, D] (written)
 *   lse        fp32 [B, T, HQ] (written), natural log of the softmax denominator; or NULL
 *   workspace  device memory of workspace_bytes >= gdn_spec_tree_attn_workspace, 16-byte
 *              aligned; its contents need not be kept or cleared, and calls that may run at
 *              the same time need one each
 * Two kernels (gdn_spec_tree_attn_path): "tc" -- bf16, at most 128 query heads a kv
 * head, n_layers * num_pages * HKV * P below 2^31: TMA and tcgen05, the probabilities
 * rounded to bf16 for the second product; "generic" -- otherwise: fp32 throughout on
 * the CUDA cores.  1 <= T <= 64; HQ / HKV is at most 4096, B * T below 2^31, and B * HKV
 * times (8 + the tiles of 32 tokens that a slot can hold) at most 2e9.
 * Device status: SLOT_OOR, ACCEPT_RANGE (tree_len), CURSOR_CORRUPT, NO_PAGES (the row
 * gives zeros), PAGE_OOR, TIMEOUT.
 */
int gdn_spec_tree_attn(const gdn_spec_kv_cache *cache, int32_t layer, const int32_t *slot_idx, int32_t B,
                       int32_t T, int32_t HQ, const void *q, const uint64_t *tree_mask,
                       const int32_t *tree_len, float scale, void *out, float *lse, void *workspace,
                       int64_t workspace_bytes, void *stream);

/* Bytes of workspace for such a call on the current device, or a negative GDN_SPEC_E* code. */
int64_t gdn_spec_tree_attn_workspace(const gdn_spec_kv_cache *cache, int32_t B, int32_t T, int32_t HQ);

/* Name of the kernel gdn_spec_tree_attn would launch ("tc", "generic"), or NULL if the descriptor is
 * invalid.  Host only. */
const char *gdn_spec_tree_attn_path(const gdn_spec_kv_cache *cache, int32_t T, int32_t HQ);

/* ----------------------------------------------------------------------
 * Prompts of any length, packed: row b of a call owns tokens starts[b] ..
 * starts[b + 1] of tensors that hold N tokens, one row behind another.  Per layer:
 * gdn_spec_norm_rope_append, then gdn_spec_prompt_attn; before them
 * gdn_spec_kv_reserve and after all layers gdn_spec_kv_commit with path = NULL,
 * both with the rows' counts.  Rows of one token (decode) go beside prompts in the
 * same call.
 *   starts  int32 [B + 1], device: ascending, 0 <= starts[b] <= starts[b + 1] <= N.
 *           A row whose two entries are not so owns nothing (ACCEPT_RANGE), nor does a
 *           row whose first token a row before it, whose entries are so, reaches past;
 *           the other rows are served.  What belongs to tokens that no row owns is left
 *           as it was.
 * Rows with slot_idx < 0, and rows refused with a status bit, get zeros.
 * ---------------------------------------------------------------------- */

/* The norm of a head x of D dims: x / sqrt(mean(x^2) + eps) * (weight + offset). */
typedef struct {
    const float *weight;  /* fp32 [D], device                                          */
    float eps;            /* >= 2^-126, finite                                         */
    float offset;         /* 0; 1 where a model keeps weights around zero              */
} gdn_spec_head_norm;

/*
 * gdn_spec_norm_rope -- out = R norm(x): every head of token n normed, then turned
 * to position pos[n] as by gdn_spec_rope.  fp32 throughout, rounded once; the sum
 * of squares has to be finite in fp32.
 *   arguments and limits as gdn_spec_rope; out may be x itself with the same stride
 */
int gdn_spec_norm_rope(const gdn_spec_rope_plan *plan, const gdn_spec_head_norm *norm, int32_t N,
                       int32_t heads, int32_t io_dtype, const int32_t *pos, const void *x,
                       int64_t x_stride, void *out, int64_t out_stride, void *stream);

/*
 * gdn_spec_norm_rope_grad -- the gradients of gdn_spec_norm_rope's x and weight from
 * that of its result: with g = R^T dy, r = 1 / sqrt(mean(x^2) + eps), w = weight + offset,
 *   dx = r (w g - r^2 x mean(w g x)),   dw = sum over tokens and heads of r x g
 * The same call gives the same bits.
 *   x, dy, dx  io_dtype [N, heads, D], strides as gdn_spec_rope's; dx (written) may be x or
 *              dy itself with the same stride
 *   dw         fp32 [D], 16-byte aligned (written; zeros where N = 0)
 *   workspace  device memory of workspace_bytes >= gdn_spec_norm_rope_grad_workspace, 16-byte
 *              aligned, as gdn_spec_tree_attn's; may be NULL where that is 0
 */
int gdn_spec_norm_rope_grad(const gdn_spec_rope_plan *plan, const gdn_spec_head_norm *norm, int32_t N,
                            int32_t heads, int32_t io_dtype, const int32_t *pos, const void *x,
                            int64_t x_stride, const void *dy, int64_t dy_stride, void *dx,
                            int64_t dx_stride, float *dw, void *workspace, int64_t workspace_bytes,
                            void *stream);

/* Bytes of workspace for such a call on the current device, and for every one with at most as many tokens, or a
 * negative GDN_SPEC_E* code. */
int64_t gdn_spec_norm_rope_grad_workspace(int32_t N, int32_t heads, int32_t D);

/*
 * gdn_spec_norm_rope_append -- q_out = R norm(q) of packed prompts; R norm(k) and v are
 * written behind the committed tokens of their rows' slots, token t of row b at length + t.
 * length is not changed, and the pages must have been reserved, as for
 * gdn_spec_rope_append.
 *   q_norm, k_norm  NULL: no norm on that side
 *   starts          int32 [B + 1], above
 *   pos             int32 [N], device; NULL: length + t
 *   q               io_dtype [N, HQ, D], k, v io_dtype [N, HKV, D]: token n at n * {q,k,v}_stride
 *                   elements, its heads dense.  Strides are multiples of 8 elements.
 *   q_out           io_dtype [N, HQ, D], dense (written)
 * (HQ + 2 HKV) * D is at most 2^22.  q_out overlaps none of q, k, v.
 * Device status: SLOT_OOR, ACCEPT_RANGE (starts), CURSOR_CORRUPT, NO_PAGES: such a row
 * writes zeros to q_out only.  PAGE_OOR: as gdn_spec_rope_append.
 */
int gdn_spec_norm_rope_append(const gdn_spec_rope_plan *plan, const gdn_spec_head_norm *q_norm,
                              const gdn_spec_head_norm *k_norm, const gdn_spec_kv_cache *cache,
                              int32_t layer, const int32_t *slot_idx, const int32_t *starts, int32_t B,
                              int32_t N, const int32_t *pos, int32_t HQ, const void *q, int64_t q_stride,
                              const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                              void *q_out, void *stream);

/*
 * gdn_spec_prompt_attn -- causal softmax attention of packed prompts over one layer of the
 * cache.  Token t of row b attends to the length committed tokens of its slot and to the
 * row's tokens 0..t (cache positions length ..  length + t, written before):
 *   out = sum_j p_j v_j,  p = softmax_j(scale <q, k_j>)
 * What a token does not attend to has no effect on it, whatever its bits.
 * Where all of a token's scores are -inf its softmax has no value: NaN, with an lse of -inf.
 *   q          io_dtype [N, HQ, D], dense; HKV divides HQ, head h reads kv head h / (HQ / HKV);
 *              out does not overlap it
 *   starts     int32 [B + 1], above
 *   scale      > 0, and scale * log2(e) a finite fp32 number
 *   out        io_dtype [N, HQ, D], dense (written)
 *   lse        fp32 [N, HQ] (written), natural log of the softmax denominator; -inf for rows
 *              that get zeros; or NULL
 *   workspace  as gdn_spec_tree_attn's, workspace_bytes >= gdn_spec_prompt_attn_workspace
 * Two kernels (gdn_spec_prompt_attn_path): "tc" -- bf16: TMA and tcgen05, the probabilities
 * rounded to bf16 for the second product; n_layers * num_pages * HKV * P is below 2^31 --
 * and "generic" -- fp32 throughout on the CUDA cores.  HQ / HKV is at most 4096,
 * max_pages * P at most 2^31 - 1025, and (N + B) * HKV * (1 + HQ / HKV / 64) *
 * (max_pages * P + 1024) at most 4e18.
 * Device status: SLOT_OOR, ACCEPT_RANGE (starts), CURSOR_CORRUPT, NO_PAGES (the row gets
 * zeros), PAGE_OOR (the row's outputs are not valid), TIMEOUT.
 */
int gdn_spec_prompt_attn(const gdn_spec_kv_cache *cache, int32_t layer, const int32_t *slot_idx,
                         const int32_t *starts, int32_t B, int32_t N, int32_t HQ, const void *q,
                         float scale, void *out, float *lse, void *workspace, int64_t workspace_bytes,
                         void *stream);

/* Bytes of workspace for such a call on the current device, and for every one with at most as many rows and
 * tokens, or a negative GDN_SPEC_E* code.  At most: bf16 some 21 MB for heads of up to 64 dims and 41 MB above, where
 * a layer of the pool (its num_pages) is below 96 MB or the tokens are few, else up to four times as much as the pool is larger;
 * fp32 some 20 MB. */
int64_t gdn_spec_prompt_attn_workspace(const gdn_spec_kv_cache *cache, int32_t B, int32_t N, int32_t HQ);

/* Name of the kernel gdn_spec_prompt_attn would launch ("tc", "generic"), or NULL if the
 * descriptor or the head count is invalid.  Host only. */
const char *gdn_spec_prompt_attn_path(const gdn_spec_kv_cache *cache, int32_t HQ);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SPEC_H */
