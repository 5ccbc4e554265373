/*
 * fl_attn.h -- C ABI of the GB300 fused attention-variant forward.
 *
 * One call computes, for every (batch, query head, query row i),
 *
 *     O_i   = sum_j softmax_j( z_ij ) v_j
 *     LSE_i = ln sum_j exp( z_ij )
 *     z_ij  = score_mod( scale * q_i . k_j ) + bias_ij    (or -inf where masked)
 *
 * in a single pass over the keys with an online softmax: a running maximum and
 * a running sum per query row, the sum (and the output accumulator) rescaled
 * whenever the maximum moves, so that no S x S score or probability tensor is
 * ever written to device memory.  This is the fused kernel shape the
 * Flashlight pages describe (gist.science summary, "Methodology" items 2-4:
 * dimension demotion fuses max() into QK^T, the homomorphism
 * e^(x-y) = e^x / e^y turns the two-pass stable softmax into a one-pass
 * online one, and tiling-aware dimension elimination fuses softmax(QK^T)V;
 * talk notes, "Compiler design" 1-4).  The variants are the ones the talk
 * notes evaluate ("Evaluation: FlexAttention-supported variants" and
 * "Evaluation: complex variants"): vanilla, ALiBi, softcap, causal, sliding
 * window, PrefixLM, document mask, MHA and GQA, differential attention, and
 * the AlphaFold Evoformer row- and column-wise gated self-attention with pair
 * bias.  The pages give no formula for these; the ones used are stated at
 * each enum below.
 *
 * Conventions shared by every entry point
 *  - Every tensor is a caller-owned DEVICE buffer of the current CUDA device
 *    (e.g. a torch tensor).  The library never allocates, frees or retains
 *    caller memory.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream).  A returned FL_OK means the work was enqueued.
 *  - Functions never throw.  Argument validation happens before any CUDA
 *    call; a failed validation launches nothing and leaves outputs
 *    untouched.  fl_attn_last_error() then describes the failure.
 *  - The library is thread-safe for concurrent calls on different streams.
 */
#ifndef FL_ATTN_H
#define FL_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FL_ATTN_VERSION 1

typedef struct CUstream_st *fl_stream_t; /* identical to cudaStream_t */

typedef enum {
    FL_OK = 0,
    FL_ERR_INVALID_ARG = 1,    /* null pointer, bad rank/shape/dtype, bad parameter */
    FL_ERR_UNSUPPORTED = 2,    /* valid request outside the compiled kernel set */
    FL_ERR_ALIGNMENT = 3,      /* base pointer or stride not 16-byte aligned */
    FL_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed */
    FL_ERR_DEVICE_TIMEOUT = 5, /* reported through error_word: a device wait ran out */
    FL_ERR_NO_DEVICE = 6       /* no CUDA device, or not an sm_103 (GB300) device */
} fl_status;

typedef enum { FL_BF16 = 0, FL_F32 = 1 } fl_dtype;

/* A strided view.  sizes/strides are in ELEMENTS, outermost first; the
 * innermost stride must be 1.  All other strides of bf16 tensors must be
 * multiples of 8 elements (16 bytes) and every ptr 16-byte aligned. */
typedef struct {
    void *ptr;
    int32_t dtype; /* fl_dtype */
    int32_t ndim;
    int64_t sizes[5];
    int64_t strides[5];
} fl_tensor;

typedef enum {
    FL_KIND_STANDARD = 0, /* MHA / GQA with score_mod and mask */
    FL_KIND_DIFF = 1,     /* differential attention, two softmax streams, one V */
    FL_KIND_EVO_ROW = 2,  /* Evoformer MSA row-wise gated attention + pair bias */
    FL_KIND_EVO_COL = 3   /* Evoformer MSA column-wise gated attention */
} fl_kind;

typedef enum {
    FL_MOD_NONE = 0,
    FL_MOD_ALIBI = 1,   /* z += -slope_h * |i - j|, slope_h = 2^(-8 (h+1) / Hq) by default */
    FL_MOD_SOFTCAP = 2, /* z = cap * tanh(z / cap) */
    FL_MOD_EXPR = 3     /* z = the expression desc->score_mod_expr (FL_KIND_STANDARD) */
} fl_score_mod;

/*
 * score_mod expressions (FL_MOD_EXPR).  The logit of (query row q_idx, key
 * kv_idx) of batch b and query head h is the value of a user expression over
 *     score   scale * q . k (the scaled dot product)
 *     b, h, q_idx, kv_idx
 * in this grammar (every value fp32; a comparison gives 1 or 0; '/' is the
 * fast division, within 2 ulp; exp and exp2 use the hardware 2^x, relative
 * error about 2^-22; tanh is 1 - 2 / (1 + e^(2x)) on it, absolute error
 * about 1e-7):
 *     expr    := sum [ relop sum ]        relop: < <= > >= == !=  (no chains)
 *     sum     := term { (+ | -) term }
 *     term    := unary { (* | /) unary }
 *     unary   := (- | +) unary | primary
 *     primary := number | score | b | h | q_idx | kv_idx | inf
 *              | tanh(e) | exp(e) | exp2(e) | log(e) | log2(e) | sqrt(e)
 *              | abs(e) | floor(e) | min(e, e) | max(e, e)
 *              | where(c, x, y)           (x where c != 0, else y)
 *              | ( expr )
 * e.g. "20 * tanh(score / 20)" (softcap), "score - 0.5 * abs(q_idx - kv_idx)"
 * (ALiBi with slope 0.5), "where(kv_idx <= q_idx, score, -inf)" (a causal
 * mask written as a score_mod).  -inf removes the pair; the mask in the desc
 * still applies on top.  This is the pages' generic-variant interface: the
 * expression is fused into the same single-pass kernel as the built-in
 * variants (talk notes, "Compiler design" and the comparison with
 * FlexAttention).  The first call with a new expression on a device compiles
 * the kernel for it at run time (NVRTC, about two seconds; the CUDA toolkit's
 * libnvrtc.so.13 and include directory -- $CUDA_HOME, else /usr/local/cuda --
 * must be present, or the call returns FL_ERR_UNSUPPORTED); later calls reuse
 * it.  A string outside the grammar returns FL_ERR_INVALID_ARG.
 */

typedef enum {
    FL_MASK_NONE = 0,
    FL_MASK_CAUSAL = 1, /* key j allowed for query i iff j <= i */
    FL_MASK_WINDOW = 2, /* j <= i and i - j < window */
    FL_MASK_PREFIX = 3, /* j <= i or j < prefix (bidirectional over the first prefix keys) */
    FL_MASK_DOC = 4     /* same document and j <= i */
} fl_mask;

/* Test-only fault injection: the library itself never sets these. */
typedef enum {
    FL_INJECT_NONE = 0,
    FL_INJECT_DROP_KV_LOAD = 1 /* one K/V tile load of CTA 0 is never issued, so the
                                  consumer's bounded wait runs out */
} fl_inject;

/* Bits the kernel ORs into error_word. */
#define FL_DEVERR_TIMEOUT 0x1u        /* a bounded wait ran out; the CTA quit cleanly */
#define FL_DEVERR_PAGES 0x2u          /* fl_kv_plan: a new token got no page (slot -1) */
#define FL_DEVERR_LENGTHS 0x4u        /* lengths on the device exceed what the host stated (fl_kv_plan's
                                         tokens, fl_attn_chunk's offsets and, where asked for,
                                         kv_lens) */
#define FL_DEVERR_WHERE_SHIFT 8       /* bits 8..15: which wait (diagnostic) */

typedef struct {
    int32_t kind;            /* fl_kind */
    int32_t score_mod;       /* fl_score_mod (FL_KIND_STANDARD only) */
    float softcap;           /* cap > 0 for FL_MOD_SOFTCAP */
    int32_t mask;            /* fl_mask (STANDARD and DIFF; DIFF takes NONE or CAUSAL) */
    int32_t window;          /* FL_MASK_WINDOW, >= 1 */
    int32_t prefix;          /* FL_MASK_PREFIX, >= 0 */
    const int32_t *doc_offsets; /* FL_MASK_DOC: device int32 [B][doc_stride]; row b holds the
                                   ascending document starts of batch b (first 0), padded
                                   with S */
    int32_t doc_stride;      /* entries per row of doc_offsets (max documents + 1) */
    int32_t gqa_group;       /* Hq / Hk; 0 derives it from the shapes, else must match */
    float diff_lambda;       /* FL_KIND_DIFF: O = O_1 - lambda O_2 */
    float scale;             /* 0 means 1 / sqrt(D) */
    const float *alibi_slopes; /* device float [Hq], or NULL for 2^(-8 (h+1) / Hq) */
    int32_t *debug_tile_counts; /* NULL, or device int32 [batch][heads][ceil(S/128)]: the
                                   number of key tiles each 128-row query block visited
                                   (key-tile width from fl_attn_tile_shape: 128 for the
                                   standard kind at D = 32, 112 at D = 64, 64 at D = 128; 112 for
                                   the differential kind at Dv = 64, 80 at Dv = 128; 128
                                   for the Evoformer kinds) */
    uint32_t *error_word;    /* NULL, or a device word the kernel ORs FL_DEVERR_* into */
    int32_t debug_inject;    /* fl_inject; 0 in normal use */
    uint32_t wait_timeout_us; /* bound of every device-side wait; 0 means 2,000,000 */
    const char *score_mod_expr; /* FL_MOD_EXPR: the expression (host string), else unused */
} fl_attn_variant_desc;

/*
 * fl_attn_fwd -- fused attention forward.
 *
 * Layouts (sizes in this logical order; any strides subject to the fl_tensor
 * rules), all bf16 except lse (fp32):
 *   FL_KIND_STANDARD  q [B,S,Hq,D]  k [B,S,Hk,D]  v [B,S,Hk,Dv]  out [B,S,Hq,Dv]
 *                     lse [B,Hq,S] or NULL.        bias, gate: NULL.
 *   FL_KIND_DIFF      q [2,B,S,H,D] k [2,B,S,Hk,D] v [B,S,Hk,Dv] out [B,S,H,Dv]
 *                     lse [2,B,H,S] or NULL (one LSE per softmax stream).
 *                     out = softmax(scale Q1 K1^T) V - lambda softmax(scale Q2 K2^T) V.
 *   FL_KIND_EVO_ROW   q,k,v,gate,out [N_seq,N_res,H,c]; bias [H,N_res,N_res];
 *                     attention over residues for each MSA row:
 *                     out = sigmoid(gate) * softmax(scale q k^T + bias) v;
 *                     lse [N_seq,H,N_res] or NULL.
 *   FL_KIND_EVO_COL   q,k,v,gate,out [N_seq,N_res,H,c]; bias NULL;
 *                     attention over MSA rows for each residue (axis 0);
 *                     lse [N_res,H,N_seq] or NULL.
 * lse is natural-log; its innermost stride must be 1.
 *
 * Supported shapes: STANDARD D = Dv in {32, 64, 128}; DIFF D = 64, Dv = 64
 * or 128 with mask none or causal; EVO c = 32 or 64, any N_res (the row pass
 * keeps a query block's bias rows in shared memory for c = 32 and N_res <= 384,
 * and streams them per key tile otherwise).  Other shapes return
 * FL_ERR_UNSUPPORTED.  The bias may be passed with any strides obeying the
 * fl_tensor rules (for example a [N_res,N_res,H] tensor viewed as
 * [H,N_res,N_res]).  Evoformer sequence lengths must keep every stride a
 * multiple of 16 bytes (c = 32 bf16 rows always do; the bias row stride must
 * be a multiple of 8 elements: pad N_res or the bias rows otherwise).
 * STANDARD launches of 2^31 or more work items (pairs of 128-row query
 * blocks per batch and head) also return FL_ERR_UNSUPPORTED.
 *
 * Returns FL_OK when enqueued.  Device-side failures (a wait that ran out)
 * are reported asynchronously through desc->error_word.
 */
fl_status fl_attn_fwd(const fl_tensor *q, const fl_tensor *k, const fl_tensor *v,
                      const fl_tensor *out, const fl_tensor *lse,
                      const fl_attn_variant_desc *desc, const fl_tensor *bias,
                      const fl_tensor *gate, fl_stream_t stream);

/*
 * fl_attn_evoformer -- the Evoformer kinds over a batch of MSA stacks, with an
 * optional MSA mask (AlphaFold2 context: talk notes, "End-to-end: AlphaFold2").
 *
 * desc->kind is FL_KIND_EVO_ROW or FL_KIND_EVO_COL; everything fl_attn_fwd
 * says of those kinds holds per stack.  Shapes (bf16 unless noted):
 *   q, k, v, gate, out  [B, N_seq, N_res, H, c]   (or [N_seq, N_res, H, c]: B = 1)
 *   bias (row pass)     [B, H, N_res, N_res], or [H, N_res, N_res] shared by all stacks
 *   msa_mask            NULL, or [B, N_seq, N_res] / [N_seq, N_res] shared, bf16 or
 *                       fp32: where msa_mask[s, r] is 0 the entry is removed as a key --
 *                       residue r for MSA row s in the row pass, MSA row s for residue
 *                       r in the column pass.  A query row left with no key gives
 *                       O = 0 and LSE = -inf.
 *   lse                 NULL, or [B, N_seq, H, N_res] (row) / [B, N_res, H, N_seq] (col)
 * The stack axis may have any stride that is a positive multiple of 16 bytes.
 * Each stack is one kernel launch on `stream`.  Every argument is validated
 * before the first launch.
 */
fl_status fl_attn_evoformer(const fl_tensor *q, const fl_tensor *k, const fl_tensor *v,
                            const fl_tensor *out, const fl_tensor *lse,
                            const fl_attn_variant_desc *desc, const fl_tensor *bias,
                            const fl_tensor *gate, const fl_tensor *msa_mask, fl_stream_t stream);

/*
 * fl_attn_bwd -- backward of the standard kind: dQ, dK, dV of
 *     O = softmax(scale Q K^T + mask) V
 * given the forward's out and (natural-log) lse and the output gradient
 * dout.  The pages name the backward pass as the fused kernels' next step
 * (gist.science summary, "Limitations and future work").  P is recomputed
 * from Q, K and the LSE; dS = P (dP - D) with D_i = sum_d dout_id out_id.
 *   q, out, dout, dq [B, S, Hq, 64]; k, v, dk, dv [B, S, Hk, 64]; lse [B, Hq, S] fp32
 *   desc: kind FL_KIND_STANDARD, any score_mod (FL_MOD_EXPR included: the
 *   backward kernels are compiled at run time with the expression and its
 *   derivative with respect to `score`, derived through the grammar), any
 *   mask of the standard kind, scale (0: 1/8).  GQA heads are summed into
 *   dk, dv.
 * `workspace`: device memory of at least fl_attn_bwd_workspace_size bytes,
 * 256-byte aligned, owned by the caller, no initialisation needed.  Three
 * kernel launches on `stream`; every output element is written once (no
 * atomics: the result does not depend on scheduling).
 */
fl_status fl_attn_bwd_workspace_size(const fl_tensor *q, const fl_tensor *k,
                                     const fl_attn_variant_desc *desc, size_t *bytes);
fl_status fl_attn_bwd(const fl_tensor *q, const fl_tensor *k, const fl_tensor *v,
                      const fl_tensor *out, const fl_tensor *lse, const fl_tensor *dout,
                      const fl_tensor *dq, const fl_tensor *dk, const fl_tensor *dv,
                      const fl_attn_variant_desc *desc, void *workspace, size_t workspace_bytes,
                      fl_stream_t stream);

/*
 * fl_attn_diff_bwd -- backward of the differential kind: dQ1, dQ2, dK1, dK2
 * and dV of
 *     O = softmax(scale Q1 K1^T + mask) V - lambda softmax(scale Q2 K2^T + mask) V
 * given the forward's per-stream (natural-log) lse and the output gradient
 * dout (the pages name differential attention among the complex variants,
 * gist.science summary, "Results", and the backward as the fused kernels'
 * next step, "Limitations and future work").
 *   q, dq [2, B, S, H, 64]; k, dk [2, B, S, Hk, 64]; v, dv [B, S, Hk, Dv],
 *   Dv 64 or 128; dout [B, S, H, Dv]; lse [2, B, H, S] fp32 (fl_attn_fwd's).
 *   desc: kind FL_KIND_DIFF, mask none or causal, no score_mod, scale (0:
 *   1/8), diff_lambda; GQA heads are summed into dk, dv.
 * Stream t's gradients are those of one softmax attention whose output
 * gradient is c_t dout (c = 1, -lambda); the library recomputes each stream's
 * output from q, k and v and runs the standard backward on it, per 64-column
 * half of V when Dv = 128, then adds the partial gradients with their
 * coefficients in fp32 and rounds once to bf16.
 * `workspace`: device memory of at least fl_attn_diff_bwd_workspace_size
 * bytes, 256-byte aligned, owned by the caller, no initialisation needed.
 * All launches go to `stream`, validation happens before the first one, and
 * every output element is written exactly once (no atomics).
 */
fl_status fl_attn_diff_bwd_workspace_size(const fl_tensor *q, const fl_tensor *k, const fl_tensor *v,
                                          const fl_attn_variant_desc *desc, size_t *bytes);
fl_status fl_attn_diff_bwd(const fl_tensor *q, const fl_tensor *k, const fl_tensor *v,
                           const fl_tensor *lse, const fl_tensor *dout, const fl_tensor *dq,
                           const fl_tensor *dk, const fl_tensor *dv, const fl_attn_variant_desc *desc,
                           void *workspace, size_t workspace_bytes, fl_stream_t stream);

/* Query-block and key-tile sizes the kernel for `desc` uses (for the
 * visited-tile accounting).  `head_dim` is D for the standard and Evoformer
 * kinds and the value head dimension Dv for FL_KIND_DIFF (whose D is 64).
 * Never touches the device. */
fl_status fl_attn_tile_shape(const fl_attn_variant_desc *desc, int32_t head_dim,
                             int32_t *block_m, int32_t *block_n);

/* Checks a score_mod expression against the FL_MOD_EXPR grammar (FL_OK or
 * FL_ERR_INVALID_ARG, with the position in fl_attn_last_error()).  With
 * `compile` 1 it also runs the runtime compilation of the forward kernel for
 * it, with 2 also that of the backward kernels for it and its derivative (no
 * device needed; FL_ERR_UNSUPPORTED without NVRTC). */
fl_status fl_attn_score_expr_check(const char *expr, int32_t compile);

/* Static text for a status code. */
const char *fl_attn_status_string(fl_status status);

/* Detail of the last failure on the calling thread ("" if none). */
const char *fl_attn_last_error(void);

/* FL_ATTN_VERSION of the loaded library. */
int32_t fl_attn_version(void);

/* ------------------------------------------------------------------------
 * Serving with a KV cache (decode).
 *
 * A few new query tokens per sequence attend to that sequence's cached keys
 * and values: the LLaMA-3.2-1B serving workload of the talk notes ("End-to-end:
 * LLaMA-3.2-1B (vLLM / Mooncake)"), whose attention is made causal or
 * softcapped.  out = softmax(score_mod(scale q k^T) + mask) v over the keys
 * 0 .. kv_lens[b] - 1 of sequence b; with `causal`, new token s of a sequence
 * of L cached keys (the new tokens included) sits at position L - Sq + s and
 * sees the keys up to it.
 */
typedef struct {
    int32_t score_mod;          /* FL_MOD_NONE or FL_MOD_SOFTCAP */
    float softcap;              /* FL_MOD_SOFTCAP: the cap (> 0) */
    int32_t causal;             /* 1: decode-causal as above; 0: every cached key */
    float scale;                /* 0 means 1 / sqrt(D) */
    const int32_t *kv_lens;     /* device int32 [B]: cache length of each sequence */
    int32_t max_kv_len;         /* host bound on kv_lens[] (sizes the launch and the workspace);
                                   larger entries are clamped to it */
    const int32_t *block_table; /* NULL: contiguous cache; else device int32
                                   [B][block_table_stride]: page index of each page of a
                                   sequence */
    int32_t block_table_stride; /* entries per row of block_table */
    uint32_t *error_word;       /* NULL, or a device word the kernel ORs FL_DEVERR_* into */
    uint32_t wait_timeout_us;   /* bound of every device-side wait; 0 means 2,000,000 */
} fl_decode_desc;

/*
 * Layouts (bf16 except lse):
 *   q        [B, Sq, Hq, 64]
 *   k_cache, v_cache
 *            contiguous (block_table NULL): [B, S_max, Hk, 64], S_max >= max_kv_len;
 *            paged: [num_pages, page_size, Hk, 64] with page_size in
 *            {16, 32, 64, 128, 256}; key p of sequence b is row p % page_size of
 *            page block_table[b][p / page_size]
 *   out      [B, Sq, Hq, 64]
 *   lse      [B, Hq, Sq] fp32 (natural log) or NULL
 * Hq must be a multiple of Hk, and (Hq / Hk) * Sq <= 64.  The kernel splits
 * every sequence's keys into splits of 128, 256, 512 or 1024 keys (the
 * longest that leaves B * Hk * splits-of-max_kv_len >= 2048, else 128) and
 * merges the splits' partial results through `workspace`: device memory of
 * at least the size
 * fl_attn_decode_workspace_size reports, 256-byte aligned, owned by the
 * caller; its contents need no initialisation (the call clears what must
 * start at zero).  Calls sharing one workspace must not overlap on the GPU.
 */
fl_status fl_attn_decode_workspace_size(const fl_tensor *q, const fl_tensor *k_cache,
                                        const fl_decode_desc *desc, size_t *bytes);

fl_status fl_attn_decode(const fl_tensor *q, const fl_tensor *k_cache, const fl_tensor *v_cache,
                         const fl_tensor *out, const fl_tensor *lse, const fl_decode_desc *desc,
                         void *workspace, size_t workspace_bytes, fl_stream_t stream);

/*
 * fl_attn_decode_static -- fl_attn_decode without a workspace argument, for
 * callers that cannot allocate device memory: for example a serving loop that
 * must not take the device-wide synchronisation a cudaMalloc or cudaFree can
 * cause, or a plug-in that does not own the process's device allocator, and
 * that has no buffer of its own to pass.  (The pages have no counterpart: it
 * is an interface for such callers, not part of the method.)
 *
 * The call allocates nothing.  Its scratch is a static device array of
 * FL_DECODE_STATIC_SCRATCH_BYTES (64 MiB) inside this library, which every GPU
 * that loads the library holds until the process exits; shapes that need more
 * (see fl_attn_decode_workspace_size) return FL_ERR_UNSUPPORTED.  The first
 * call in each CUDA context -- a device's primary context, a context the
 * caller made current, or the new primary context after cudaDeviceReset --
 * looks up the array's device address in that context (which may load the
 * library's device code there): make that first call before any stream
 * capture.  Every call shares the one array and finds the previous
 * call's contents; the call clears what must start at zero, but calls that
 * overlap on the GPU race: issue them on one stream, or order them.
 * Arguments, layouts and results are those of fl_attn_decode.
 */
#define FL_DECODE_STATIC_SCRATCH_BYTES (64u << 20)
fl_status fl_attn_decode_static(const fl_tensor *q, const fl_tensor *k_cache,
                                const fl_tensor *v_cache, const fl_tensor *out,
                                const fl_tensor *lse, const fl_decode_desc *desc,
                                fl_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions.
 *
 * Pair i of a head's first rot_dim elements turns by the angle pos * f_i and
 * is multiplied by a magnitude m:
 *     y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t),  t = pos f_i
 * with (a, b) = (i, i + rot_dim / 2) (FL_ROPE_HALF) or (2 i, 2 i + 1)
 * (FL_ROPE_INTERLEAVED); elements from rot_dim on are copied.  The backward
 * turns the other way, with the same m.  The frequencies are
 * f_i = base^(-2 i / rot_dim), stretched for contexts longer than the trained
 * `context` by one of
 *     LINEAR  f_i / factor
 *     BASE    base replaced by base * factor^(rot_dim / (rot_dim - 2))
 *     BANDS   by the turns n_i = context f_i / 2 pi a pair makes in the
 *             trained context: f_i where n_i >= high, f_i / factor where
 *             n_i <= low, w f_i + (1 - w) f_i / factor between, with
 *             w = (n_i - low) / (high - low)
 *     RAMP    by the pair's index: the same blend, w falling linearly from 1
 *             at index floor(d(high)) to 0 at ceil(d(low)) (clamped to
 *             [0, rot_dim - 1]), d(n) = rot_dim ln(context / 2 pi n) / (2 ln base);
 *             m is 0.1 ln(factor) + 1 for factors above 1 and 1 up to it, unless given
 * f_i / 2 pi is kept as a 64-bit fraction of a turn, so that pos times it wraps
 * by itself: the reduction modulo a turn is exact at any int32 position.  What
 * grows with the position is the frequency's own error, a few 2^-53 of it (about
 * 10^-6 rad at 2^31).
 */
typedef enum { FL_ROPE_HALF = 0, FL_ROPE_INTERLEAVED = 1 } fl_rope_layout;
typedef enum {
    FL_ROPE_SCALE_NONE = 0,
    FL_ROPE_SCALE_LINEAR = 1,
    FL_ROPE_SCALE_BASE = 2,
    FL_ROPE_SCALE_BANDS = 3,
    FL_ROPE_SCALE_RAMP = 4
} fl_rope_scaling;

typedef struct {
    int32_t rot_dim;   /* even, 2 .. 256 */
    int32_t layout;    /* fl_rope_layout */
    int32_t scaling;   /* fl_rope_scaling */
    double base;       /* > 1 */
    double factor;     /* > 0; every scaling but NONE */
    double context;    /* trained context length (> 0); BANDS and RAMP */
    double low, high;  /* turns, 0 < low < high; 0, 0 means 1, 4 (BANDS) or 1, 32 (RAMP) */
    double magnitude;  /* 0 means 1, or RAMP's default */
} fl_rope_config;

#define FL_ROPE_MAX_PAIRS 128
/* Host memory, filled by fl_rope_make_table; the caller keeps it (one per
 * model) and every call copies it. */
typedef struct {
    int32_t rot_dim, layout;
    float magnitude;
    uint32_t valid;                    /* set by fl_rope_make_table */
    uint64_t turns[FL_ROPE_MAX_PAIRS]; /* f_i / 2 pi modulo 1, in units of 2^-64 */
} fl_rope_table;

/* Never touches the device. */
fl_status fl_rope_make_table(const fl_rope_config *config, fl_rope_table *table);

typedef struct {
    const fl_rope_table *table;
    const int32_t *positions; /* NULL, or device int32: [B, S] with positions_stride elements
                                 between the rows (0: one row for all), [T] for 3-D tensors */
    int64_t positions_stride;
    int32_t offset;           /* position = offset + (positions ? positions[b][s] : s) */
    int32_t backward;         /* 1: the transposed map, for gradients of the outputs */
} fl_rope_desc;

/*
 * fl_rope -- rotary positions of q and, unless NULL, k in one launch.
 *   q, q_out [B, S, Hq, D], k, k_out [B, S, Hk, D], or [T, Hq, D] and
 *   [T, Hk, D] (rows of any batch one after another); bf16 or fp32, all the
 *   same; rot_dim <= D.  Strides of bf16 tensors are multiples of 16 bytes,
 *   those of fp32 ones anything; the innermost is 1.  At least one token.  An
 *   output may be its input (same pointer and strides); other overlaps are
 *   undefined.  Arithmetic is fp32 on the fp32 sine and cosine, rounded once.
 */
fl_status fl_rope(const fl_tensor *q, const fl_tensor *k, const fl_tensor *q_out,
                  const fl_tensor *k_out, const fl_rope_desc *desc, fl_stream_t stream);

/* ------------------------------------------------------------------------
 * A serving step over a paged KV cache: fl_kv_plan once per step, then per
 * layer fl_kv_append and fl_attn_chunk (or fl_attn_decode).
 *
 * fl_kv_plan -- the step's book-keeping on the GPU, from request lengths.
 * Request b holds kv_lens[b] keys and brings q_lens[b] new tokens (entries
 * below 0 count as 0).  Its pages are block_table[b][0 .. ceil(kv_lens[b] /
 * page_size)); further pages are taken from free_pages[free_head[0] ...] in
 * the order of the requests and written to the block table.  All pointers are
 * device memory:
 */
typedef struct {
    int32_t batch;              /* B >= 1 requests */
    int32_t page_size;          /* 16, 32, 64, 128 or 256 keys */
    int32_t max_tokens;         /* entries of positions and slots (0: none wanted), at most 2^31 - 1024 */
    int32_t n_free;             /* entries of free_pages */
    int32_t block_table_stride; /* entries per row of block_table */
    const int32_t *q_lens;      /* [B] */
    const int32_t *kv_lens;     /* [B] */
    const int32_t *free_pages;  /* [n_free]; may be NULL when n_free is 0 */
    const int32_t *free_head;   /* [1]: pages of free_pages taken so far */
    int32_t *block_table;       /* [B][block_table_stride]: new pages are written, the rest kept */
    int32_t *kv_lens_out;       /* [B]: kv_lens + q_lens; must not overlap kv_lens */
    int32_t *cu_q;              /* [B + 1]: first token of each request, then their number */
    int32_t *positions;         /* [max_tokens]: position of each token in its sequence */
    int64_t *slots;             /* [max_tokens]: page * page_size + row of its key; NULL: none */
    int32_t *free_head_out;     /* [1]: free_head plus the pages asked for; must not be free_head */
    uint32_t *error_word;       /* NULL, or a device word FL_DEVERR_* is ORed into */
} fl_kv_plan_desc;
/*
 * Entries of positions and slots past the last token are -1 (so a captured
 * step may be padded).  A token without a page (the free list ran out, or the
 * block table's row is full) gets slot -1, its table entry -1, and
 * FL_DEVERR_PAGES.  Tokens past max_tokens are not listed, with
 * FL_DEVERR_LENGTHS unless max_tokens is 0; they count in everything else, and
 * their pages are taken and written to the block table.
 * Requests' block-table entries are taken as they are.
 */
fl_status fl_kv_plan(const fl_kv_plan_desc *desc, fl_stream_t stream);

/*
 * fl_kv_append -- writes the new keys and values to their slots of a paged
 * cache, rotating q and k on the way.
 *   q, q_out  [T, Hq, D] or both NULL; k, v [T, Hk, D]; bf16, T >= 1
 *   k_cache, v_cache [num_pages, page_size, Hk, D]; any page_size
 *   slots     device int64 [T] (fl_kv_plan's): row slots[t] % page_size of page
 *             slots[t] / page_size; a token whose slot is outside
 *             [0, num_pages * page_size) is skipped: nothing is written for it
 *   rope      NULL (copies), or as in fl_rope, with positions [T] required
 *             and not backward
 * Slots must differ from one another: of two tokens with one slot either may
 * win, element by element.  q_out may be q.
 */
fl_status fl_kv_append(const fl_tensor *q, const fl_tensor *k, const fl_tensor *v,
                       const fl_tensor *q_out, const fl_tensor *k_cache, const fl_tensor *v_cache,
                       const int64_t *slots, const fl_rope_desc *rope, fl_stream_t stream);

/*
 * fl_attn_chunk -- attention of ragged chunks of new tokens over the cache
 * that holds them: prompts, parts of prompts and single tokens in one call.
 * Request b's queries are rows cu_q[b] .. cu_q[b + 1] - 1 of q and are its
 * last tokens: row cu_q[b] + s sits at position kv_lens[b] - n_b + s (n_b its
 * number of rows) and sees the keys j <= that position (causal) that are less
 * than `window` before it (window > 0), or every key j < kv_lens[b].
 */
typedef struct {
    int32_t score_mod;          /* FL_MOD_NONE or FL_MOD_SOFTCAP */
    float softcap;              /* FL_MOD_SOFTCAP: the cap, > 0 and at most 16384; capped scores are off
                                   by about 2^-22 cap */
    int32_t causal;             /* 1: as above; 0: every cached key */
    int32_t window;             /* 0: no window; else needs causal */
    float scale;                /* 0 means 1 / sqrt(D) */
    int32_t batch;              /* B requests */
    const int32_t *cu_q;        /* device int32 [B + 1], ascending, within 0 .. T (entries that are
                                   not are clamped, with FL_DEVERR_LENGTHS) */
    const int32_t *kv_lens;     /* device int32 [B]: cached keys, the new ones included */
    int32_t max_kv_len;         /* host bound on kv_lens[], below 2^31 - 255; a larger entry counts as
                                   this many keys, with the request's rows at the end of them */
    const int32_t *block_table; /* as in fl_decode_desc; NULL: contiguous cache */
    int32_t block_table_stride;
    uint32_t *error_word;       /* NULL, or a device word the kernel ORs FL_DEVERR_* into */
    uint32_t wait_timeout_us;   /* bound of every device-side wait, at least 1,000; 0 means
                                   2,000,000 */
    int32_t strict_lengths;     /* 1: entries of kv_lens above max_kv_len set FL_DEVERR_LENGTHS; 0: they
                                   are cut without a word, as fl_attn_decode does.  Entries below 0
                                   count as 0 and set it either way */
} fl_chunk_desc;
/*
 * Layouts (bf16 except lse):
 *   q, out    [T, Hq, D], T >= 1, D = 64 or 128, Hq a multiple of Hk, Hq / Hk <= 128
 *   k_cache, v_cache
 *             paged: [num_pages, page_size, Hk, D], page_size in {16, 32, 64, 128, 256};
 *             contiguous (block_table NULL): [B, S_max, Hk, D], S_max >= max_kv_len
 *   lse       [Hq, T] fp32 (natural log) or NULL
 * out and lse overlap no input.  Rows of no request (past cu_q[B]) are neither
 * read into a result nor written.  A row that sees no key gives O = 0, LSE = -inf.  Keys and values
 * that no row of their request sees (rows kv_lens[b] and later of the last
 * page, keys the window has left) may hold anything; the others must be
 * finite, also where the mask hides them from some rows.  Requests of at most 16
 * rows a KV head sum weights between 2^-60 and 2^60 times values, in fp32:
 * values above 2^37 in size may overflow there, and below 2^-60 vanish.
 * Page indices outside the cache read as zero keys and values.
 * `workspace`, as for fl_attn_decode, holds the call's plan and the partial
 * results of rows whose keys were split over several SMs; they are joined in
 * a fixed order, so that results do not depend on scheduling: a row's bits follow
 * from its own request's data and the lengths of all.
 * Calls sharing one workspace must not overlap on the GPU.
 * For steps of nothing but single tokens over short caches at D = 64
 * fl_attn_decode is faster (it needs no plan); for long ones they are even.
 */
fl_status fl_attn_chunk_workspace_size(const fl_tensor *q, const fl_tensor *k_cache,
                                       const fl_chunk_desc *desc, size_t *bytes);
fl_status fl_attn_chunk(const fl_tensor *q, const fl_tensor *k_cache, const fl_tensor *v_cache,
                        const fl_tensor *out, const fl_tensor *lse, const fl_chunk_desc *desc,
                        void *workspace, size_t workspace_bytes, fl_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FL_ATTN_H */
