// launch.h -- host-side interface between the C-ABI layer (api.cu) and the
// kernel translation units.  Internal to the library.  Under the runtime
// compiler (NVRTC) only the parameter structs are seen.
#pragma once

#include <cuda_bf16.h>
#ifndef __CUDACC_RTC__
#include <cuda.h>
#include <cuda_runtime.h>
#endif

#include "common.cuh"

namespace fl {

// Parameters of the standard (MHA / GQA) kernel.  Strides are in elements.
struct StdParams {
    GridSpec grid;
    MaskSpec mask;
    int head_dim;         // D = Dv: 32, 64 or 128
    int score_mod;
    float qk_log2;        // scale * log2(e)
    float softcap_in;     // 2 * scale * log2(e) / cap
    float softcap_out;    // cap * log2(e)
    float scale;          // scale (the `score` of a score_mod expression is scale * q.k)
    const float *alibi_slopes;
    float alibi_exp_coef; // default slopes: 2^(alibi_exp_coef * (h + 1)), coef = -8 / Hq
    __nv_bfloat16 *out;
    int64_t o_sb, o_ss, o_sh;
    float *lse;
    int64_t l_sb, l_sh;
    int32_t *tile_counts; // [B][Hq][nq] or null
    uint32_t *err_user;
    int inject;
    uint64_t timeout_ns;
};

// Parameters of the differential-attention kernel (D = 64, Dv = 64 or 128).
struct DiffParams {
    int B, H, Hk, G, nq;
    int dv;               // 64 or 128
    int64_t n_items;
    int lpt, group;
    MaskSpec mask;        // none or causal
    float qk_log2;        // scale * log2(e)
    float lambda;
    __nv_bfloat16 *out;   // [B, S, H, Dv]
    int64_t o_sb, o_ss, o_sh;
    float *lse;           // [2, B, H, S] or null
    int64_t l_s2, l_sb, l_sh;
    int32_t *tile_counts; // [B][H][nq] or null
    uint32_t *err_user;
    uint64_t timeout_ns;
};

#ifndef __CUDACC_RTC__
cudaError_t launch_diff(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                        const DiffParams &p, int grid, cudaStream_t stream);
#endif

// Parameters of the Evoformer kernel (c = 32 or 64) over a [batch, sequence, head, c]
// view: row pass batch = MSA row, sequence = residue; column pass the reverse.
// Work items are (head, query block, chunk of `chunk` batch indices).
struct EvoParams {
    GridSpec grid;          // B, Hq (= heads), nq used
    MaskSpec mask;          // kind NONE; S = length of the attended axis
    int head_dim;           // c: 32 or 64
    int64_t n_items;
    int chunk;
    float qk_log2;          // scale * log2(e)
    float qk_scale;         // scale
    const __nv_bfloat16 *bias; // row pass only (its TMA map is passed separately)
    int bias_rows;          // 0: one bias for every batch index; else a bias per stack of
                            //   bias_rows consecutive batch indices (work items never
                            //   straddle two stacks)
    const __nv_bfloat16 *gate;
    int64_t g_sb, g_si, g_sh;
    __nv_bfloat16 *out;
    int64_t o_sb, o_si, o_sh;
    float *lse;             // [batch, head, sequence] or null
    int64_t l_sb, l_sh;
    int32_t *tile_counts;   // [batch][head][nq] or null
    const void *kmask;      // MSA mask or null: key j of batch index b is removed where
    int64_t km_sb, km_sk;   //   kmask[b * km_sb + j * km_sk] is zero (element strides)
    int km_f32;             //   fp32 entries (else bf16)
    uint32_t *err_user;
    uint64_t timeout_ns;
};

// ---- backward of the standard kind (bwd_standard.cu)
constexpr int kBwdBlock = 64;   // query / key rows per streamed tile
constexpr int kBwdDqRows = 128; // query rows per dQ CTA
constexpr int kBwdKvKeys = 128; // keys per dK / dV CTA
constexpr int kBwdThreads = 384;

// Per query row of the backward's workspace: LSE log2 e, rowsum(dO O) and the
// row's allowed key interval [lo, hi).
struct BwdRowStat {
    float lse2, d;
    int lo, hi;
};

struct BwdParams {
    int B, Hq, Hk, S, S_pad;      // S_pad: S rounded up to 128 (a multiple of kBwdBlock)
    MaskSpec mask;
    float scale;
    int score_mod;                // MOD_NONE, MOD_ALIBI or MOD_SOFTCAP
    float softcap;                // cap (softcap)
    const float *alibi_slopes;    // [Hq] or null: 2^(alibi_exp_coef (h + 1))
    float alibi_exp_coef;
    const __nv_bfloat16 *q, *k, *v, *o, *dout; // element strides (batch, position, head):
    int64_t q_sb, q_ss, q_sh, k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;
    int64_t o_sb, o_ss, o_sh, do_sb, do_ss, do_sh;
    const float *lse;             // [B, Hq, S] natural log
    int64_t l_sb, l_sh;
    __nv_bfloat16 *dq, *dk, *dv;
    int64_t dq_sb, dq_ss, dq_sh, dk_sb, dk_ss, dk_sh, dv_sb, dv_ss, dv_sh;
    BwdRowStat *ws_stats;         // [B][Hq][S_pad]
    uint32_t *err_user;
    uint64_t timeout_ns;
};

// ---- backward of the differential kind (bwd_diff.cu): the combining step
// out[row, 0:64] = sum_p coef[p] in_p[row, 0:64] (fp32 sum of bf16 partials);
// row = (b * S + position) * heads + head of the output view.
struct DiffCombine {
    int64_t rows, S, heads;
    const __nv_bfloat16 *in[2]; // contiguous [rows][64]; in[1] may be null
    float coef[2];
    __nv_bfloat16 *out;         // element strides (batch, position, head); 64 columns contiguous
    int64_t o_sb, o_ss, o_sh;
};

// ---- serving with a KV cache (fwd_decode.cu)
constexpr int kDecodeChunk = 128; // keys per pipeline stage
constexpr int kDecodeMaxSplitChunks = 8; // chunks per CTA (split) at most
constexpr int kDecodeMaxRows = 64; // G * Sq query rows per (sequence, KV head)

struct DecodeParams {
    int B, Hk, G, Sq;
    int max_kv;
    int split_chunks, max_splits; // chunks per split; splits of the longest sequence
    int page;                     // keys per page (paged cache)
    int64_t bt_stride;            // block_table row stride
    const int32_t *kv_lens;       // [B]
    const int32_t *block_table;   // [B][bt_stride] or null (contiguous cache)
    const __nv_bfloat16 *q;       // [B, Sq, Hq, 64] element strides:
    int64_t q_sb, q_ss, q_sh;
    __nv_bfloat16 *out;
    int64_t o_sb, o_ss, o_sh;
    float *lse;                   // [B, Hq, Sq] or null
    int64_t l_sb, l_sh;
    float scale, softcap;         // softcap 0: none
    int causal;
    float *ws_o;                  // [B][Hk][max_splits][R][64]
    float *ws_ml;                 // [B][Hk][max_splits][R][2]: base-2 max, sum
    int *ws_cnt;                  // [B][Hk], zero before the launch
    uint32_t *err_user;
    uint64_t timeout_ns;
};

#ifndef __CUDACC_RTC__
cudaError_t launch_decode(const CUtensorMap &tk, const CUtensorMap &tv, const DecodeParams &p,
                          cudaStream_t stream);
size_t decode_smem_bytes(int R);

// Size of the library's own decode scratch array (fl_attn_decode_static).
constexpr size_t kDecodeStaticScratch = size_t(64) << 20;
cudaError_t decode_static_scratch(void **ptr);

cudaError_t launch_diff_bwd_combine(const DiffCombine &c, int sm_count, cudaStream_t stream);

cudaError_t launch_evo(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                       const CUtensorMap &tb, const EvoParams &p, int grid, cudaStream_t stream);
cudaError_t launch_bwd_prep(const BwdParams &p, cudaStream_t stream);
// Dynamic shared memory and block count of the fused dK/dV + dQ launch.
size_t bwd_smem_bytes();
int64_t bwd_fused_blocks(const BwdParams &p);
// The main backward kernel specialised for a translated expression `cuda`
// with derivative `grad` (run-time compiled, like launch_standard_expr);
// launch_bwd_prep must have run first on the same stream.
cudaError_t launch_bwd_expr(const CUtensorMap &tq, const CUtensorMap &tdo, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &tq128, const CUtensorMap &tdo128,
                            const CUtensorMap &tk128, const CUtensorMap &tv128, const BwdParams &p,
                            cudaStream_t stream, const char *cuda, const char *grad, char *err, size_t err_n);
cudaError_t launch_bwd(const CUtensorMap &tq, const CUtensorMap &tdo, const CUtensorMap &tk,
                       const CUtensorMap &tv, const CUtensorMap &tq128, const CUtensorMap &tdo128,
                       const CUtensorMap &tk128, const CUtensorMap &tv128, const BwdParams &p,
                       cudaStream_t stream);
#endif

// Keys per K/V tile of the standard kernel for head dimension D (its TMEM
// budget: see fwd_standard.cu), its threads per CTA and the registers per
// thread it must be compiled to.
__host__ __device__ constexpr int std_key_tile(int D) { return D == 128 ? 64 : D == 64 ? 112 : 128; }
constexpr int kStdThreads = 384;
constexpr int kStdRegs = 168;
// Keys per K/V tile of the differential kernel for value head dimension Dv
// (its TMEM budget: see fwd_diff.cu).
__host__ __device__ constexpr int diff_key_tile(int dv) { return dv == 128 ? 80 : 112; }

#ifndef __CUDACC_RTC__
cudaError_t launch_standard(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const StdParams &p, int grid, cudaStream_t stream);
size_t standard_smem_bytes(int head_dim);

// ---- score_mod expressions (score_expr.cu)
// Checks `expr` against the expression grammar of fl_attn.h and writes the
// equivalent fp32 CUDA expression to `cuda` (NUL-terminated, at most `n`
// bytes); false with a message in `err` otherwise.
bool score_expr_translate(const char *expr, char *cuda, size_t n, char *err, size_t err_n);
// The same, also writing the derivative of the expression with respect to
// `score` (forward-mode differentiation through the grammar) to `grad`.
bool score_expr_translate_grad(const char *expr, char *cuda, size_t n, char *grad, size_t grad_n, char *err,
                               size_t err_n);
// Runs the runtime compilation of the standard kernel for the translated
// expression `cuda`, and of the backward kernels for it and its derivative
// `grad` (unless null), without loading them (needs no device).
bool score_expr_compile_only(const char *cuda, const char *grad, char *err, size_t err_n);
// The standard kernel specialised for the translated expression `cuda`:
// compiled at run time on first use (per device and expression), then
// launched like launch_standard.  Errors other than CUDA ones are described
// in `err`.
cudaError_t launch_standard_expr(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                 const StdParams &p, int grid, cudaStream_t stream, const char *cuda,
                                 char *err, size_t err_n);
#endif

// ---- rotary positions and the cache append (rope.cu)
// One tensor's way through the kernel: `heads` heads of every token from src
// to dst (element strides; the batch and sequence strides of dst are the page
// and row strides for a tensor that goes to the cache).
struct RopeStream {
    const void *src;
    void *dst;
    int64_t s_b, s_s, s_h;
    int64_t d_b, d_s, d_h;
    int heads;
    FastDiv div_heads;
    int rotate;   // 0: copied
    int to_cache; // dst row by slot instead of by token
    int tile;     // tokens per block (set by launch_rope)
};

struct RopeParams {
    RopeStream st[3];
    int n_streams;
    int tokens;                // B * S
    int pairs, pass;           // rotated pairs and copied elements of a head
    int rot;
    int units, uy;             // vector units of a head; rows a block walks at a time
    FastDiv div_ux, div_pairs, div_seq;
    int64_t page_rows;
    const int32_t *positions;  // [B][positions_stride] or null
    int64_t positions_stride;
    int64_t offset;
    const int64_t *slots;      // [tokens] or null
    int64_t n_slots;           // rows of the cache
    int backward;
    float magnitude;
    uint64_t turns[128];
};

// ---- a cache of e4m3 codes written and read back (kv_fp8.cu)
// One tensor's way into the cache (element strides; scales have heads innermost).
struct Fp8Stream {
    const __nv_bfloat16 *src;
    int64_t s_s, s_h;
    uint8_t *cache;
    int64_t d_p, d_r, d_h;
    float *scale;
    int64_t s_p, s_b;
};
struct Fp8AppendParams {
    RopeParams rope;           // of q, where given, and k; the slots
    Fp8Stream k, v;
    int heads, lane_shift;     // KV heads; log2 of a row's 16-element pieces
    int block_shift;           // log2 of the keys per scale
    FastDiv div_group;         // heads of a group; groups, tokens per chunk of a
    int groups, chunk, tile;   // run and window, rows of the grid for q (set by
    int q_rows;                // launch_append_fp8)
};
struct Fp8ReadStream {
    const uint8_t *cache;
    int64_t d_p, d_r, d_h;
    const float *scale;
    int64_t s_p, s_b;
    void *out;
    int64_t o_t, o_h;
};
struct Fp8ReadParams {
    Fp8ReadStream st[2];
    int n_streams, tokens;
    const int64_t *slots;
    int64_t n_slots, page_rows;
    int block_shift;
    int units, head_shift;     // 16-byte units of a token's output, log2 of those of a head
    FastDiv div_units;         // units and tokens that a block walks at a time, its tokens
    int uy, tile;              // (set by launch_read_fp8)
};

// ---- the book-keeping of a serving step (kv_plan.cu)
struct KvPlanParams {
    int batch, max_tokens, n_free, bt_stride;
    int page_shift;
    const int32_t *q_lens, *kv_lens, *free_pages, *free_head;
    int32_t *block_table, *kv_out, *cu_q, *positions, *head_out;
    int64_t *slots;
    uint32_t *err_user;
};

// ---- attention of ragged chunks over the cache (fwd_chunk.cu)
constexpr int kChunkMaxCtas = 160; // persistent CTAs the workspace has room for
// Keys per K/V tile (the standard kernel's, for the same TMEM budget), and of
// the few-row path.
__host__ __device__ constexpr int chunk_key_tile(int D) { return D == 128 ? 64 : 112; }
__host__ __device__ constexpr int few_tile(int D, bool f8) { return f8 && D == 64 ? 256 : 128; }
constexpr int kFewRows = 16; // query rows of a request and KV head, at most

// One or two row blocks of a request, as the planning kernel lists them.
struct alignas(16) ChunkEntry {
    int b, t0, n_tok, pos0;    // request, first token row, tokens, position of the first
    int L, key_lo;             // cached keys; lowest key that the rows see
    int lo, n_tiles;           // key tiles [lo, lo + n_tiles)
    int tile_cost, pad;
    int64_t cum;               // cost of everything before it on its list, all heads
};
// A CTA's part of the work: [first, end) of the cost units of its list.
struct alignas(16) ChunkPart {
    int64_t total, end;        // cost of the whole list; the part's end
    int parts, cta;            // parts of the list (0: none); this part among those of both
    int n_entries;
    int entry, item, tile, pad[2]; // where the part begins
    ChunkEntry at;             // that entry
};
// An item whose keys were cut, by the CTA it begins in.
struct ChunkJoin {
    int n_parts;               // 0 or 1: nothing to join
    int mode;                  // how its parts are laid out (chunk_plan.cuh)
    int kvh;
    int t0[2], rows[2];        // per slot: first token row, rows
    int pad;
};

struct ChunkParams {
    int T, batch, Hq, Hk, G, head_dim;
    int TQ;                    // tokens per 128-row block: 128 / G
    FastDiv div_g;
    FastDiv div_per;           // 2 TQ, tokens per entry
    int few_tq;                // tokens of few rows: kFewRows / G
    int few_shift;             // log2 of the keys per TMA box of the few-row path
    int max_kv, page_shift;    // page_shift < 0: contiguous cache
    int strict;                // lengths above max_kv are reported
    int64_t bt_stride;
    const int32_t *cu_q, *kv_lens, *block_table;
    int causal, window;        // window 0: none
    int score_mod;
    float qk_log2;             // scale * log2(e)
    float softcap_in;          // 2 * scale * log2(e) / cap
    float softcap_out;         // cap * log2(e)
    __nv_bfloat16 *out;        // element strides (token, head)
    int64_t o_st, o_sh;
    float *lse;                // [Hq, T] or null
    int64_t l_sh;
    int device, n_cta;
    int cost_pair, cost_single, cost_few, cost_item, cost_few_item, cost_least; // see api.cu
    int max_entries;
    int second;                // the other path's kernel comes first (chunk_plan.cuh)
    uint64_t *seen;            // holds seen_mark once that one has seen the plan
    uint64_t seen_mark;        // this call's; 0: one path alone
    int warm;                  // few rows: run a tile of no keys first
    ChunkPart *parts;          // the workspace: [2][n_cta], row blocks and few rows
    ChunkJoin *joins;          // [n_cta]
    ChunkEntry *entries;       // [2][max_entries]
    float *partials;           // [n_cta][2][2][D + 4][128]
    uint32_t *err_user;
    uint64_t timeout_ns;
    // a cache in 8 bits: scales [page][block of keys][head], element strides
    const float *k_scale, *v_scale;
    int64_t ks_p, ks_b, vs_p, vs_b;
    int scale_shift;           // log2 of the keys per block
    int n_pages;
    int cost_more;             // of a tile of few rows that are more than 8, at least cost_few
    const __nv_bfloat16 *q;    // element strides (token, head)
    int64_t q_st, q_sh;
    uint8_t *q8;               // the workspace: [2][T][Hq][D], q's e4m3 terms
    float *q_scale;            // [T][Hq], their scales
};

#ifndef __CUDACC_RTC__
// vec: elements per vector access (a power of two up to 16 bytes' worth)
cudaError_t launch_rope(const RopeParams &p, bool fp32, bool interleaved, int vec, int sm_count,
                        cudaStream_t stream);
cudaError_t launch_append_fp8(const Fp8AppendParams &p, bool interleaved, int sm_count, cudaStream_t stream);
cudaError_t launch_read_fp8(const Fp8ReadParams &p, bool fp32, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t stream);
// Tensor maps: a row block of q and boxes of 16 keys; few rows of q and boxes
// of few_box keys.
struct ChunkMaps {
    CUtensorMap q, k, v, few_q, few_k, few_v;
};
cudaError_t launch_chunk(const ChunkMaps &maps, const ChunkParams &p, cudaStream_t stream);
cudaError_t launch_chunk_fp8(const ChunkMaps &maps, const ChunkParams &p, cudaStream_t stream);
#endif

}  // namespace fl
