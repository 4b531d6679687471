// kernels.h -- internal launchers of the library's CUDA kernels.
// Every launcher enqueues on `st` and returns the cudaGetLastError() of its
// launch; none allocates or synchronises.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dc {

// ---------------------------------------------------------------- top-K
// Segmented top-K: each logits row is cut into `nchunks` segments of
// `chunk_vecs` 16-byte vectors, one CTA per (row, segment).  With several
// segments, every CTA publishes its best K to `part` (rows * nchunks * K
// packed keys) and the last CTA of the row, counted in `row_count` (rows
// entries, zero between calls), merges them.  With `pdl` the launch may
// overlap the end of the previous kernel in the stream (the kernel waits for
// it before its first global write).
struct TopkPlan {
  int nchunks;     // segments per row
  int chunk_vecs;  // 16-byte vectors per segment
};
constexpr int kTopkThreads = 256;
constexpr int kTopkMaxChunks = 64;
// Segment count that gives the shortest launch for `rows` rows on a device
// holding `slots_per_wave` resident top-K CTAs.
TopkPlan topk_plan(int V, int rows, int slots_per_wave);
int topk_min_segments(int V);  // fewest segments whose per-vector maxima fit a CTA
int topk_max_segment_vecs();   // 16-byte vectors a segment may hold
int topk_max_segments(int V);
int topk_occupancy(int K);  // resident top-K CTAs per SM
// With `feat` (fp32 [rows][K][5]) the same pass also accumulates each row's
// log-sum-exp and writes the candidates' vocabulary-normalised features
// [log p, p, l_0 - l_k, k / K, k == 0]; part_lse (float2 [rows][nchunks]) is
// then needed when nchunks > 1.
// Handoff to a projection already running beside the top-K (launched
// before it): the grid is one-dimensional with a row's segments adjacent, so
// rows finish in order; each finished row releases row_ready[row] = 1 (the
// projection clears it) and its candidates' embedding rows E[id] (d bf16
// each) are prefetched into L2.  The kernel then does not wait for the
// previous kernel in the stream (it is the projection, which waits for it).
struct TopkHandoff {
  unsigned *row_ready = nullptr;
  const uint16_t *E = nullptr;
  int d = 0;
};
cudaError_t launch_topk(int K, const uint16_t *logits, int64_t stride, int slots, int N, int V,
                        const TopkPlan &plan, unsigned long long *part, unsigned *row_count,
                        int32_t *ids, float *vals, cudaStream_t st, bool pdl, float2 *part_lse = nullptr,
                        float *feat = nullptr, const TopkHandoff &hand = TopkHandoff());

// ---------------------------------------------------------------- projections
// C[m][o] = sum_k A_m[k] * W[o][k] with A_m a bf16 row of length d, on the
// tensor cores.  A job with `ids` gathers A_m = table[ids[m]] (ids < V, else
// the device status word gets kErrBadCandidateId and row 0 is used); a job
// without takes A_m = table[(m / B) * slots + (m % B) + 1] (the draft-slot
// rows of a [N][slots][d] tensor).  W comes as bf16 hi and lo halves ([No][d]
// each, No % 128 == 0, d % 64 == 0) through two TMA maps (box 64 x 128).
// A CTA owns 256 rows x 128 outputs of one job; `splits` (a power of two
// <= 8, from proj_tc_splits) splits the k range over the CTAs of one
// cluster, which add their partial tiles through distributed shared memory.
// One launch runs one or two jobs, the second one's tiles after the first's.
// With `pdl` the launch may overlap the end of the previous kernel in the
// stream (a gathering job waits for it before it reads the row ids; a
// draft-slot job does not wait).
struct ProjJob {
  const uint16_t *table;  // bf16 [rows][d]
  const int32_t *ids;     // [M] table rows, or null for draft-slot rows
  float *C;               // fp32 [M][No]
  int M, No;
  int tiles;              // proj_tc_tiles(M, No)
  // With ln_hi set (No == 128), each output row leaves as LN0(row) (non-
  // affine, eps ln_eps) split into bf16 hi ([M][128], ln_hi) and lo (the
  // rounding remainder, ln_lo) instead of fp32 in C.
  uint16_t *ln_hi = nullptr, *ln_lo = nullptr;
  float ln_eps = 0.f;
  // With row_ready set (a gathering job launched before the top-K that
  // fills it, see TopkHandoff), a tile waits for the flags of its draft-slot
  // rows (candidate m belongs to row m / cands_per_row) instead of for the
  // previous kernel, and clears them when done.
  unsigned *row_ready = nullptr;
  int cands_per_row = 0;
  // fp16 instead of bf16 hi + lo: A is converted in shared memory (its values
  // must lie within the fp16 range, |a| < 65504) and W comes as one fp16
  // matrix through the `hi` map (the `lo` map is not read).
  bool f16 = false;
};
int proj_tc_splits(int d, int requested);
int proj_tc_tiles(int M, int No);
// 2D bf16 [rows][d] tensor map, 128B swizzle, box 64 x box_rows.
bool encode_bf16_rows_map(CUtensorMap *map, const void *base, int rows, int d, int box_rows);
// The same for fp16 elements.
bool encode_f16_rows_map(CUtensorMap *map, const void *base, int rows, int d, int box_rows);
// 2D fp32 [rows][cols] tensor map, 128B swizzle, box 32 x box_rows
// (cols % 32 == 0).
bool encode_f32_rows_map(CUtensorMap *map, const void *base, int rows, int cols, int box_rows);
cudaError_t launch_proj_tc(const ProjJob &a, const CUtensorMap &a_hi, const CUtensorMap &a_lo,
                           const ProjJob *b, const CUtensorMap *b_hi, const CUtensorMap *b_lo, int slots,
                           int B, int d, int V, int splits, int *err, cudaStream_t st, bool pdl);

// ---------------------------------------------------------------- representations
struct MlpWeightsDev {
  const float *w_la;    // [H]     W1[:, 3r]
  const float *w_lb;    // [H]     W1[:, 3r+1]
  const float *b1;      // [H]  b1 + W1[:, r:2r] beta + W1[:, 2r:3r] beta
  const float *w2;      // [H]
  const float *b2;      // [1]
  const float *w_fg;    // [r][r]  W_fuse[:, r:], in the candidate maps' register order
};

// Tensor-core forms of the per-slot and per-candidate steps.  The maps
// address bf16 hi / lo halves (box 64 x 128, 128B swizzle) of W_fuse[:, :r]
// and W_fuse[:, r:] ([r][r] each), [W1[:, r:2r] ; W1[:, 2r:3r]] diag(gamma)
// ([2H][r]) and W1[:, :r] ([H][r]).
struct MlpMaps {
  CUtensorMap fb_hi, fb_lo, w1_hi, w1_lo, fg_hi, fg_lo, w1s_hi, w1s_lo;
};
// The per-slot and per-candidate maps, in one launch (no block waits for
// another).  Per draft slot i (used for i < B-1):
// P_i = W1[:, :r] (W_pair[:, :d] h_i + W_pair[:, d:] h_{i+1}) + b1' ([rows][H]),
// b1' = b1 + W1[:, r:2r] beta + W1[:, 2r:3r] beta.
// slot_proj is [N*B][3r] = (W_ctx h | W_pair[:, :d] h | W_pair[:, d:] h).
// Per candidate: b = LN0(W_cand E[c]) (from the projection, as bf16 hi and
// lo), g = LN0(W_ctx h) of its slot,
// z = gamma*LN0(W_fuse[:, :r] b + W_fuse[:, r:] g) + beta,
// U = W1_a z + w_la l, V = W1_b z + w_lb l, computed as U = (W1_a diag(gamma))
// n + w_la l with n = LN0(...) (beta's share W1_a beta + W1_b beta is in P,
// so P + U + V is unchanged).  M = N * B * K candidates
// (8 <= K, K divides 128), candidate m belongs to draft slot m / K.
// Tiles move by TMA: `slot.sp` reads slot_proj, `slot.p` writes P,
// `cand.u` / `cand.v` write U and V ([rows][H]) -- fp32 maps with box
// 32 x 128 -- and `cand.bh` / `cand.bl` read b's hi and lo halves (bf16
// [rows][r], box 64 x 128), all over at least the call's rows (rows of the
// last tile past the call's count receive the outputs of stale or all-zero
// input rows).  The launch may overlap the end of the previous kernel
// (programmatic serialization).
struct SlotIoMaps {
  CUtensorMap sp, p;
};
struct CandIoMaps {
  CUtensorMap bh, bl, u, v;
};
cudaError_t launch_maps_tc(const MlpMaps &maps, const SlotIoMaps &slot, const CandIoMaps &cand,
                           const float *slot_proj, const float *topk_val, const MlpWeightsDev &w, int N, int B,
                           int K, float eps, int *err, cudaStream_t st);

// Step 5 outputs and state for a launch that ends with the walk: per-request
// arrays (tokens, choice, accept_len [N][B] / [N]; margin [N][B-1]; target or
// null) and req_count (N entries, zero between calls) counting each
// request's finished pairs.  path_rule 0: prefix-first greedy walk; 1:
// highest-scoring path (Viterbi); 2: beam walk (beam_width 1..4, beam_topm
// 1..K).
struct WalkArgs {
  const int32_t *topk_ids;
  const int32_t *target;  // or null
  int32_t *tokens, *choice, *accept_len;
  float *margin;
  unsigned *req_count;
  int path_rule;    // 0: prefix-first greedy walk, 1: highest-scoring path, 2: beam walk
  int beam_width;   // path rule 2: partial paths kept, 1..4
  int beam_topm;    // path rule 2: successors per predecessor, 1..K
};

// S[n,p,a,b] = l_{p+1}(b) + b2 + sum_j w2_j GELU(P_pj + U_{p,a,j} + V_{p+1,b,j}),
// with P indexed by draft slot ([N*B][H]),
// then, in the last block of each request, its path selection and verify.
cudaError_t launch_pair_score_walk(int K, const float *U, const float *V, const float *P,
                                   const float *topk_val, const float *w2, const float *b2, int N, int B,
                                   float *scores, const WalkArgs &wk, cudaStream_t st);

// ---------------------------------------------------------------- cosine variant
// y = cand_io[m] + slot_io[slot(m)] ([M][2r] and [N*B][2r]), the out half
// (columns 0..r-1) and the in half L2-normalised (x / max(|x|, 1e-12));
// S[n,p,a,b] = sigma <o_{p,a}, i_{p+1,b}> + l_{p+1}(b); then, in the last
// block of each request, its path selection and verify.
cudaError_t launch_cos_pair_walk(int K, const float *cand_io, const float *slot_io, const float *topk_val,
                                 float sigma, int N, int B, float *scores, const WalkArgs &wk, cudaStream_t st);

// ---------------------------------------------------------------- stochastic verify
// Point-mass proposal `tokens` [N][B] against target logits [N][B+1][stride]
// (bf16; row B of a request is the bonus position), temperature 1: slot j is
// accepted iff u_acc[n][j] < q_j(y_j); at the first rejection the corrected
// token is drawn from q_j without y_j, after B acceptances from row B; a draw
// takes the smallest token whose cumulative weight (vocabulary order)
// exceeds u_draw[n] times the total.  Scratch: chunk_m / chunk_s
// [N*(B+1)][verify_chunks(V)], row_lse [N*(B+1)], req_count [N] (zero
// between calls).  q_acc [N][B] receives q_j(y_j).
int verify_chunks(int V);
cudaError_t launch_verify_stochastic(const uint16_t *target, int64_t stride, int V, int N, int B,
                                     const int32_t *tokens, const float *u_acc, const float *u_draw,
                                     float *chunk_m, float *chunk_s, float *row_lse, float *q_acc,
                                     unsigned *req_count, int32_t *accept_len, int32_t *next_token,
                                     cudaStream_t st);

// ---------------------------------------------------------------- tree attention
// Strides in elements; see dcoco_tree_attention.  `group` query heads a K/V
// head; rows of a K/V head are packed t * group + j.
struct TreeAttnParams {
  const uint16_t *q, *k_new, *v_new, *k_cache, *v_cache;
  int64_t q_sn, q_st, q_sh, kn_sn, kn_st, kn_sh, vn_sn, vn_st, vn_sh;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  const int32_t *page_table;
  int64_t pt_stride;
  const int32_t *ctx_len, *tree_len, *tree_mask;  // tree_len, tree_mask: or null
  int64_t mask_sn;
  int num_pages, max_pages, page_shift;
  int N, T, kv_heads, group, head_dim;
  bool f16;
  bool few;  // at most 64 rows a K/V head: launch_tree_attention_few's kernel
  float scale;
  uint16_t *out;  // [N][T][kv_heads * group][head_dim]
  float *lse;     // [N][T][kv_heads * group] or null
  int *err;
  // rows of a K/V head in tiles of tile_nodes nodes (tile_rows = tile_nodes *
  // group <= 128 rows); tree_box: nodes of a K/V copy
  int mtiles, tile_nodes, tile_rows, tree_box;
  // chunks (see tree_chunk_tiles): (request, head, row tile) items of a full
  // batch, SMs, the largest chunk, the most chunks of a request (for this call's
  // kernel and row tiles)
  int items, sms, chunk_cap, max_chunks;
  int part_rows;    // tile_rows as the partial results are laid out: padded by the kernel for few rows
  float4 *part_o;   // [item][max_chunks][part_rows][head_dim], fp32
  float2 *part_ml;  // [item][max_chunks][part_rows] (log2 reference, sum)
};
constexpr int kTreeTile = 128;  // tokens of a K/V tile
struct TreeAttnMaps {
  CUtensorMap q, k_new, v_new, k_cache, v_cache;
};
// Tiles of a chunk for a request of nt tiles: as few as spread a full batch
// of such requests over the SMs, at most `cap` (so that requests of unlike
// lengths balance), and at least nt / kTreeMaxChunks.
constexpr int kTreeMaxChunks = 64;
__host__ __device__ inline int tree_chunk_tiles(int nt, int items, int sms, int cap) {
  const long long want = ((long long)nt * items + sms - 1) / sms;
  int c = want < cap ? (int)want : cap;
  const int least = (nt + kTreeMaxChunks - 1) / kTreeMaxChunks;
  if (c < least) c = least;
  return c < 1 ? 1 : c;
}
cudaError_t launch_tree_attention(const TreeAttnParams &p, cudaStream_t st);
// The kernel for at most 64 rows a K/V head (one row tile), padded to
// tree_few_rows.
inline int tree_few_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
cudaError_t launch_tree_attention_few(const TreeAttnParams &p, const TreeAttnMaps &maps, unsigned grid,
                                      cudaStream_t st);

// ---------------------------------------------------------------- tree commit
struct TreeCommitParams {
  const int32_t *tokens, *parents, *sampled, *tree_len, *ctx_len, *page_table;
  int64_t pt_stride;
  const uint16_t *k_new, *v_new;
  uint16_t *k_cache, *v_cache;
  int64_t kn_sl, kn_sn, kn_st, kn_sh, vn_sl, vn_sn, vn_st, vn_sh;
  int64_t kc_sl, kc_sp, kc_st, kc_sh, vc_sl, vc_sp, vc_st, vc_sh;
  int num_pages, max_pages, page_shift, layers;
  int N, T, kv_heads, head_dim;
  int32_t *path, *accept_len, *next_token, *new_len;
  int *err;
};
cudaError_t launch_tree_commit(const TreeCommitParams &p, cudaStream_t st);

// ---------------------------------------------------------------- K/V in 8 bits
// Attention over a cache of e4m3 payloads with fp32 scales.  Of `t` the cache,
// the row tiles (but tree_box) and the workspace are not used: rows here are (node, query head
// of the K/V head) in one sequence, in tiles of kQuantRows (one tile, padded to
// quant_rows, where they are fewer).
constexpr int kQuantRows = 64, kQuantNodes = 64;  // (nodes of a tile of the tree)
inline int quant_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : kQuantRows; }
struct QuantAttnParams {
  TreeAttnParams t;
  const uint8_t *k_cache, *v_cache;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  const float *k_scale, *v_scale;  // [page][block][kv head]
  int64_t ks_sp, ks_sb, ks_sh, vs_sp, vs_sb, vs_sh;
  int scale_shift;                 // tokens of a block: 1 << scale_shift
  int mtiles, R;                   // row tiles of a K/V head, rows of a tile
  // chunks of the context (see quant_chunk_tiles), and the most units of a
  // request: its chunks and the tree; a unit leaves kQuantRows / R partial results
  int items, sms, chunk_cap, slots;
  uint8_t *q_parts; // [(n, K/V head, row tile)], quant_q_bytes each
  float *part_o;   // [(n, K/V head, row tile)][slots][kQuantRows / R][R][head_dim]
  float2 *part_ml; // the same without head_dim (log2 reference, sum)
};
// Tiles of a chunk for a context of nt tiles: as tree_chunk_tiles, but at most
// kTreeMaxChunks - 1 chunks, so that with the tree's there are kTreeMaxChunks.
__host__ __device__ inline int quant_chunk_tiles(int nt, int items, int sms, int cap) {
  const long long want = ((long long)nt * items + sms - 1) / sms;
  int c = want < cap ? (int)want : cap;
  const int least = (nt + kTreeMaxChunks - 2) / (kTreeMaxChunks - 1);
  if (c < least) c = least;
  return c < 1 ? 1 : c;
}
// Bytes of a row tile's Q: `parts` of 8 bits and one form of 16, and two factors a row.
__host__ __device__ inline int64_t quant_q_bytes(int parts, int R, int D) { return (int64_t)(parts + 2) * R * D + 8 * R; }
cudaError_t launch_quant_attention(const QuantAttnParams &p, cudaStream_t st);

// Tokens' K/V into such a cache: a tree's accepted path, or ragged prompts.
struct QuantWriteParams {
  const uint16_t *k_new, *v_new;
  int64_t kn_sl, kn_sn, kn_st, kn_sh, vn_sl, vn_sn, vn_st, vn_sh;
  uint8_t *k_cache, *v_cache;
  int64_t kc_sl, kc_sp, kc_st, kc_sh, vc_sl, vc_sp, vc_st, vc_sh;
  float *k_scale, *v_scale;
  int64_t ks_sl, ks_sp, ks_sb, ks_sh, vs_sl, vs_sp, vs_sb, vs_sh;
  const int32_t *ctx_len, *page_table;
  int64_t pt_stride;
  int num_pages, max_pages, page_shift, scale_shift, layers;
  int N, kv_heads, head_dim;
  bool f16;
  int *err;
  int32_t *new_len;
  // the tree's path
  const int32_t *tokens, *parents, *sampled, *tree_len;
  int T;
  int32_t *path, *accept_len, *next_token;
  // prompts: rows first[n] .. first[n + 1] - 1 of `total`
  const int32_t *first;
  int total;
};
cudaError_t launch_quant_commit(const QuantWriteParams &p, cudaStream_t st);
cudaError_t launch_quant_append(const QuantWriteParams &p, cudaStream_t st);

// ---------------------------------------------------------------- sampling
// See dcoco_sample.  `f32`: fp32 logits, else bf16.
struct SampleParams {
  const void *logits;
  int64_t stride;
  int rows, V;
  const float *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p, *u;
  int32_t *tokens;
  float *logprob;
};
cudaError_t launch_sample(const SampleParams &p, bool f32, cudaStream_t st);

// ---------------------------------------------------------------- distillation
// See dcoco_distill_loss / _grad / _step.  grad null: the loss alone; loss
// null: the gradient alone, from lse; both: one pass.
struct DistillParams {
  const void *logits;
  int64_t stride;
  int rows, V, K;
  const int32_t *ids;
  const float *teacher, *teacher_lse;
  float temperature;
  const float *grad_loss;
  float *loss, *lse;
  void *grad;
  int64_t grad_stride;
};
cudaError_t launch_distill(const DistillParams &p, bool f32, cudaStream_t st);

// One CTA waits (tc::mbar_wait, limit_ns) on an mbarrier nothing completes:
// the wait expires and ORs kErrTimeout into *err.
cudaError_t launch_wait_timeout(unsigned long long limit_ns, int *err, cudaStream_t st);

}  // namespace dc
