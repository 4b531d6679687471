// tree.cu -- C ABI of the tree calls (declared in include/dcoco.h): handle,
// argument checks and launches of tree attention and tree commit, and the
// handle-free sampling and distillation entries.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>
#include <new>

#include "../../include/dcoco.h"
#include "kernels.h"

struct dcoco_tree_handle {
  dcoco_tree_config cfg;
  int device = 0;
  int page_shift = 0, sms = 1;
  // the most chunks of a request (see TreeAttnParams): of the kernel for few
  // rows, and of the other by the number of row tiles
  int few_chunks = 0;
  uint8_t many_chunks[257] = {};
  void *block = nullptr;              // one device allocation: status word, partial results
  int *err = nullptr;
  float2 *part_ml = nullptr;
  float4 *part_o = nullptr;
  cudaStream_t last_stream = nullptr;
  long long launches = 0;
};

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool good(const void *p) { return p && aligned16(p); }
// Strides of axes with these extents: multiples of 8 elements (16 bytes), and
// positive where the axis has more than one entry.
bool steps8(std::initializer_list<int64_t> strides, std::initializer_list<int> extents) {
  const int *n = extents.begin();
  for (int64_t s : strides)
    if (*n++ > 1 && (s <= 0 || s % 8 != 0 || s >= (1ll << 39))) return false;
  return true;
}
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? DCOCO_OK : DCOCO_ECUDA; }

int validate_tree_config(const dcoco_tree_config *c) {
  if (!c) return DCOCO_EINVAL;
  if (c->max_batch < 1 || c->max_batch > 4096 || c->max_tree < 1 || c->max_tree > 256) return DCOCO_EINVAL;
  if (c->kv_heads < 1 || c->q_heads < c->kv_heads || c->q_heads > 1024 || c->q_heads % c->kv_heads != 0)
    return DCOCO_EINVAL;
  if (c->page_size < 1 || c->max_pages < 1 || (int64_t)c->page_size * c->max_pages > (1ll << 30)) return DCOCO_EINVAL;
  if (c->q_heads / c->kv_heads > 128) return DCOCO_EUNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return DCOCO_EUNSUPPORTED;
  if (c->dtype != DCOCO_BF16 && c->dtype != DCOCO_FP16) return DCOCO_EUNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return DCOCO_EUNSUPPORTED;
  return DCOCO_OK;
}

// Rows of a K/V head (nodes x group) in tiles of at most 128, whole nodes each.
struct RowTiles {
  int tile_nodes, tile_rows, mtiles, part_rows;
  bool few;
  RowTiles(const dcoco_tree_config &c, int nodes) {
    const int group = c.q_heads / c.kv_heads, most = 128 / group;
    tile_nodes = nodes < most ? nodes : most;
    tile_rows = tile_nodes * group;
    mtiles = (nodes + tile_nodes - 1) / tile_nodes;
    few = mtiles == 1 && tile_rows <= 64;
    part_rows = few ? dc::tree_few_rows(tile_rows) : tile_rows;
  }
};

// The largest chunk in tiles.  One request at a time: whatever spreads it over
// the SMs.  Several differ in length, and small chunks balance them, but each
// costs its block a unit border and leaves a partial result.  Measured: 32
// requests x 16 nodes, 64 rows, to 8000 tokens: 136 / 133 / 133 us at 8 / 16 /
// 32 tiles; 24 x 1, 4 rows, to 16001: 114 / 103 / 105 us.  The kernel for many
// rows, whose borders cost more, at 32 / 48 / 64 / 96 tiles: 8 x 64, three
// tiles of 125 rows, to 32000: 310 / 305 / 314 / 308 us; 32 x 64 to 8000: 369 /
// 352 / 341 / 342 us; 16 x 128 to 16000: 641 / 605 / 583 / 560 us.  (96 was as
// good or better in these and is not taken yet.)
//
// The handle's batch, not the call's, so that a request's result has the same
// bits whatever runs beside it.  Its price: one request on a handle for 32, 8
// K/V heads of 128, in a graph, against a handle for one: 16 nodes x 4 heads at
// 1000 tokens 20 us (13), at 8000 28 (20); 64 nodes x 5 at 4000 50 (25), at 8000
// 83 (31).  Four requests: 21 (16), 30 (27), 55 (42), 91 (60).
int chunk_cap(const dcoco_tree_config &c, bool few) { return c.max_batch == 1 ? 1 << 30 : few ? 16 : 64; }

// The most chunks that a request of up to max_tiles tiles is cut into, with
// `items` (request, head, row tile) items in a full batch.
int most_chunks(int64_t max_tiles, int items, int sms, int cap) {
  // (from 64 tiles a chunk on, the largest cap, the rule's other limit holds: kTreeMaxChunks)
  const int64_t scan = max_tiles < 64 * dc::kTreeMaxChunks ? max_tiles : 64 * dc::kTreeMaxChunks;
  int most = max_tiles > scan ? dc::kTreeMaxChunks : 1;
  for (int nt = 1; nt <= scan; ++nt) {
    const int per = dc::tree_chunk_tiles(nt, items, sms, cap), n = (nt + per - 1) / per;
    if (n > most) most = n;
  }
  return most;
}

int check_distill(int rows, int vocab, const void *logits, int dtype, int64_t row_stride, int topk,
                  const int32_t *ids, const float *teacher, float temperature) {
  if (rows < 0 || vocab < 1 || vocab > (1 << 20) || topk < 1 || topk > 1024) return DCOCO_EINVAL;
  if (dtype != DCOCO_BF16 && dtype != DCOCO_FP32) return DCOCO_EINVAL;
  if (row_stride < vocab || row_stride % 8 != 0) return DCOCO_EINVAL;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return DCOCO_EINVAL;
  if (rows > 0 && (!good(logits) || !ids || !teacher)) return DCOCO_EINVAL;
  return DCOCO_OK;
}

}  // namespace

extern "C" {

int dcoco_tree_create(const dcoco_tree_config *cfg, dcoco_tree_handle **out) {
  if (!out) return DCOCO_EINVAL;
  const int rc = validate_tree_config(cfg);
  if (rc != DCOCO_OK) return rc;
  dcoco_tree_handle *h = new (std::nothrow) dcoco_tree_handle();
  if (!h) return DCOCO_ENOMEM;
  h->cfg = *cfg;
  while ((1 << h->page_shift) < cfg->page_size) ++h->page_shift;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
    delete h;
    return DCOCO_ECUDA;
  }
  const int64_t max_tiles = ((int64_t)cfg->page_size * cfg->max_pages + dc::kTreeTile - 1) / dc::kTreeTile +
                            (cfg->max_tree + dc::kTreeTile - 1) / dc::kTreeTile;
  // Partial results of the largest call, over the numbers of nodes up to max_tree:
  // of either kernel its own chunks and rows (the most nodes that a number of row
  // tiles stands for have the most rows)
  const int group = cfg->q_heads / cfg->kv_heads, pairs = cfg->max_batch * cfg->kv_heads;
  size_t rows = 0;
  const auto reach = [&](int nodes) {
    const RowTiles rt(*cfg, nodes);
    const int n = most_chunks(max_tiles, pairs * rt.mtiles, h->sms, chunk_cap(*cfg, rt.few));
    if (rt.few) h->few_chunks = n;
    else h->many_chunks[rt.mtiles] = (uint8_t)n;
    const size_t r = (size_t)pairs * rt.mtiles * n * rt.part_rows;
    if (r > rows) rows = r;
  };
  const int few_nodes = 64 / group, tile_nodes = 128 / group;
  if (few_nodes >= 1) reach(few_nodes < cfg->max_tree ? few_nodes : cfg->max_tree);
  for (int nodes = tile_nodes; nodes - tile_nodes < cfg->max_tree; nodes += tile_nodes)
    if (!RowTiles(*cfg, nodes < cfg->max_tree ? nodes : cfg->max_tree).few)
      reach(nodes < cfg->max_tree ? nodes : cfg->max_tree);
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t at_ml = 256, at_o = at_ml + up(rows * sizeof(float2));
  const size_t bytes = at_o + rows * cfg->head_dim * sizeof(float);
  if (cudaMalloc(&h->block, bytes) != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return DCOCO_ENOMEM;
  }
  char *base = static_cast<char *>(h->block);
  h->err = reinterpret_cast<int *>(base);
  h->part_ml = reinterpret_cast<float2 *>(base + at_ml);
  h->part_o = reinterpret_cast<float4 *>(base + at_o);
  if (cudaMemset(base, 0, 256) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    cudaFree(h->block);
    delete h;
    return DCOCO_ECUDA;
  }
  *out = h;
  return DCOCO_OK;
}

int dcoco_tree_attention(dcoco_tree_handle *h, int batch, int nodes, const dcoco_tree_attention_args *a,
                         void *out, float *lse, void *stream) {
  if (!h || !a) return DCOCO_EINVAL;
  const dcoco_tree_config &c = h->cfg;
  if (batch < 0 || batch > c.max_batch) return DCOCO_EBATCH;
  if (nodes < 0 || nodes > c.max_tree) return DCOCO_EINVAL;
  if (batch == 0 || nodes == 0) return DCOCO_OK;
  if (!good(a->q) || !good(a->k_new) || !good(a->v_new) || !good(a->k_cache) || !good(a->v_cache) || !good(out) ||
      !a->page_table || !a->ctx_len)
    return DCOCO_EINVAL;
  if (!steps8({a->q_stride_n, a->q_stride_t, a->q_stride_h}, {batch, nodes, c.q_heads}) ||
      !steps8({a->k_new_stride_n, a->k_new_stride_t, a->k_new_stride_h}, {batch, nodes, c.kv_heads}) ||
      !steps8({a->v_new_stride_n, a->v_new_stride_t, a->v_new_stride_h}, {batch, nodes, c.kv_heads}) ||
      !steps8({a->k_cache_stride_page, a->k_cache_stride_token, a->k_cache_stride_h},
              {a->num_pages, c.page_size, c.kv_heads}) ||
      !steps8({a->v_cache_stride_page, a->v_cache_stride_token, a->v_cache_stride_h},
              {a->num_pages, c.page_size, c.kv_heads}))
    return DCOCO_EINVAL;
  if (a->num_pages < 1 || a->page_table_stride < c.max_pages || a->tree_mask_stride_n < 0 || !std::isfinite(a->scale))
    return DCOCO_EINVAL;
  dc::TreeAttnParams p;
  p.q = (const uint16_t *)a->q, p.k_new = (const uint16_t *)a->k_new, p.v_new = (const uint16_t *)a->v_new;
  p.k_cache = (const uint16_t *)a->k_cache, p.v_cache = (const uint16_t *)a->v_cache;
  p.q_sn = a->q_stride_n, p.q_st = a->q_stride_t, p.q_sh = a->q_stride_h;
  p.kn_sn = a->k_new_stride_n, p.kn_st = a->k_new_stride_t, p.kn_sh = a->k_new_stride_h;
  p.vn_sn = a->v_new_stride_n, p.vn_st = a->v_new_stride_t, p.vn_sh = a->v_new_stride_h;
  p.kc_sp = a->k_cache_stride_page, p.kc_st = a->k_cache_stride_token, p.kc_sh = a->k_cache_stride_h;
  p.vc_sp = a->v_cache_stride_page, p.vc_st = a->v_cache_stride_token, p.vc_sh = a->v_cache_stride_h;
  p.page_table = a->page_table, p.pt_stride = a->page_table_stride;
  p.ctx_len = a->ctx_len, p.tree_len = a->tree_len, p.tree_mask = a->tree_mask, p.mask_sn = a->tree_mask_stride_n;
  p.num_pages = a->num_pages, p.max_pages = c.max_pages, p.page_shift = h->page_shift;
  p.N = batch, p.T = nodes, p.kv_heads = c.kv_heads, p.group = c.q_heads / c.kv_heads, p.head_dim = c.head_dim;
  p.f16 = c.dtype == DCOCO_FP16;
  p.scale = a->scale;
  p.out = (uint16_t *)out, p.lse = lse, p.err = h->err;
  const RowTiles rt(c, nodes);
  p.mtiles = rt.mtiles, p.tile_nodes = rt.tile_nodes, p.tile_rows = rt.tile_rows;
  p.part_rows = rt.part_rows, p.few = rt.few;
  p.tree_box = nodes < dc::kTreeTile ? (nodes + 7) / 8 * 8 : dc::kTreeTile;
  p.items = c.max_batch * c.kv_heads * rt.mtiles, p.sms = h->sms;
  p.chunk_cap = chunk_cap(c, rt.few), p.max_chunks = rt.few ? h->few_chunks : h->many_chunks[rt.mtiles];
  p.part_o = h->part_o, p.part_ml = h->part_ml;
  h->last_stream = static_cast<cudaStream_t>(stream);
  h->launches += 2;
  return cuda_status(dc::launch_tree_attention(p, h->last_stream));
}

int dcoco_tree_commit(dcoco_tree_handle *h, int batch, int nodes, const dcoco_tree_commit_args *a, int32_t *path,
                      int32_t *accept_len, int32_t *next_token, int32_t *new_len, void *stream) {
  if (!h || !a) return DCOCO_EINVAL;
  const dcoco_tree_config &c = h->cfg;
  if (batch < 0 || batch > c.max_batch) return DCOCO_EBATCH;
  if (nodes < 0 || nodes > c.max_tree) return DCOCO_EINVAL;
  if (batch == 0 || nodes == 0) return DCOCO_OK;
  if (!a->tokens || !a->parents || !a->sampled || !a->ctx_len || !a->page_table || !path || !accept_len ||
      !next_token || !new_len || !good(a->k_new) || !good(a->v_new) || !good(a->k_cache) || !good(a->v_cache))
    return DCOCO_EINVAL;
  if (!steps8({a->k_new_stride_l, a->k_new_stride_n, a->k_new_stride_t, a->k_new_stride_h},
              {a->layers, batch, nodes, c.kv_heads}) ||
      !steps8({a->v_new_stride_l, a->v_new_stride_n, a->v_new_stride_t, a->v_new_stride_h},
              {a->layers, batch, nodes, c.kv_heads}) ||
      !steps8({a->k_cache_stride_l, a->k_cache_stride_page, a->k_cache_stride_token, a->k_cache_stride_h},
              {a->layers, a->num_pages, c.page_size, c.kv_heads}) ||
      !steps8({a->v_cache_stride_l, a->v_cache_stride_page, a->v_cache_stride_token, a->v_cache_stride_h},
              {a->layers, a->num_pages, c.page_size, c.kv_heads}))
    return DCOCO_EINVAL;
  if (a->num_pages < 1 || a->layers < 1 || a->layers > 65535 || a->page_table_stride < c.max_pages ||
      new_len == a->ctx_len)
    return DCOCO_EINVAL;
  dc::TreeCommitParams p;
  p.tokens = a->tokens, p.parents = a->parents, p.sampled = a->sampled, p.tree_len = a->tree_len;
  p.ctx_len = a->ctx_len, p.page_table = a->page_table, p.pt_stride = a->page_table_stride;
  p.k_new = (const uint16_t *)a->k_new, p.v_new = (const uint16_t *)a->v_new;
  p.k_cache = (uint16_t *)a->k_cache, p.v_cache = (uint16_t *)a->v_cache;
  p.kn_sl = a->k_new_stride_l, p.kn_sn = a->k_new_stride_n, p.kn_st = a->k_new_stride_t, p.kn_sh = a->k_new_stride_h;
  p.vn_sl = a->v_new_stride_l, p.vn_sn = a->v_new_stride_n, p.vn_st = a->v_new_stride_t, p.vn_sh = a->v_new_stride_h;
  p.kc_sl = a->k_cache_stride_l, p.kc_sp = a->k_cache_stride_page;
  p.kc_st = a->k_cache_stride_token, p.kc_sh = a->k_cache_stride_h;
  p.vc_sl = a->v_cache_stride_l, p.vc_sp = a->v_cache_stride_page;
  p.vc_st = a->v_cache_stride_token, p.vc_sh = a->v_cache_stride_h;
  p.num_pages = a->num_pages, p.max_pages = c.max_pages, p.page_shift = h->page_shift, p.layers = a->layers;
  p.N = batch, p.T = nodes, p.kv_heads = c.kv_heads, p.head_dim = c.head_dim;
  p.path = path, p.accept_len = accept_len, p.next_token = next_token, p.new_len = new_len, p.err = h->err;
  h->last_stream = static_cast<cudaStream_t>(stream);
  ++h->launches;
  return cuda_status(dc::launch_tree_commit(p, h->last_stream));
}

int dcoco_tree_status(dcoco_tree_handle *h) {
  if (!h) return DCOCO_EINVAL;
  if (cudaStreamSynchronize(h->last_stream) != cudaSuccess) return DCOCO_ECUDA;
  int flag = 0;
  if (cudaMemcpy(&flag, h->err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return DCOCO_ECUDA;
  if (flag != 0) {
    if (cudaMemset(h->err, 0, sizeof(int)) != cudaSuccess) return DCOCO_ECUDA;
    return DCOCO_EDEVICE;
  }
  return DCOCO_OK;
}

long long dcoco_tree_launches(const dcoco_tree_handle *h) { return h ? h->launches : -1; }

void dcoco_tree_destroy(dcoco_tree_handle *h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->block);
  delete h;
}

int dcoco_sample(int rows, int vocab, const void *logits, int dtype, int64_t row_stride, const float *temperature,
                 const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *tokens,
                 float *logprob, void *stream) {
  if (rows < 0 || vocab < 1 || vocab > (1 << 20) || row_stride < vocab || row_stride % 8 != 0) return DCOCO_EINVAL;
  if (dtype != DCOCO_BF16 && dtype != DCOCO_FP32) return DCOCO_EINVAL;
  if (rows == 0) return DCOCO_OK;
  if (!good(logits) || !u || !tokens) return DCOCO_EINVAL;
  const dc::SampleParams p{logits, row_stride, rows, vocab, temperature, top_k, top_p, min_p, u, tokens, logprob};
  return cuda_status(dc::launch_sample(p, dtype == DCOCO_FP32, static_cast<cudaStream_t>(stream)));
}

int dcoco_distill_loss(int rows, int vocab, const void *logits, int dtype, int64_t row_stride, int topk,
                       const int32_t *teacher_ids, const float *teacher_logits, const float *teacher_lse,
                       float temperature, float *loss, float *lse, void *stream) {
  const int rc = check_distill(rows, vocab, logits, dtype, row_stride, topk, teacher_ids, teacher_logits, temperature);
  if (rc != DCOCO_OK || rows == 0) return rc;
  if (!loss || !lse) return DCOCO_EINVAL;
  const dc::DistillParams p{logits, row_stride, rows, vocab, topk, teacher_ids, teacher_logits, teacher_lse,
                            temperature, nullptr, loss, lse, nullptr, 0};
  return cuda_status(dc::launch_distill(p, dtype == DCOCO_FP32, static_cast<cudaStream_t>(stream)));
}

int dcoco_distill_grad(int rows, int vocab, const void *logits, int dtype, int64_t row_stride, int topk,
                       const int32_t *teacher_ids, const float *teacher_logits, const float *teacher_lse,
                       float temperature, const float *lse, const float *grad_loss, void *grad, int64_t grad_stride,
                       void *stream) {
  const int rc = check_distill(rows, vocab, logits, dtype, row_stride, topk, teacher_ids, teacher_logits, temperature);
  if (rc != DCOCO_OK) return rc;
  if (grad_stride < vocab || grad_stride % 8 != 0) return DCOCO_EINVAL;
  if (rows == 0) return DCOCO_OK;
  if (!lse || !grad_loss || !good(grad) || (grad == logits && grad_stride != row_stride)) return DCOCO_EINVAL;
  const dc::DistillParams p{logits, row_stride, rows, vocab, topk, teacher_ids, teacher_logits, teacher_lse,
                            temperature, grad_loss, nullptr, const_cast<float *>(lse), grad, grad_stride};
  return cuda_status(dc::launch_distill(p, dtype == DCOCO_FP32, static_cast<cudaStream_t>(stream)));
}

int dcoco_distill_step(int rows, int vocab, const void *logits, int dtype, int64_t row_stride, int topk,
                       const int32_t *teacher_ids, const float *teacher_logits, const float *teacher_lse,
                       float temperature, const float *grad_loss, float *loss, float *lse, void *grad,
                       int64_t grad_stride, void *stream) {
  const int rc = check_distill(rows, vocab, logits, dtype, row_stride, topk, teacher_ids, teacher_logits, temperature);
  if (rc != DCOCO_OK) return rc;
  if (grad_stride < vocab || grad_stride % 8 != 0) return DCOCO_EINVAL;
  if (rows == 0) return DCOCO_OK;
  if (!loss || !lse || !grad_loss || !good(grad) || (grad == logits && grad_stride != row_stride)) return DCOCO_EINVAL;
  const dc::DistillParams p{logits, row_stride, rows, vocab, topk, teacher_ids, teacher_logits, teacher_lse,
                            temperature, grad_loss, loss, lse, grad, grad_stride};
  return cuda_status(dc::launch_distill(p, dtype == DCOCO_FP32, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
