// tree_commit.cu -- the accepted path of a drafted tree, and its K/V into the
// paged cache of every layer.
//
// With s(t) the target's token after node t: the path starts at node 0 and
// goes from node t to the lowest child c (parent c = t) with token c = s(t),
// until there is none; s(last) is the next token.
//
// One block a (request, layer).  Every block walks the tree itself (a walk is
// a few steps over lists that fit in shared memory, so a second launch or a
// grid-wide wait would cost more than repeating it) and copies its layer's
// rows of the path, 16 bytes a thread.
// Bound by latency: lengths and tree, the walk, the page table, the copy, each
// waiting for the one before; 32 requests x 64 nodes x 16 layers 8.6 us in a
// graph, one request x 16 nodes 4.6 us.
#include "common.cuh"
#include "kernels.h"

namespace dc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxNodes = 256;

__global__ void __launch_bounds__(kThreads) k_tree_commit(const TreeCommitParams p) {
  __shared__ int s_tok[kMaxNodes], s_par[kMaxNodes], s_want[kMaxNodes], s_path[kMaxNodes];
  __shared__ int s_count;
  const int n = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int64_t base = (int64_t)n * p.T;
  const int capacity = p.max_pages << p.page_shift;
  int bad = 0;
  int len = p.tree_len ? p.tree_len[n] : p.T, ctx = p.ctx_len[n];
  if (len < 0 || len > p.T) bad |= kErrBadLength, len = len < 0 ? 0 : p.T;
  if (ctx < 0 || ctx > capacity) bad |= kErrBadLength, ctx = ctx < 0 ? 0 : capacity;
  for (int t = tid; t < len; t += kThreads) {
    s_tok[t] = p.tokens[base + t];
    s_par[t] = p.parents[base + t];
    s_want[t] = p.sampled[base + t];
  }
  __syncthreads();
  if (tid < 32) {
    int count = 0, cur = len > 0 ? 0 : -1;
    while (cur >= 0) {
      if (lane == 0) s_path[count] = cur;
      ++count;
      const int want = s_want[cur];
      int next = -1;
      for (int t0 = cur + 1; t0 < len && next < 0; t0 += 32) {
        const int t = t0 + lane;
        const unsigned hit = __ballot_sync(DC_FULL_MASK, t < len && s_par[t] == cur && s_tok[t] == want);
        if (hit) next = t0 + __ffs(hit) - 1;
      }
      cur = next;  // a child is a later node: at most len steps
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  if (layer == 0) {
    for (int t = tid; t < p.T; t += kThreads) p.path[base + t] = t < count ? s_path[t] : -1;
    if (tid == 0) {
      p.accept_len[n] = count > 0 ? count - 1 : 0;
      p.next_token[n] = count > 0 ? s_want[s_path[count - 1]] : -1;
      p.new_len[n] = ctx + count;
    }
  }
  const int vecs = p.head_dim / 8, row = p.kv_heads * vecs;  // 16-byte vectors of a head, of a token
  const uint16_t *kn = p.k_new + layer * p.kn_sl + n * p.kn_sn, *vn = p.v_new + layer * p.vn_sl + n * p.vn_sn;
  uint16_t *kc = p.k_cache + layer * p.kc_sl, *vc = p.v_cache + layer * p.vc_sl;
  for (int i = tid; i < count * row; i += kThreads) {
    const int a = i / row, r = i - a * row, h = r / vecs, e = (r - h * vecs) * 8;
    const int pos = ctx + a, t = s_path[a];
    if (pos >= capacity) {
      bad |= kErrBadPage;
      continue;
    }
    const int page = p.page_table[n * p.pt_stride + (pos >> p.page_shift)];
    if (page < 0 || page >= p.num_pages) {
      bad |= kErrBadPage;
      continue;
    }
    const int slot = pos & ((1 << p.page_shift) - 1);
    const uint4 kv = *reinterpret_cast<const uint4 *>(kn + t * p.kn_st + h * p.kn_sh + e);
    const uint4 vv = *reinterpret_cast<const uint4 *>(vn + t * p.vn_st + h * p.vn_sh + e);
    *reinterpret_cast<uint4 *>(kc + page * p.kc_sp + slot * p.kc_st + h * p.kc_sh + e) = kv;
    *reinterpret_cast<uint4 *>(vc + page * p.vc_sp + slot * p.vc_st + h * p.vc_sh + e) = vv;
  }
  if (bad) atomicOr(p.err, bad);
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitParams &p, cudaStream_t st) {
  k_tree_commit<<<dim3(p.N, p.layers), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dc
