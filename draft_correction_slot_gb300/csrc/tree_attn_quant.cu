// tree_attn_quant.cu -- attention of a drafted tree over a paged cache held in
// 8 bits.  A warp a query row: its head's elements over the lanes, the tokens
// one after another with a running maximum and sum.
#include "quant.cuh"
#include "tree_attn.cuh"

namespace dc {
namespace {

template <int D>
__global__ void __launch_bounds__(256) k_quant_attn(const QuantAttnParams p) {
  const TreeAttnParams &t = p.t;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, heads = t.kv_heads * t.group;
  const int n = blockIdx.x, of_n = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (of_n >= t.T * heads) return;
  const int node = of_n / heads, hq = of_n - node * heads, h = hq / t.group;
  const int capacity = t.max_pages << t.page_shift;
  int ctx = t.ctx_len[n], len = t.tree_len ? t.tree_len[n] : t.T;
  if ((ctx < 0 || ctx > capacity || len < 0 || len > t.T) && of_n == 0 && lane == 0) atomicOr(t.err, kErrBadLength);
  ctx = min(max(ctx, 0), capacity), len = len < 0 ? 0 : min(len, t.T);
  const auto value = [&](uint32_t w) { return t.f16 ? unpack_lo<true>(w) : unpack_lo<false>(w); };
  float q[E], acc[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = value(t.q[n * t.q_sn + node * t.q_st + hq * t.q_sh + lane * E + e]);
  const auto step = [&](const float (&k)[E], const float (&v)[E]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s) * t.scale * kLog2e;
    const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : ex2(m - top), w = ex2(s - top);
    m = top, l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, w * v[e]);
  };
  for (int j = 0; node < len && j < ctx; ++j) {
    int page = t.page_table[n * t.pt_stride + (j >> t.page_shift)];
    if (page < 0 || page >= t.num_pages) {
      if (lane == 0) atomicOr(t.err, kErrBadPage);
      page = 0;
    }
    const int slot = j & ((1 << t.page_shift) - 1), b = slot >> p.scale_shift;
    const float ks = p.k_scale[page * p.ks_sp + b * p.ks_sb + h * p.ks_sh];
    const float vs = p.v_scale[page * p.vs_sp + b * p.vs_sb + h * p.vs_sh];
    const uint8_t *kp = p.k_cache + page * p.kc_sp + slot * p.kc_st + h * p.kc_sh + lane * E;
    const uint8_t *vp = p.v_cache + page * p.vc_sp + slot * p.vc_st + h * p.vc_sh + lane * E;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) k[e] = from_e4m3x2(kp[e]).x * ks, v[e] = from_e4m3x2(vp[e]).x * vs;
    step(k, v);
  }
  for (int j = 0; node < len && j < len; ++j) {
    if (!((tree_sees(t, n, len, node, j >> 5) >> (j & 31)) & 1u)) continue;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = value(t.k_new[n * t.kn_sn + j * t.kn_st + h * t.kn_sh + lane * E + e]);
      v[e] = value(t.v_new[n * t.vn_sn + j * t.vn_st + h * t.vn_sh + lane * E + e]);
    }
    step(k, v);
  }
  const int64_t orow = (int64_t)n * t.T * heads + of_n;
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t w = t.f16 ? pack2<true>(acc[e] * inv, 0.f) : pack2<false>(acc[e] * inv, 0.f);
    t.out[orow * D + lane * E + e] = (uint16_t)w;
  }
  if (t.lse && lane == 0) t.lse[orow] = l != 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_quant_attention(const QuantAttnParams &p, cudaStream_t st) {
  const int rows = p.t.T * p.t.kv_heads * p.t.group;
  const dim3 grid((unsigned)p.t.N, (unsigned)((rows + 7) / 8));
  if (p.t.head_dim == 128) k_quant_attn<128><<<grid, 256, 0, st>>>(p);
  else k_quant_attn<64><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dc
