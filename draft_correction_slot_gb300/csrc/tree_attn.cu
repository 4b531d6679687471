// tree_attn.cu -- attention of a drafted tree's nodes over a paged K/V cache
// and the tree itself.
//
//   out_i = sum_j e^{s_ij - m_i} v_j / sum_j e^{s_ij - m_i},  s_ij = scale q_i.k_j,
// over the context (every token before the tree) and the nodes that the mask
// shows to node i.  One warp a (request, node, query head): 32 tokens at a
// time, a lane's token each for the scores, then all lanes over the value's
// elements.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace dc {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  } else {
    return make_float2(bf16_bits_to_float(w & 0xFFFFu), bf16_bits_to_float(w >> 16));
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    return bf16_rn_bits(a) | bf16_rn_bits(b) << 16;
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(128) k_tree_attn(const TreeAttnParams p) {
  __shared__ float s_q[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = p.kv_heads * p.group;
  const int64_t item = (int64_t)blockIdx.x * 4 + warp;
  const bool live = item < (int64_t)p.N * p.T * heads;
  const int64_t it = live ? item : 0;
  const int hq = (int)(it % heads), t = (int)(it / heads % p.T), n = (int)(it / heads / p.T), h = hq / p.group;
  constexpr int E = D / 32;  // elements a lane holds
  if (live) {
    const uint16_t *q = p.q + n * p.q_sn + t * p.q_st + hq * p.q_sh;
    for (int e = lane; e < D / 2; e += 32) {
      const float2 f = unpack2<F16>(reinterpret_cast<const uint32_t *>(q)[e]);
      s_q[warp][2 * e] = f.x, s_q[warp][2 * e + 1] = f.y;
    }
  }
  __syncwarp();
  if (!live) return;
  const int capacity = p.max_pages << p.page_shift;
  int len = p.tree_len ? p.tree_len[n] : p.T, ctx = p.ctx_len[n], bad = 0;
  if (len < 0 || len > p.T) bad |= kErrBadLength, len = len < 0 ? 0 : p.T;
  if (ctx < 0 || ctx > capacity) bad |= kErrBadLength, ctx = ctx < 0 ? 0 : capacity;
  const int words = (p.T + 31) / 32;
  const int32_t *mask = p.tree_mask ? p.tree_mask + n * p.mask_sn + t * words : nullptr;
  float m = -INFINITY, l = 0.f, acc[E] = {};
  const int total = t < len ? ctx + len : 0;
  for (int c0 = 0; c0 < total; c0 += 32) {
    const int c = c0 + lane;
    const uint16_t *k = nullptr, *v = nullptr;
    if (c < ctx) {
      const int page = p.page_table[n * p.pt_stride + (c >> p.page_shift)];
      const int slot = c & ((1 << p.page_shift) - 1);
      if (page >= 0 && page < p.num_pages) {
        k = p.k_cache + page * p.kc_sp + slot * p.kc_st + h * p.kc_sh;
        v = p.v_cache + page * p.vc_sp + slot * p.vc_st + h * p.vc_sh;
      } else {
        bad |= kErrBadPage;
      }
    } else if (c < total) {
      const int j = c - ctx;
      if (mask ? (mask[j >> 5] >> (j & 31)) & 1 : j <= t) {
        k = p.k_new + n * p.kn_sn + j * p.kn_st + h * p.kn_sh;
        v = p.v_new + n * p.vn_sn + j * p.vn_st + h * p.vn_sh;
      }
    }
    float s = -INFINITY;
    if (k) {
      s = 0.f;
#pragma unroll 4
      for (int e = 0; e < D; e += 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(k + e);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<F16>(x[i]);
          s = fmaf(s_q[warp][e + 2 * i], f.x, s);
          s = fmaf(s_q[warp][e + 2 * i + 1], f.y, s);
        }
      }
      s *= p.scale;
    }
    const float m_new = fmaxf(m, warp_max(s));
    const unsigned seen = __ballot_sync(DC_FULL_MASK, k != nullptr);
    if (m_new == -INFINITY) {  // nothing seen yet, or scores without a value
      if (__any_sync(DC_FULL_MASK, s != s)) l = NAN;
      continue;
    }
    const float scale_old = exp2f((m - m_new) * kLog2e);
    const float w = k ? exp2f((s - m_new) * kLog2e) : 0.f;
    l = l * scale_old + warp_sum(w);
    m = m_new;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= scale_old;
    for (unsigned rest = seen; rest; rest &= rest - 1) {
      const int src = __ffs(rest) - 1;
      const uint16_t *vj = reinterpret_cast<const uint16_t *>(
          __shfl_sync(DC_FULL_MASK, reinterpret_cast<unsigned long long>(v), src));
      const float wj = __shfl_sync(DC_FULL_MASK, w, src);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float2 f = unpack2<F16>(reinterpret_cast<const uint32_t *>(vj)[lane * (E / 2) + e]);
        acc[2 * e] = fmaf(wj, f.x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(wj, f.y, acc[2 * e + 1]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t *out = reinterpret_cast<uint32_t *>(p.out + it * D);
#pragma unroll
  for (int e = 0; e < E / 2; ++e)
    out[lane * (E / 2) + e] = pack2<F16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (p.lse && lane == 0) p.lse[it] = l == 0.f ? -INFINITY : m + logf(l);
  if (bad) atomicOr(p.err, bad);
}

}  // namespace

cudaError_t launch_tree_attention(const TreeAttnParams &p, cudaStream_t st) {
  const int64_t items = (int64_t)p.N * p.T * p.kv_heads * p.group;
  const unsigned grid = (unsigned)((items + 3) / 4);
  if (p.head_dim == 128) {
    if (p.f16) k_tree_attn<128, true><<<grid, 128, 0, st>>>(p);
    else k_tree_attn<128, false><<<grid, 128, 0, st>>>(p);
  } else {
    if (p.f16) k_tree_attn<64, true><<<grid, 128, 0, st>>>(p);
    else k_tree_attn<64, false><<<grid, 128, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace dc
