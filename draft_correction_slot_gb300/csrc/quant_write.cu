// quant_write.cu -- tokens' K/V into a paged cache held in 8 bits: the accepted
// path of a drafted tree, and ragged prompts.
//
// A block of `1 << scale_shift` tokens of a K/V head shares the scale s.  With
// `a` the largest finite magnitude of the new tokens' elements in the block and
// need(a) the least power of two with a <= 448 need:
//   s = need (no token of the block committed before), else max(s0, need)
//   new payload rn(x / s);  committed payload y: rn(y s0 / s) where s > s0.
//
// A warp has a block: 16 bytes of a token a lane, so 32 / (D / 8) tokens a step, four
// (append) or eight (commit) steps in flight.  What fits in these stays in registers
// between the maximum and the rounding; longer blocks are read again (from L1 or L2).
// Nothing is shared between warps, so a request's result depends on its own
// tokens alone.
// Append: 8 prompts of up to 2000 tokens, 16 layers x 8 heads of 64, blocks of 64: 138 us (132 to
// 174 by the draw of the lengths), 3.5 TB/s of the 6.8 that a copy reaches; bound by the chain lengths,
// page, tokens, maximum, rounding of each warp.  Commit: 32 trees of 64 nodes, 16 layers: 18 us with
// its call, bound by latency as tree_commit.cu's.
#include "kernels.h"
#include "quant.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxNodes = 256;
constexpr int kTailBlocks = 8;  // see k_quant_append
constexpr int kAppendSteps = 4;  // 8 prompts of up to 2000 tokens, mean of six draws: 156 us; 175 with 8 steps, 220 with 16 (fewer warps an SM)

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}

// One block's `count` new tokens, the first at place `old` of the block; row(i)
// is the i-th one's source.  dst: the block's first token in the cache.
template <int D, bool F16, int kSteps, class Row>
__device__ __forceinline__ void write_block(int old, int count, Row row, uint8_t *dst, int64_t stride,
                                            float *scale) {
  constexpr int per = D / 8, step = 32 / per;
  const int lane = threadIdx.x & 31, sub = lane / per, e = lane % per * 8;
  uint4 w[kSteps];
  float most = 0.f, odd = 0.f;  // (odd becomes NaN with an infinity or NaN)
  for (int i0 = 0; i0 < count; i0 += step * kSteps) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = i0 + k * step + sub;
      w[k] = i < count ? __ldg(reinterpret_cast<const uint4 *>(row(i) + e)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (i0 + k * step >= count) break;
      float x[8];
      unpack8<F16>(w[k], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) odd = fmaf(x[j], 0.f, odd), most = fmaxf(most, fabsf(x[j]));
    }
  }
  const bool finite = !__any_sync(DC_FULL_MASK, odd != odd);
  if (!finite) {  // rare: once more over what does count
    most = 0.f;
    for (int i = sub; i < count; i += step) {
      float x[8];
      unpack8<F16>(__ldg(reinterpret_cast<const uint4 *>(row(i) + e)), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]) < INFINITY ? fabsf(x[j]) : 0.f);
    }
  }
  most = warp_max(most);
  const float need = least_scale(most), was = old > 0 ? *scale : need, s = fmaxf(was, need);
  __syncwarp();  // every lane has read the scale
  if (lane == 0 && (old == 0 || s != was)) *scale = s;
  if (s != was) {  // (only with tokens before)
    const float ratio = was / s;
    for (int i = sub; i < old; i += step) {
      uint2 *at = reinterpret_cast<uint2 *>(dst + i * stride + e);
      const uint2 y = *at;
      const uint32_t u[4] = {y.x & 0xFFFFu, y.x >> 16, y.y & 0xFFFFu, y.y >> 16};
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = from_e4m3x2(u[j]);
        r[j] = to_e4m3x2(f.x * ratio, f.y * ratio);
      }
      *at = make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
    }
  }
  // A power of two (any scale that was made here) is divided by exactly by its inverse; divisions
  // of 8 elements took as long as all the rest (8 prompts of up to 2000 tokens: 183 us with them, 169 without).
  const bool power = (__float_as_uint(s) & 0x7FFFFFu) == 0u;
  const float inv = power ? 1.f / s : 1.f;
  const bool kept = count <= step * kSteps;
  for (int i0 = 0; i0 < count; i0 += step * kSteps) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = i0 + k * step + sub;
      if (!kept) w[k] = i < count ? __ldg(reinterpret_cast<const uint4 *>(row(i) + e)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = i0 + k * step + sub;
      if (i0 + k * step >= count) break;
      float x[8];
      unpack8<F16>(w[k], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = power ? x[j] * inv : x[j] / s;
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = finite ? finite_e4m3x2(x[2 * j], x[2 * j + 1]) : to_e4m3x2(x[2 * j], x[2 * j + 1]);
      if (i < count) *reinterpret_cast<uint2 *>(dst + (old + i) * stride + e) = make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
    }
  }
}

// A cache's tensors of one layer, K or V.
struct Side {
  const uint16_t *fresh;
  int64_t st, sh;  // strides of fresh
  uint8_t *cache;
  int64_t cp, ct, ch;
  float *scale;
  int64_t sp, sb, ss;
  __device__ Side(const QuantWriteParams &p, int layer, bool v)
      : fresh(v ? p.v_new + layer * p.vn_sl : p.k_new + layer * p.kn_sl), st(v ? p.vn_st : p.kn_st),
        sh(v ? p.vn_sh : p.kn_sh), cache(v ? p.v_cache + layer * p.vc_sl : p.k_cache + layer * p.kc_sl),
        cp(v ? p.vc_sp : p.kc_sp), ct(v ? p.vc_st : p.kc_st), ch(v ? p.vc_sh : p.kc_sh),
        scale(v ? p.v_scale + layer * p.vs_sl : p.k_scale + layer * p.ks_sl), sp(v ? p.vs_sp : p.ks_sp),
        sb(v ? p.vs_sb : p.ks_sb), ss(v ? p.vs_sh : p.ks_sh) {}
};

// The new tokens of request n in the block of position pos (the first of them)
// up to position `end`; row(i): source of the token at pos + i.  -> error bits
template <int D, bool F16, int kSteps, class Row>
__device__ __forceinline__ int write_at(const QuantWriteParams &p, const Side &a, int n, int h, int pos, int end, Row row) {
  const int block = 1 << p.scale_shift, b0 = pos & ~(block - 1);
  if ((pos >> p.page_shift) >= p.max_pages) return kErrBadPage;
  const int page = __ldg(p.page_table + n * p.pt_stride + (pos >> p.page_shift));
  if (page < 0 || page >= p.num_pages) return kErrBadPage;
  const int slot = b0 & ((1 << p.page_shift) - 1);
  write_block<D, F16, kSteps>(pos - b0, min(end, b0 + block) - pos, row, a.cache + page * a.cp + slot * a.ct + h * a.ch,
              a.ct, a.scale + page * a.sp + (slot >> p.scale_shift) * a.sb + h * a.ss);
  return 0;
}

// One block (of threads) a request, layer and K or V; each walks the tree itself.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) k_quant_commit(const QuantWriteParams p) {
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
  if (layer == 0 && blockIdx.z == 0) {
    for (int t = tid; t < p.T; t += kThreads) p.path[base + t] = t < count ? s_path[t] : -1;
    if (tid == 0) {
      p.accept_len[n] = count > 0 ? count - 1 : 0;
      p.next_token[n] = count > 0 ? s_want[s_path[count - 1]] : -1;
      p.new_len[n] = ctx + count;
    }
  }
  const Side a(p, layer, blockIdx.z);
  const uint16_t *rows = a.fresh + n * (blockIdx.z ? p.vn_sn : p.kn_sn);
  const int first = ctx >> p.scale_shift, blocks = count > 0 ? ((ctx + count - 1) >> p.scale_shift) - first + 1 : 0;
  for (int u = tid >> 5; u < blocks * p.kv_heads; u += kWarps) {
    const int b = u / p.kv_heads, h = u - b * p.kv_heads;
    const int pos = max(ctx, (first + b) << p.scale_shift);
    bad |= write_at<D, F16, 8>(p, a, n, h, pos, ctx + count,
                    [&](int i) { return rows + s_path[pos - ctx + i] * a.st + h * a.sh; });
  }
  if (bad) atomicOr(p.err, bad);
}

// The most blocks of `scale` tokens that requests with rows of their own lie in.
__host__ __device__ inline int64_t append_blocks(const QuantWriteParams &p) {
  return ((int64_t)p.total >> p.scale_shift) + 2ll * p.N;
}

// 32 requests' rows, one a lane: what it has before, its first row, how many rows and blocks of
// tokens, and the blocks up to and with it.  A request with lengths out of range has none.
struct AppendLanes {
  int ctx = 0, row0 = 0, len = 0, blocks = 0, upto = 0, all = 0;
  bool bad = false;
  __device__ AppendLanes(const QuantWriteParams &p, int n) {
    const int lane = threadIdx.x & 31, capacity = p.max_pages << p.page_shift;
    if (n < p.N) {
      ctx = p.ctx_len[n], row0 = p.first[n], len = p.first[n + 1] - row0;
      bad = ctx < 0 || ctx > capacity || row0 < 0 || len < 0 || row0 > p.total || len > p.total - row0 || len > capacity - ctx;
      if (bad) ctx = min(max(ctx, 0), capacity), len = 0;
      if (len > 0) blocks = ((ctx + len - 1) >> p.scale_shift) - (ctx >> p.scale_shift) + 1;
    }
    upto = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(DC_FULL_MASK, upto, o);
      if (lane >= o) upto += y;
    }
    all = __shfl_sync(DC_FULL_MASK, upto, 31);
  }
  // Block b of theirs (of the requests from n0 on), head h.  -> error bits
  template <int D, bool F16>
  __device__ __forceinline__ int write(const QuantWriteParams &p, int n0, int b, int h) const {
    const int src = __ffs(__ballot_sync(DC_FULL_MASK, upto > b)) - 1;
    const int rel = b - __shfl_sync(DC_FULL_MASK, upto - blocks, src);
    const int c = __shfl_sync(DC_FULL_MASK, ctx, src), r = __shfl_sync(DC_FULL_MASK, row0, src);
    const int end = c + __shfl_sync(DC_FULL_MASK, len, src);
    const Side a(p, blockIdx.y >> 1, blockIdx.y & 1);
    const int pos = max(c, ((c >> p.scale_shift) + rel) << p.scale_shift);
    const uint16_t *rows = a.fresh + (int64_t)(r + pos - c) * a.st + h * a.sh;
    return write_at<D, F16, kAppendSteps>(p, a, n0 + src, h, pos, end, [&](int i) { return rows + i * a.st; });
  }
};

// A warp a block of tokens and head; blockIdx.y: the layer's K or V.
// (64 registers a thread: the 80 that it would take leave three blocks an SM; 187 us where 138.)
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 4) k_quant_append(const QuantWriteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), covered = append_blocks(p);
  const int h = (int)(u % p.kv_heads);
  const int64_t b = u / p.kv_heads;  // block of tokens, over all requests
  const bool first_warp = u == 0 && blockIdx.y == 0;
  int64_t base = 0;                  // blocks of the requests before n0
  int bad = 0;
  for (int n0 = 0; n0 < p.N; n0 += 32) {
    const AppendLanes w(p, n0 + lane);
    if (w.bad) bad |= kErrBadLength;
    if (first_warp && n0 + lane < p.N) p.new_len[n0 + lane] = w.ctx + w.len;
    if (b >= base && b < base + w.all && b < covered) {
      bad |= w.write<D, F16>(p, n0, (int)(b - base), h);
      if (!first_warp && b >= kTailBlocks) break;
    }
    base += w.all;
  }
  // Where rows go back (first decreases), requests may share rows and have more blocks than
  // the grid: what lies past it is taken by the warps of the first few, which have seen them all.
  const int tail = (int)min(covered, (int64_t)kTailBlocks);
  if (b < tail && base > covered) {
    base = 0;
    int64_t t = covered + b;
    for (int n0 = 0; n0 < p.N; n0 += 32) {
      const AppendLanes w(p, n0 + lane);
      for (; t < base + w.all; t += tail) bad |= w.write<D, F16>(p, n0, (int)(t - base), h);
      base += w.all;
    }
  }
  if (bad && (first_warp || (bad & kErrBadPage))) atomicOr(p.err, bad);
}

}  // namespace

cudaError_t launch_quant_commit(const QuantWriteParams &p, cudaStream_t st) {
  const auto kernel = p.head_dim == 128 ? (p.f16 ? k_quant_commit<128, true> : k_quant_commit<128, false>)
                                        : (p.f16 ? k_quant_commit<64, true> : k_quant_commit<64, false>);
  kernel<<<dim3(p.N, p.layers, 2), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_quant_append(const QuantWriteParams &p, cudaStream_t st) {
  const auto kernel = p.head_dim == 128 ? (p.f16 ? k_quant_append<128, true> : k_quant_append<128, false>)
                                        : (p.f16 ? k_quant_append<64, true> : k_quant_append<64, false>);
  const int64_t grid = (append_blocks(p) * p.kv_heads + kWarps - 1) / kWarps;
  kernel<<<dim3((unsigned)grid, p.layers * 2), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dc
