// tree_attn.cu -- attention of a drafted tree's nodes over a paged K/V cache
// and the tree itself.
//
//   out_i = sum_j e^{s_ij - m_i} v_j / sum_j e^{s_ij - m_i},  s_ij = scale q_i.k_j,
// over the context (every token before the tree) and the nodes that the mask
// shows to node i.
//
// All T * group query rows of a K/V head share that head's K and V, so a tile
// of up to 128 of them is the M of two tensor-core products over each tile of
// 128 tokens: S = Q K^T (both from shared memory, accumulated in TMEM) and
// O += P V with P = e^{S - m} rounded to the inputs' type and kept in
// TMEM.  K and V arrive by TMA, a page's tokens a copy, and are read
// once; the running maximum and sum stay in the registers of the thread that
// owns the row.  The running output is rescaled only when a row's maximum has
// grown by more than 2^8 since the last time (the weights stay below 2^8,
// their relative rounding is the same), which keeps it in TMEM nearly always.
//
// The tiles of a request (context first, then the tree) are cut into chunks,
// by a rule on the handle's sizes and the request's own length, so that a
// result does not depend on the batch.  A unit is a (request, K/V head, row
// tile, chunk); a persistent block an SM takes every gridDim-th unit, and its
// products run on across unit borders.  Where a request has several chunks,
// each leaves its unnormalised output with its maximum and sum, and the last
// to finish joins them in chunk order.
//
// Roles: warps 0-3 softmax and output (thread = row = TMEM lane), warp 4 TMA,
// warp 5 the tensor core.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace dc {
namespace {

using namespace tc;

constexpr float kLn2 = 0.693147180559945f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTile = kTreeTile;      // tokens of a K/V tile
constexpr int kSoftWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + 2);
constexpr float kRescale = 8.f;       // log2 growth of a row's maximum before the output is rescaled

template <int D>
struct Geom {
  static constexpr int kHalves = D / 64;                 // 64-element column blocks (128 bytes, one swizzle span)
  static constexpr uint32_t kHalfBytes = kTile * 128;    // a tile's column block
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  static constexpr int kNK = D == 128 ? 2 : 4, kNV = D == 128 ? 3 : 4;  // K and V stages
  static constexpr uint32_t kQ = 0, kK = 2 * kTileBytes, kV = kK + kNK * kTileBytes;
  static constexpr uint32_t kSmem = kV + kNV * kTileBytes;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool F16>
__device__ __forceinline__ float unpack_lo(uint32_t w) {
  if constexpr (F16) return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
  else return __uint_as_float(w << 16);
}
// Whether either 16-bit element of w is an infinity or NaN.
template <bool F16>
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return (w & e) == e || ((w >> 16) & e) == e;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// D[tmem] += A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of a V tile as the B operand with its rows (tokens) along K and
// its columns along N (N-major, 128-byte swizzle): 8-token groups 1024 bytes
// apart, 64-column blocks kHalfBytes apart.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((kTile * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// ---------------------------------------------------------------- units
struct Unit {
  int n, h, mt, chunk, nchunks;  // request, K/V head, row tile, chunk of the request's nchunks
  int ctx, len;                  // clamped lengths
  int tile0, ntiles, nctx;       // first tile, tiles (0: no live rows), context tiles of the request
};

// Every gridDim-th unit in the order (request, chunk, head, row tile), warp
// by warp without communication: 32 requests' lengths at a time in the lanes.
struct UnitIter {
  const TreeAttnParams &p;
  int lane, base = 0, n0 = 0, u;
  int ctx = 0, len = 0, chunks = 0, before = 0, upto = 0, window = 0;
  __device__ UnitIter(const TreeAttnParams &p_, bool flag) : p(p_), lane(threadIdx.x & 31), u(blockIdx.x) { load(flag); }
  __device__ void load(bool flag) {
    const int n = n0 + lane;
    chunks = 0;
    if (n < p.N) {
      const int capacity = p.max_pages << p.page_shift;
      ctx = p.ctx_len[n];
      len = p.tree_len ? p.tree_len[n] : p.T;
      if ((ctx < 0 || ctx > capacity || len < 0 || len > p.T) && flag) atomicOr(p.err, kErrBadLength);
      ctx = min(max(ctx, 0), capacity);
      len = len < 0 ? 0 : min(len, p.T);
      const int nt = len > 0 ? (ctx + kTile - 1) / kTile + (len + kTile - 1) / kTile : 0;
      const int per = tree_chunk_tiles(nt, p.items, p.sms, p.chunk_cap);
      chunks = nt > 0 ? (nt + per - 1) / per : 1;
    }
    const int count = chunks * p.kv_heads * p.mtiles;
    int s = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(DC_FULL_MASK, s, o);
      if (lane >= o) s += y;
    }
    upto = s;
    before = s - count;
    window = __shfl_sync(DC_FULL_MASK, s, 31);
  }
  __device__ bool next(Unit &w, bool flag = false) {
    while (u - base >= window) {
      base += window;
      n0 += 32;
      if (n0 >= p.N) return false;
      load(flag);
    }
    const int rel = u - base;
    const int src = __ffs(__ballot_sync(DC_FULL_MASK, upto > rel)) - 1;
    int i = rel - __shfl_sync(DC_FULL_MASK, before, src);
    w.n = n0 + src;
    w.ctx = __shfl_sync(DC_FULL_MASK, ctx, src);
    w.len = __shfl_sync(DC_FULL_MASK, len, src);
    w.nchunks = __shfl_sync(DC_FULL_MASK, chunks, src);
    w.mt = i % p.mtiles, i /= p.mtiles;
    w.h = i % p.kv_heads, w.chunk = i / p.kv_heads;
    w.nctx = (w.ctx + kTile - 1) / kTile;
    const int nt = w.mt * p.tile_nodes < w.len ? w.nctx + (w.len + kTile - 1) / kTile : 0;
    w.tile0 = (int)((int64_t)nt * w.chunk / w.nchunks);  // chunks as even as they come
    w.ntiles = (int)((int64_t)nt * (w.chunk + 1) / w.nchunks) - w.tile0;
    u += gridDim.x;
    return true;
  }
};

struct Bars {
  unsigned long long q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4], v_empty[4];
  unsigned long long s_full[2], p_full[2], pv_done[2], o_free, soft, done;
};

// TMEM columns: S of even and odd tiles, O, P of even and odd tiles.
constexpr uint32_t kS = 0, kO = 256, kP = 384;

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
k_tree_attn(const TreeAttnParams p, const __grid_constant__ TreeAttnMaps maps) {
  using G = Geom<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) Bars b;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last;
  __shared__ uint32_t s_odd[4];  // tree tile: nodes whose V holds an infinity or NaN
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b.q_full[i]), 1);
      mbar_init(smem_u32(&b.q_empty[i]), 1);
      mbar_init(smem_u32(&b.s_full[i]), 1);
      mbar_init(smem_u32(&b.p_full[i]), kSoftWarps);
      mbar_init(smem_u32(&b.pv_done[i]), 1);
    }
    for (int i = 0; i < G::kNK; ++i) mbar_init(smem_u32(&b.k_full[i]), 1), mbar_init(smem_u32(&b.k_empty[i]), 1);
    for (int i = 0; i < G::kNV; ++i) mbar_init(smem_u32(&b.v_full[i]), 1), mbar_init(smem_u32(&b.v_empty[i]), 1);
    mbar_init(smem_u32(&b.o_free), kSoftWarps);
    mbar_init(smem_u32(&b.soft), kSoftWarps);
    mbar_init(smem_u32(&b.done), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSoftWarps + 1) tmem_alloc(smem_u32(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  int g = 0, live = 0;  // tiles and units with tiles that this role has begun

  if (warp == kSoftWarps) {
    // ------------------------------------------------------------ TMA
    UnitIter it(p, blockIdx.x == 0);
    Unit w;
    const int page_size = 1 << p.page_shift;
    const int box = min(page_size, kTile);       // tokens of one copy
    const int boxes = kTile / box;               // copies of a tile's column block
    bool ok = true;
    while (ok && it.next(w, blockIdx.x == 0)) {
      if (w.ntiles == 0) continue;
      const int qb = live & 1;
      if (live >= 2) ok = mbar_wait(smem_u32(&b.q_empty[qb]), ((live >> 1) - 1) & 1, &s_abort, p.err);
      ok = __all_sync(DC_FULL_MASK, ok);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&b.q_full[qb]), (uint32_t)(G::kHalves * p.tile_nodes * p.group * 128));
        for (int c = 0; c < G::kHalves; ++c)
          tma_load_4d(sbase + G::kQ + qb * G::kTileBytes + c * G::kHalfBytes, &maps.q, c * 64, w.h * p.group,
                      w.mt * p.tile_nodes, w.n, smem_u32(&b.q_full[qb]));
      }
      ++live;
      for (int i = 0; ok && i < w.ntiles; ++i, ++g) {
        const int tile = w.tile0 + i;
        const bool tree = tile >= w.nctx;
        // this lane's copy: column block lane / boxes, tokens lane % boxes
        const int tok0 = (tree ? tile - w.nctx : tile) * kTile;
        const int c = lane / boxes, r = lane % boxes;
        int page = 0, used = boxes;
        if (!tree) {
          used = min(boxes, (w.ctx - tok0 + box - 1) / box);
          if (r < used && c < G::kHalves) {
            page = __ldg(p.page_table + w.n * p.pt_stride + ((tok0 + r * box) >> p.page_shift));
            if (page < 0 || page >= p.num_pages) {
              atomicOr(p.err, kErrBadPage);
              page = 0;
            }
          }
        }
        const uint32_t bytes = tree ? (uint32_t)(G::kHalves * p.tree_box * 128) : (uint32_t)(G::kHalves * used * box * 128);
        const bool mine = tree ? lane < G::kHalves : (c < G::kHalves && r < used);
        auto copy = [&](uint32_t dst, uint32_t bar, const CUtensorMap *cache, const CUtensorMap *fresh) {
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (!mine) return;
          if (tree) tma_load_4d(dst + lane * G::kHalfBytes, fresh, lane * 64, tok0, w.h, w.n, bar);
          else tma_load_4d(dst + c * G::kHalfBytes + r * box * 128, cache, c * 64, tok0 & (page_size - 1), w.h, page, bar);
        };
        const int ks = g % G::kNK, vs = g % G::kNV;
        if (g >= G::kNK) ok = mbar_wait(smem_u32(&b.k_empty[ks]), (g / G::kNK - 1) & 1, &s_abort, p.err);
        ok = __all_sync(DC_FULL_MASK, ok);
        if (!ok) break;
        copy(sbase + G::kK + ks * G::kTileBytes, smem_u32(&b.k_full[ks]), &maps.k_cache, &maps.k_new);
        if (g >= G::kNV) ok = mbar_wait(smem_u32(&b.v_empty[vs]), (g / G::kNV - 1) & 1, &s_abort, p.err);
        ok = __all_sync(DC_FULL_MASK, ok);
        if (!ok) {
          if (lane == 0) mbar_drain(smem_u32(&b.k_full[ks]), (g / G::kNK) & 1);
          break;
        }
        copy(sbase + G::kV + vs * G::kTileBytes, smem_u32(&b.v_full[vs]), &maps.v_cache, &maps.v_new);
      }
    }
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------------------ tensor core
    constexpr uint32_t kIdS = F16 ? idesc_f16(128, kTile) : idesc_bf16(128, kTile);
    constexpr uint32_t kIdO = (F16 ? idesc_f16(128, D) : idesc_bf16(128, D)) | (1u << 16);  // B is N-major
    UnitIter it(p, false);
    Unit w;
    bool ok = true;
    // O (+)= P V of tile t, the first of the block's unit number `unit` if `first`
    auto pv = [&](int t, bool first, int unit) {
      const int vs = t % G::kNV;
      if (!mbar_wait(smem_u32(&b.v_full[vs]), (t / G::kNV) & 1, &s_abort, p.err) ||
          (first && unit > 0 && !mbar_wait(smem_u32(&b.o_free), (unit - 1) & 1, &s_abort, p.err)) ||
          !mbar_wait(smem_u32(&b.p_full[t & 1]), (t >> 1) & 1, &s_abort, p.err))
        return false;
      tc_fence_after();
      const uint32_t sv = sbase + G::kV + vs * G::kTileBytes;
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_ts(tmem + kO, tmem + kP + (t & 1) * 64 + k * 8, v_desc(sv + k * 2048), kIdO, (!first || k > 0) ? 1u : 0u);
      mma_commit(smem_u32(&b.v_empty[vs]));
      mma_commit(smem_u32(&b.pv_done[t & 1]));
      return true;
    };
    bool prev_first = false;
    int prev_unit = 0;
    while (__all_sync(DC_FULL_MASK, ok) && it.next(w)) {
      if (w.ntiles == 0) continue;
      if (lane == 0) {
        const int qb = live & 1;
        ok = mbar_wait(smem_u32(&b.q_full[qb]), (live >> 1) & 1, &s_abort, p.err);
        for (int i = 0; ok && i < w.ntiles; ++i, ++g) {
          const int ks = g % G::kNK;
          ok = mbar_wait(smem_u32(&b.k_full[ks]), (g / G::kNK) & 1, &s_abort, p.err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sq = sbase + G::kQ + qb * G::kTileBytes, sk = sbase + G::kK + ks * G::kTileBytes;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * G::kHalfBytes + (k & 3) * 32;
            mma_bf16(tmem + kS + (g & 1) * 128, sw128_desc(sq + off), sw128_desc(sk + off), kIdS, k > 0 ? 1u : 0u);
          }
          mma_commit(smem_u32(&b.s_full[g & 1]));
          mma_commit(smem_u32(&b.k_empty[ks]));
          if (i == w.ntiles - 1) mma_commit(smem_u32(&b.q_empty[qb]));
          if (g > 0) ok = pv(g - 1, prev_first, prev_unit);
          prev_first = i == 0, prev_unit = live;
        }
      }
      ++live;
    }
    if (lane == 0) {
      if (ok && g > 0) pv(g - 1, prev_first, prev_unit);
      mma_commit(smem_u32(&b.done));  // nothing is in flight when the block frees its TMEM
      mbar_drain(smem_u32(&b.done), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, output
    UnitIter it(p, false);
    Unit w;
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const int row = tid;                          // row of the tile: node row / group, head row % group
    const int rnode = row / p.group, rhead = row - rnode * p.group;
    const bool used = row < p.tile_rows;
    float c = p.scale * kLog2e;
    const bool flip = c < 0.f, zero = c == 0.f;
    c = zero ? 1.f : fabsf(c);
    int syncs = 0;
    bool ok = true;
    // the four warps meet (a bounded wait, unlike bar.sync: a warp that gave up does not come)
    auto meet = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&b.soft));
      const bool met = mbar_wait(smem_u32(&b.soft), syncs++ & 1, &s_abort, p.err);
      return (bool)__all_sync(DC_FULL_MASK, met);
    };
    while (ok && it.next(w)) {
      const int node = w.mt * p.tile_nodes + rnode;
      const bool mine = used && node < p.T;       // a row of the output
      const bool live_row = mine && node < w.len;
      float mref = -INFINITY, l = 0.f;            // reference (log2 units) and sum of this row
      uint32_t odd[8] = {0, 0, 0, 0, 0, 0, 0, 0};  // seen nodes with an infinity or NaN in V
      bool any_odd = false;
      for (int i = 0; i < w.ntiles; ++i, ++g) {
        const int tile = w.tile0 + i;
        const bool tree = tile >= w.nctx;
        const int tok0 = (tree ? tile - w.nctx : tile) * kTile;
        const int valid = min(kTile, (tree ? w.len : w.ctx) - tok0);
        ok = mbar_wait(smem_u32(&b.s_full[g & 1]), (g >> 1) & 1, &s_abort, p.err);
        if (valid < kTile || tree) {
          // V rows past the end hold what a page or a copy left there: zeros
          // in their place, since a zero weight does not cancel an infinity
          ok = ok && mbar_wait(smem_u32(&b.v_full[g % G::kNV]), (g / G::kNV) & 1, &s_abort, p.err);
          ok = __all_sync(DC_FULL_MASK, ok);
          if (!ok) break;
          const uint32_t sv = G::kV + (g % G::kNV) * G::kTileBytes + row * 128;  // token `row`
          bool bad = false;
          if (row >= valid) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
              *reinterpret_cast<uint4 *>(smem + sv + (e >> 3) * G::kHalfBytes + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          } else if (tree) {
            // a node's infinities and NaN stay out of the product (they would
            // reach nodes that do not see it) and are added at the end
            for (int e = 0; e < D / 8; ++e) {
              uint4 *v = reinterpret_cast<uint4 *>(smem + sv + (e >> 3) * G::kHalfBytes + (e & 7) * 16);
              const uint4 x = *v;
              uint32_t xs[4] = {x.x, x.y, x.z, x.w};
              bool any = false;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (nonfinite2<F16>(xs[k])) {
                  if (nonfinite2<F16>(xs[k] & 0xFFFFu)) xs[k] &= 0xFFFF0000u;
                  if (nonfinite2<F16>(xs[k] >> 16)) xs[k] &= 0xFFFFu;
                  any = true;
                }
              if (any) *v = make_uint4(xs[0], xs[1], xs[2], xs[3]);
              bad |= any;
            }
          }
          if (tree) {
            const uint32_t bits = __ballot_sync(DC_FULL_MASK, bad);
            ok = meet();  // the previous tree tile's bits have been read
            if (lane == 0) s_odd[warp] = bits;
            ok = ok && meet();
          }
          fence_proxy_async();
        }
        if (g >= 2)  // P's columns are free
          ok = ok && mbar_wait(smem_u32(&b.pv_done[g & 1]), ((g >> 1) - 1) & 1, &s_abort, p.err);
        ok = __all_sync(DC_FULL_MASK, ok);
        if (!ok) break;
        tc_fence_after();
        float v[kTile];
        const uint32_t ts = trow + kS + (g & 1) * 128, tp = trow + kP + (g & 1) * 64;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[32];
          tmem_ld32(ts + q * 32, x);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[q * 32 + k] = x[k];
        }
        if (flip | zero) {
#pragma unroll
          for (int k = 0; k < kTile; ++k) v[k] = zero ? 0.f : -v[k];
        }
        if (valid < kTile || tree) {
          uint32_t see[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int left = valid - q * 32;  // tokens of this word that exist
            see[q] = left >= 32 ? 0xFFFFFFFFu : left > 0 ? (1u << left) - 1u : 0u;
          }
          if (tree) {
            const int words = (p.T + 31) / 32, w0 = tok0 / 32;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t m = 0;
              if (live_row && w0 + q < words) {
                if (p.tree_mask) {
                  m = (uint32_t)__ldg(p.tree_mask + w.n * p.mask_sn + (int64_t)node * words + w0 + q);
                } else {
                  const int left = node + 1 - (w0 + q) * 32;  // nodes 0..node
                  m = left >= 32 ? 0xFFFFFFFFu : left > 0 ? (1u << left) - 1u : 0u;
                }
              }
              see[q] &= m;
              const uint32_t o = see[q] & s_odd[q];
              if (tok0 == 0) odd[q] = o;
              else odd[4 + q] = o;
              any_odd |= o != 0;
            }
          }
#pragma unroll
          for (int k = 0; k < kTile; ++k) v[k] = (see[k >> 5] >> (k & 31)) & 1u ? v[k] : -INFINITY;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < kTile; ++k) m4[k & 3] = fmaxf(m4[k & 3], v[k]);
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
        if (i == 0) {
          mref = mt;
        } else {
          const bool grow = mt > mref + kRescale;  // from -inf: any finite maximum
          if (__any_sync(DC_FULL_MASK, grow)) {
            const float f = grow ? ex2(mref - mt) : 1.f;
            if (grow) mref = mt, l *= f;
            ok = mbar_wait(smem_u32(&b.pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, &s_abort, p.err);
            ok = __all_sync(DC_FULL_MASK, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float x[32];
              uint32_t y[32];
              tmem_ld32(trow + kO + q * 32, x);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(x[k] * f);
              tmem_st32(trow + kO + q * 32, y);
            }
            tmem_st_wait();
          }
        }
        const float mb = mref == -INFINITY ? 0.f : mref;
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t y[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float a = ex2(fmaf(v[q * 64 + 2 * k], c, -mb)), d = ex2(fmaf(v[q * 64 + 2 * k + 1], c, -mb));
            l4[(2 * k) & 3] += a;
            l4[(2 * k + 1) & 3] += d;
            y[k] = pack2<F16>(a, d);
          }
          tmem_st32(tp + q * 32, y);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&b.p_full[g & 1]));
      }
      if (!ok) break;
      // -------------------------------------------------------- the unit's output
      const int64_t orow = ((int64_t)w.n * p.T + node) * (p.kv_heads * p.group) + w.h * p.group + rhead;
      uint32_t *out = reinterpret_cast<uint32_t *>(p.out + orow * D);
      auto add_odd = [&](float (&x)[32], int d0) {  // infinities and NaN of the seen nodes
#pragma unroll 1
        for (int q = 0; q < 8; ++q)
          for (uint32_t r = odd[q]; r; r &= r - 1) {
            const uint16_t *vn = p.v_new + w.n * p.vn_sn + (q * 32 + __ffs(r) - 1) * p.vn_st + w.h * p.vn_sh;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t e = vn[d0 + k];
              if (nonfinite2<F16>(e)) x[k] += unpack_lo<F16>(e);
            }
          }
      };
      if (w.ntiles > 0) {
        ok = mbar_wait(smem_u32(&b.pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, &s_abort, p.err);
        ok = __all_sync(DC_FULL_MASK, ok);
        if (!ok) break;
        tc_fence_after();
      }
      if (w.nchunks == 1 || w.ntiles == 0) {
        // whole: normalise and write.  (A unit without tiles has no live row;
        // its first chunk writes the zeros.)
        if (w.chunk == 0 || w.ntiles > 0) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            float x[32];
            if (w.ntiles > 0) {
              tmem_ld32(trow + kO + q * 32, x);
              if (any_odd) add_odd(x, q * 32);
            }
            if (mine) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint4 y = make_uint4(0, 0, 0, 0);
                if (live_row && l != 0.f)
                  y = make_uint4(pack2<F16>(x[8 * k] * inv, x[8 * k + 1] * inv), pack2<F16>(x[8 * k + 2] * inv, x[8 * k + 3] * inv),
                                 pack2<F16>(x[8 * k + 4] * inv, x[8 * k + 5] * inv), pack2<F16>(x[8 * k + 6] * inv, x[8 * k + 7] * inv));
                reinterpret_cast<uint4 *>(out)[q * 4 + k] = y;
              }
            }
            __syncwarp();
          }
          if (mine && p.lse) p.lse[orow] = live_row && l != 0.f ? (mref + __log2f(l)) * kLn2 : -INFINITY;
        }
      } else {
        const int64_t item = ((int64_t)w.n * p.kv_heads + w.h) * p.mtiles + w.mt;
        const int R = p.tile_rows;
        float4 *part = p.part_o + (item * p.max_chunks + w.chunk) * (D / 4) * R;  // [D / 4][rows]: rows adjacent
        float2 *ml = p.part_ml + item * p.max_chunks * R;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          float x[32];
          tmem_ld32(trow + kO + q * 32, x);
          if (any_odd) add_odd(x, q * 32);
          if (used) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              part[(q * 8 + k) * R + row] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
          __syncwarp();
        }
        if (used) ml[w.chunk * R + row] = make_float2(mref, l);
        __threadfence();
        ok = meet();
        if (!ok) break;
        if (tid == 0) s_last = atomicAdd(&p.counts[item], 1) == w.nchunks - 1;
        ok = meet();
        if (!ok) break;
        if (s_last) {
          __threadfence();
          if (tid == 0) p.counts[item] = 0;
          if (mine) {
            float M = -INFINITY, L = 0.f;
            for (int k = 0; k < w.nchunks; ++k) M = fmaxf(M, __ldcg(&ml[k * R + row]).x);
            auto weight = [&](int k) {
              const float2 a = __ldcg(&ml[k * R + row]);
              return a.x == -INFINITY && a.y == 0.f ? 0.f : ex2(a.x - M);
            };
            for (int k = 0; k < w.nchunks; ++k) L = fmaf(weight(k), __ldcg(&ml[k * R + row]).y, L);
            const bool some = live_row && L != 0.f;
            const float inv = some ? 1.f / L : 0.f;
            const float4 *po = p.part_o + item * p.max_chunks * (D / 4) * R + row;
#pragma unroll 1
            for (int d = 0; d < D / 4; d += 8) {
              float4 acc[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
              for (int k = 0; some && k < w.nchunks; ++k) {
                const float f = weight(k);
                if (f == 0.f) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 o = __ldcg(po + ((int64_t)k * (D / 4) + d + e) * R);
                  acc[e].x = fmaf(f, o.x, acc[e].x), acc[e].y = fmaf(f, o.y, acc[e].y);
                  acc[e].z = fmaf(f, o.z, acc[e].z), acc[e].w = fmaf(f, o.w, acc[e].w);
                }
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 a = acc[2 * e], d2 = acc[2 * e + 1];
                reinterpret_cast<uint4 *>(out)[d / 2 + e] =
                    make_uint4(pack2<F16>(a.x * inv, a.y * inv), pack2<F16>(a.z * inv, a.w * inv),
                               pack2<F16>(d2.x * inv, d2.y * inv), pack2<F16>(d2.z * inv, d2.w * inv));
              }
            }
            if (p.lse) p.lse[orow] = some ? (M + __log2f(L)) * kLn2 : -INFINITY;
          }
        }
      }
      if (w.ntiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&b.o_free));
        ++live;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_abort && tid == kSoftWarps * 32) {  // copies in flight land before the block gives its memory back
    for (int t = max(0, g - 4); t < g; ++t) {
      if (t >= g - G::kNK) mbar_drain(smem_u32(&b.k_full[t % G::kNK]), (t / G::kNK) & 1);
      if (t >= g - G::kNV) mbar_drain(smem_u32(&b.v_full[t % G::kNV]), (t / G::kNV) & 1);
    }
    for (int t = max(0, live - 2); t < live; ++t) mbar_drain(smem_u32(&b.q_full[t & 1]), (t >> 1) & 1);
  }
  if (warp == kSoftWarps + 1) tmem_dealloc(tmem, 512);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A 4D map (column, a, b, c) with element strides of a, b, c and a box of 64
// columns, box_a, box_b, 1.  The stride of an axis of one entry is never
// used; the encoder wants a multiple of 16 bytes there too.
bool encode_4d(CUtensorMap *map, bool f16, const void *base, int D, int na, int64_t sa, int nb, int64_t sb, int nc,
               int64_t sc, int box_a, int box_b) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const auto bytes = [&](int n, int64_t s) { return (cuuint64_t)(n > 1 ? s * 2 : D * 2); };
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)na, (cuuint64_t)nb, (cuuint64_t)nc};
  const cuuint64_t strides[3] = {bytes(na, sa), bytes(nb, sb), bytes(nc, sc)};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_a, (cuuint32_t)box_b, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F16>
cudaError_t launch(const TreeAttnParams &p, const TreeAttnMaps &maps, cudaStream_t st) {
  const size_t smem = Geom<D>::kSmem + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(k_tree_attn<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)p.N * p.kv_heads * p.mtiles * p.max_chunks;
  k_tree_attn<D, F16><<<(unsigned)(most < p.sms ? most : p.sms), kThreads, smem, st>>>(p, maps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attention(const TreeAttnParams &p, cudaStream_t st) {
  TreeAttnMaps maps;
  const int page = 1 << p.page_shift, box = page < kTile ? page : kTile, heads = p.kv_heads, D = p.head_dim;
  if (!encode_4d(&maps.q, p.f16, p.q, D, heads * p.group, p.q_sh, p.T, p.q_st, p.N, p.q_sn, p.group, p.tile_nodes) ||
      !encode_4d(&maps.k_new, p.f16, p.k_new, D, p.T, p.kn_st, heads, p.kn_sh, p.N, p.kn_sn, p.tree_box, 1) ||
      !encode_4d(&maps.v_new, p.f16, p.v_new, D, p.T, p.vn_st, heads, p.vn_sh, p.N, p.vn_sn, p.tree_box, 1) ||
      !encode_4d(&maps.k_cache, p.f16, p.k_cache, D, page, p.kc_st, heads, p.kc_sh, p.num_pages, p.kc_sp, box, 1) ||
      !encode_4d(&maps.v_cache, p.f16, p.v_cache, D, page, p.vc_st, heads, p.vc_sh, p.num_pages, p.vc_sp, box, 1))
    return cudaErrorInvalidValue;
  if (p.head_dim == 128)
    return p.f16 ? launch<128, true>(p, maps, st) : launch<128, false>(p, maps, st);
  return p.f16 ? launch<64, true>(p, maps, st) : launch<64, false>(p, maps, st);
}

}  // namespace dc
