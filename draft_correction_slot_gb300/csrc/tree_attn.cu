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
// O += P V with P = e^{S - m} rounded to the inputs' type, over half of S's
// own columns.  K and V arrive by TMA, a page's tokens a copy, and are read
// once a row tile.
//
// Two softmax groups of four warps take the tiles in turn, each with its own
// S, running reference, sum and O, so that one's exponentials run under the
// other's products (one group alone took 2870 cycles a tile, the products
// 1024); at a unit's end their two outputs are weighed together.  A thread
// owns a row: reference and sum stay in its registers.  A tile's weights are
// taken against the reference at hand; only when a score has outgrown it by
// 2^8 the reference is raised, O rescaled and the tile done again (below that
// the weights' relative rounding is the same).
//
// The tiles of a request (context first, then the tree) are cut into chunks,
// by a rule on the handle's sizes and the request's own length, so that a
// result does not depend on the batch.  A unit is a (request, K/V head, row
// tile, chunk); a persistent block an SM takes every gridDim-th unit, and its
// products run on across unit borders.  Each unit leaves its rows'
// unnormalised output with their references and sums, and a second kernel
// joins the chunks.
//
// 8 requests of up to 32000 tokens, 64 nodes x 5 heads: 310 us (floor
// 108, operations).  A pair of tiles takes 3700 cycles, of which the
// exponentials need 2050 (16 a cycle) and the products 2080; from "weights
// stored" to "next scores there" pass 2500, and a unit's border costs some 10,000.
// Half tiles with two S buffers a group took 417 us: a product of 64 columns
// takes as long as one of 128.
//
// Roles: warps 0-7 softmax and output (thread = row = TMEM lane), warp 8 the
// tensor core, warps 9-10 TMA.  After an expired wait the softmax warps run
// their loops to the end without waiting or storing, so that their block
// barriers stay complete.
#include "launch.h"
#include "tma_map.h"
#include "tree_attn.cuh"

namespace dc {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 384;           // three warpgroups; warp 11 only completes the third
// Registers a thread: 168 at launch (65,536 / 384 in steps of 8), then 224 for
// the two softmax warpgroups and 56 for the third: 2 x 224 + 56 = 3 x 168.
constexpr int kSoftRegs = 224, kOtherRegs = 56;

template <int D>
struct Geom {
  static constexpr int kHalves = D / 64;                 // 64-element column blocks (128 bytes, one swizzle span)
  static constexpr uint32_t kHalfBytes = kTile * 128;    // a tile's column block
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  static constexpr int kNK = D == 128 ? 2 : 4, kNV = D == 128 ? 3 : 4;  // K and V stages
  static constexpr uint32_t kQHalf = kHalfBytes, kQBytes = kTileBytes;
  static constexpr uint32_t kQ = 0, kK = 2 * kQBytes, kV = kK + kNK * kTileBytes;
  static constexpr uint32_t kSmem = kV + kNV * kTileBytes;
  static_assert(kSmem + 3072 <= 232448, "");
};

struct Bars : RingBars {
  unsigned long long s_full[2], p_full[2], pv_done[2], o_free, done;
};

// TMEM columns, of even and odd tiles: S, whose upper half P takes over; O.
constexpr uint32_t kS = 0, kP = 64, kO = 256;

struct Small {
  Bars bars;
  uint32_t tmem;
  int abort;
  uint32_t odd[2][8];  // nodes whose V holds an infinity or NaN, of even and odd units
  float2 ml[2][128];   // a unit's (reference, sum) of the rows, of either group
};
static_assert(sizeof(Small) <= 3072, "");

__device__ __forceinline__ void both_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }

// 32 bytes at once: a warp's lanes write rows of their own, so that a store
// takes a cycle a lane whatever its width.
__device__ __forceinline__ void store_sector(float *at, const float *x) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
k_tree_attn(const TreeAttnParams p, const __grid_constant__ TreeAttnMaps maps) {
  using G = Geom<D>;
  // all of the shared memory there is: the ring at its (1024-byte aligned) base, then Small
  extern __shared__ __align__(1024) uint8_t smem[];
  Small &sm = *reinterpret_cast<Small *>(smem + G::kSmem);
  Bars &b = sm.bars;
  uint32_t &s_tmem = sm.tmem;
  const int tid = threadIdx.x, warp = __shfl_sync(DC_FULL_MASK, tid >> 5, 0), lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // never: there is no static shared memory before it
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b.s_full[i]), 1);
      mbar_init(smem_u32(&b.p_full[i]), kSoftWarps / 2);
      mbar_init(smem_u32(&b.pv_done[i]), 1);
    }
    init_ring<G>(b);
    mbar_init(smem_u32(&b.o_free), kSoftWarps);
    mbar_init(smem_u32(&b.done), 1);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows past the unit's are zeros: what lies there would set off rescales
  for (uint32_t i = tid * 16; i < 2 * G::kQBytes; i += kThreads * 16)
    *reinterpret_cast<uint4 *>(smem + G::kQ + i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (warp == kLoadWarp && lane == 0) prefetch_maps(maps);
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(DC_FULL_MASK, s_tmem, 0);
  int g = 0, live = 0;  // tiles and units with tiles that this role has begun

  pdl_trigger();

  if (warp >= kSoftWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));

  if (warp >= kLoadWarp + kLoadWarps) {
  } else if (warp >= kLoadWarp) {
    load_tiles<G>(p, maps, sbase, b, warp - kLoadWarp, &sm.abort, g, live);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ tensor core
    constexpr uint32_t kIdS = F16 ? idesc_f16(128, kTile) : idesc_bf16(128, kTile);
    constexpr uint32_t kIdO = (F16 ? idesc_f16(128, D) : idesc_bf16(128, D)) | (1u << 16);  // B is N-major
    UnitIter it(p, false);
    Unit w;
    bool ok = true;
    // O (+)= P V of tile t, one of the first two (the groups' first) of the block's unit number `unit` if `first`
    auto pv = [&](int t, bool first, int unit) {
      const int vs = t % G::kNV;
      const bool go = bar_wait(smem_u32(&b.v_full[vs]), (t / G::kNV) & 1, &sm.abort, p.err) &&
                      (!first || unit == 0 || bar_wait(smem_u32(&b.o_free), (unit - 1) & 1, &sm.abort, p.err)) &&
                      bar_wait(smem_u32(&b.p_full[t & 1]), (t >> 1) & 1, &sm.abort, p.err);
      if (!__all_sync(DC_FULL_MASK, go)) return false;
      tc_fence_after();
      const uint32_t sv = mn_major_lo(sbase + G::kV + vs * G::kTileBytes);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(tmem + kO + (t & 1) * 128, tmem + kP + (t & 1) * 128 + k * 8, sv + k * (2048 >> 4), kIdO, (!first || k > 0) ? 1u : 0u);
        mma_commit(smem_u32(&b.v_empty[vs]));
        mma_commit(smem_u32(&b.pv_done[t & 1]));
      }
      __syncwarp();
      return true;
    };
    bool prev_first = false;
    int prev_unit = 0;
    while (ok && it.next(w)) {
      if (w.ntiles == 0) continue;
      const int qb = live & 1;
      ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.q_full[qb]), (live >> 1) & 1, &sm.abort, p.err));
      for (int i = 0; ok && i < w.ntiles; ++i, ++g) {
        const int ks = g % G::kNK;
        // S's columns hold the weights of two tiles ago until their product is done
        ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.k_full[ks]), (g / G::kNK) & 1, &sm.abort, p.err) &&
                                          (g < 2 || bar_wait(smem_u32(&b.pv_done[g & 1]), ((g >> 1) - 1) & 1, &sm.abort, p.err)));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sq = k_major_lo(sbase + G::kQ + qb * G::kQBytes);
        const uint32_t sk = k_major_lo(sbase + G::kK + ks * G::kTileBytes);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * G::kHalfBytes + (k & 3) * 32) >> 4;
            mma_ss(tmem + kS + (g & 1) * 128, sq + off, sk + off, kIdS, k > 0 ? 1u : 0u);
          }
          mma_commit(smem_u32(&b.s_full[g & 1]));
          mma_commit(smem_u32(&b.k_empty[ks]));
          if (i == w.ntiles - 1) mma_commit(smem_u32(&b.q_empty[qb]));
        }
        __syncwarp();
        if (g > 0) ok = pv(g - 1, prev_first, prev_unit);
        prev_first = i < 2, prev_unit = live;
      }
      ++live;
    }
    if (ok && g > 0) pv(g - 1, prev_first, prev_unit);
    if (elect_one()) {  // the lane that issued: nothing is in flight when the block frees its TMEM
      mma_commit(smem_u32(&b.done));
      mbar_drain(smem_u32(&b.done), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, output
    UnitIter it(p, false);
    Unit w;
    const int group = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;             // row of the tile: node row / p.group
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    const int rnode = row / p.group;
    const bool used = row < p.tile_rows;
    float c = p.scale * kLog2e;
    const bool flip = c < 0.f, zero = c == 0.f;
    c = zero ? 1.f : fabsf(c);
    bool ok = true;
    auto wait = [&](unsigned long long *bar, int phase) {
      if (ok) ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(bar), phase & 1, &sm.abort, p.err));
    };
    while (it.next(w)) {
      if (w.ntiles == 0) continue;
      const int node = w.mt * p.tile_nodes + rnode, par = live & 1;
      const bool live_row = used && node < w.len;
      float ref = kNone, l = 0.f;                 // reference (log2 units) and sum of this row
      bool seen_tree = false;
      for (int i = 0; i < w.ntiles; ++i, ++g) {
        const int tile = w.tile0 + i;
        const bool tree = tile >= w.nctx;
        seen_tree |= tree;
        if ((g & 1) != group) continue;
        const int tok0 = (tree ? tile - w.nctx : tile) * kTile;
        const int valid = min(kTile, (tree ? w.len : w.ctx) - tok0);
        wait(&b.s_full[group], g >> 1);
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};   // tokens of the tile that this row sees
        const bool masked = valid < kTile || tree;
        if (masked) {
          wait(&b.v_full[g % G::kNV], g / G::kNV);
          bool bad = false;
          if (ok)
            bad = clean_v_row<D, F16>(smem + G::kV + (g % G::kNV) * G::kTileBytes + row * 128, row < valid, tree);
          fence_proxy_async();
          const uint32_t bits = __ballot_sync(DC_FULL_MASK, bad);
          if (tree && lane == 0) sm.odd[par][tok0 / 32 + quad] = bits;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int left = valid - q * 32;      // tokens of this word that exist
            see[q] = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1u : 0u;
            if (tree) see[q] = tree_sees(p, w.n, w.len, live_row ? node : w.len, tok0 / 32 + q);
          }
        }
        tc_fence_after();
        const uint32_t ts = trow + kS + group * 128;
        uint32_t pk[2][32];                       // the tile's weights, packed
        // once, or once more when a score has outgrown the reference
        float sum;
        for (bool renew = i < 2;; renew = true) {
          float top = -INFINITY;
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
          if (renew) {
            // the row's maximum over the tile
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              const uint32_t word = q == 0 ? see[0] : q == 1 ? see[1] : q == 2 ? see[2] : see[3];
              float v[32];
              tmem_ld32(ts + q * 32, v);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float x = zero ? 0.f : flip ? -v[k] : v[k];
                top = fmaxf(top, (word >> k) & 1u ? x : -INFINITY);
              }
            }
            top *= c;
            if (i < 2) {
              ref = top > kNone ? top : kNone;
            } else {
              const float f = top > ref ? ex2(ref - top) : 1.f;
              ref = fmaxf(ref, top);
              l *= f;
              // this group's last product is done (S was written after it)
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float x[32];
                uint32_t y[32];
                tmem_ld32(trow + kO + group * 128 + q * 32, x);
#pragma unroll
                for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(x[k] * f);
                tmem_st32(trow + kO + group * 128 + q * 32, y);
              }
              tmem_st_wait();
            }
          }
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t raw[2][32];
          tmem_ld32_start(ts, raw[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t(&r)[32] = raw[q & 1];
            tmem_ld_wait(r);
            if (q < 3) tmem_ld32_start(ts + (q + 1) * 32, raw[(q + 1) & 1]);  // in flight during this part's arithmetic
            if (flip | zero) {
#pragma unroll
              for (int k = 0; k < 32; ++k) r[k] = zero ? 0u : r[k] ^ 0x80000000u;
            }
            if (masked) {
#pragma unroll
              for (int k = 0; k < 32; ++k) r[k] = (see[q] >> k) & 1u ? r[k] : 0xFF800000u;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float x = fmaf(__uint_as_float(r[2 * k]), c, -ref), y = fmaf(__uint_as_float(r[2 * k + 1]), c, -ref);
              t4[k & 3] = fmaxf(t4[k & 3], fmaxf(x, y));
              const float a = ex2(x), d = ex2(y);
              s4[(2 * k) & 3] += a;
              s4[(2 * k + 1) & 3] += d;
              pk[q >> 1][(q & 1) * 16 + k] = pack2<F16>(a, d);
            }
          }
          top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          if (renew || !__any_sync(DC_FULL_MASK, top > kRescale)) break;
        }
        l += sum;
        tmem_st32(trow + kP + group * 128, pk[0]);
        tmem_st32(trow + kP + group * 128 + 32, pk[1]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&b.p_full[group]));
      }
      // -------------------------------------------------------- the unit's output
      // Each group weighs half of the columns of both O together.
      const int last = g - 1, g0 = g - w.ntiles;  // the unit's last and first tile
      const bool lone = w.ntiles == 1;            // only group g0 & 1 had a tile
      if (!lone || group == (g0 & 1)) {
        const int mine = (last & 1) == group ? last : last - 1;
        wait(&b.pv_done[group], mine >> 1);
        // after the wait: this unit's first products waited for o_free, where
        // the other group arrives when it has read the last unit's ml
        sm.ml[group][row] = make_float2(ref, l);
      }
      both_sync();
      tc_fence_after();
      // In the order of the tiles, not of the groups: which group has a unit's
      // first tile depends on the units before it, and the result must not.
      const int ga = g0 & 1;  // has the unit's first tile (and third, ...)
      const float2 a = sm.ml[ga][row], z = lone ? make_float2(kNone, 0.f) : sm.ml[ga ^ 1][row];
      const float M = fmaxf(a.x, z.x), fa = ex2(a.x - M), fz = ex2(z.x - M);
      const int64_t item = ((int64_t)w.n * p.kv_heads + w.h) * p.mtiles + w.mt;
      const int64_t slot = (item * p.max_chunks + w.chunk) * p.part_rows + row;
      float *part = reinterpret_cast<float *>(p.part_o) + slot * D + group * (D / 2);
#pragma unroll 1
      for (int q = 0; q < D / 64; ++q) {
        const uint32_t col = trow + kO + group * (D / 2) + q * 32;
        float x[32], y[32];
        tmem_ld32(col + ga * 128, x);
        if (!lone) {
          tmem_ld32(col + (ga ^ 1) * 128, y);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = fmaf(y[k], fz, x[k] * fa);
        }
        if (used && ok) {
#pragma unroll
          for (int k = 0; k < 4; ++k) store_sector(part + q * 32 + k * 8, &x[k * 8]);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&b.o_free));
      if (group == 0 && used && ok)
        p.part_ml[slot] = lone ? a : make_float2(M, fmaf(z.y, fz, a.y * fa));
      if (seen_tree && live_row && ok) {
        // infinities and NaN of the nodes that the row sees
#pragma unroll 1
        for (int q = max(0, w.tile0 - w.nctx) * 4; q < (w.tile0 + w.ntiles - w.nctx) * 4 && q < (p.T + 31) / 32; ++q)
#pragma unroll 1
          for (uint32_t r = sm.odd[par][q]; r; r &= r - 1) {
            const int jn = q * 32 + __ffs(r) - 1;
            if (!((tree_sees(p, w.n, w.len, node, q) >> (jn & 31)) & 1u)) continue;
            const uint16_t *vn = p.v_new + w.n * p.vn_sn + jn * p.vn_st + w.h * p.vn_sh + group * (D / 2);
#pragma unroll 1
            for (int k = 0; k < D / 2; ++k) {
              const uint32_t e = vn[k];
              if (nonfinite2<F16>(e)) part[k] += unpack_lo<F16>(e);
            }
          }
      }
      __syncwarp();
      ++live;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sm.abort && warp >= kLoadWarp && warp < kLoadWarp + kLoadWarps && lane == 0) drain_copies<G>(b, warp - kLoadWarp, g, live);
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The output of each row from its chunks: sum_k 2^(m_k - M) O_k / sum_k
// 2^(m_k - M) l_k, M = max m_k, in chunk order; zeros for a node past the
// tree's length and for one that saw nothing.  One warp a row, its elements
// over the lanes.  (Joining inside the attention kernel, by the last block of
// an item, took that block 7 us for 64 rows and four chunks, and some blocks
// had four items to join.)  Bound by the latency of its loads: six blocks an
// SM with four chunks in flight a warp; four with eight took 3 us longer for
// 16,384 rows of up to 16 chunks, eight with four 2 us.
template <int D, bool F16>
__global__ void __launch_bounds__(256, 6) k_tree_join(const TreeAttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, heads = p.kv_heads * p.group;
  const int n = blockIdx.x, of_n = blockIdx.y * 8 + (threadIdx.x >> 5);  // request, row of it
  if (of_n >= p.T * heads) return;
  const int node = of_n / heads, hq = of_n - node * heads;
  const int64_t orow = (int64_t)n * p.T * heads + of_n;
  int ctx, len;
  const int nchunks = request_chunks(p, n, ctx, len);
  const int h = hq / p.group, mt = node / p.tile_nodes;
  const int row = (node - mt * p.tile_nodes) * p.group + hq - h * p.group, R = p.part_rows;
  const int64_t item = ((int64_t)n * p.kv_heads + h) * p.mtiles + mt;
  const float *po = reinterpret_cast<const float *>(p.part_o) + (item * p.max_chunks * R + row) * D + lane * E;
  const float2 *ml = p.part_ml + item * p.max_chunks * R + row;
  pdl_wait();
  float2 a[2];  // chunks lane and 32 + lane (at most kTreeMaxChunks)
  const int live = node < len ? nchunks : 0;
  for (int q = 0; q < 2; ++q) a[q] = q * 32 + lane < live ? __ldcg(&ml[(int64_t)(q * 32 + lane) * R]) : make_float2(kNone, 0.f);
  const float M = warp_max(fmaxf(a[0].x, a[1].x));
  const float w[2] = {ex2(a[0].x - M), ex2(a[1].x - M)};
  const float L = warp_sum(w[0] * a[0].y + w[1] * a[1].y);
  float acc[E] = {};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int k1 = min(live, q * 32 + 32);
#pragma unroll 4
    for (int k = q * 32; k < k1; ++k) {
      const float f = __shfl_sync(DC_FULL_MASK, w[q], k & 31);
      const float *src = po + (int64_t)k * R * D;
      if constexpr (E == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
        acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]);
        acc[2] = fmaf(f, x.z, acc[2]), acc[3] = fmaf(f, x.w, acc[3]);
      } else {
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
        acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]);
      }
    }
  }
  const bool some = node < len && L != 0.f;
  const float inv = some ? 1.f / L : 0.f;
  uint32_t *out = reinterpret_cast<uint32_t *>(p.out + orow * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = some ? pack2<F16>(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  if (p.lse && lane == 0) p.lse[orow] = some ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

template <int D, bool F16>
cudaError_t launch_join(const TreeAttnParams &p, cudaStream_t st) {
  const int rows = p.T * p.kv_heads * p.group;  // at most 256 x 1024 a request
  return launch_ex(k_tree_join<D, F16>, dim3((unsigned)p.N, (unsigned)((rows + 7) / 8)), dim3(256), 0, st, true, 0, p);
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
cudaError_t launch(const TreeAttnParams &p, const TreeAttnMaps &maps, unsigned grid, cudaStream_t st) {
  const size_t smem = Geom<D>::kSmem + sizeof(Small);
  const cudaError_t e =
      cudaFuncSetAttribute(k_tree_attn<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k_tree_attn<D, F16><<<grid, kThreads, smem, st>>>(p, maps);
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
  const int64_t most = (int64_t)p.N * p.kv_heads * p.mtiles * p.max_chunks;
  const unsigned grid = (unsigned)(most < p.sms ? most : p.sms);
  cudaError_t e;
  if (p.few) e = launch_tree_attention_few(p, maps, grid, st);
  else if (p.head_dim == 128) e = p.f16 ? launch<128, true>(p, maps, grid, st) : launch<128, false>(p, maps, grid, st);
  else e = p.f16 ? launch<64, true>(p, maps, grid, st) : launch<64, false>(p, maps, grid, st);
  if (e != cudaSuccess) return e;
  if (p.head_dim == 128) return p.f16 ? launch_join<128, true>(p, st) : launch_join<128, false>(p, st);
  return p.f16 ? launch_join<64, true>(p, st) : launch_join<64, false>(p, st);
}

}  // namespace dc
