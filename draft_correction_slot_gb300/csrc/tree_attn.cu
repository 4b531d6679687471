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
// products run on across unit borders.  Each unit leaves its rows'
// unnormalised output with their references and sums, and a second kernel
// joins the chunks.
//
// Roles: warps 0-3 softmax and output (thread = row = TMEM lane), warp 4 the
// tensor core, warps 5-6 TMA.
#include "launch.h"
#include "tree_attn.cuh"

namespace dc {
namespace {

constexpr int kSoftWarps = 4;
constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);

template <int D>
struct Geom {
  static constexpr int kHalves = D / 64;                 // 64-element column blocks (128 bytes, one swizzle span)
  static constexpr uint32_t kHalfBytes = kTile * 128;    // a tile's column block
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  static constexpr int kNK = D == 128 ? 2 : 4, kNV = D == 128 ? 3 : 4;  // K and V stages
  static constexpr uint32_t kQHalf = kHalfBytes, kQBytes = kTileBytes;
  static constexpr uint32_t kQ = 0, kK = 2 * kQBytes, kV = kK + kNK * kTileBytes;
  static constexpr uint32_t kSmem = kV + kNV * kTileBytes;
};

struct Bars : RingBars {
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
  __shared__ int s_abort;
  __shared__ uint32_t s_odd[4];  // tree tile: nodes whose V holds an infinity or NaN
  const int tid = threadIdx.x, warp = __shfl_sync(DC_FULL_MASK, tid >> 5, 0), lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b.s_full[i]), 1);
      mbar_init(smem_u32(&b.p_full[i]), kSoftWarps);
      mbar_init(smem_u32(&b.pv_done[i]), 1);
    }
    init_ring<G>(b);
    mbar_init(smem_u32(&b.o_free), kSoftWarps);
    mbar_init(smem_u32(&b.soft), kSoftWarps);
    mbar_init(smem_u32(&b.done), 1);
    s_abort = 0;
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

  if (warp >= kLoadWarp) {
    load_tiles<G>(p, maps, sbase, b, warp - kLoadWarp, &s_abort, g, live);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ tensor core
    constexpr uint32_t kIdS = F16 ? idesc_f16(128, kTile) : idesc_bf16(128, kTile);
    constexpr uint32_t kIdO = (F16 ? idesc_f16(128, D) : idesc_bf16(128, D)) | (1u << 16);  // B is N-major
    UnitIter it(p, false);
    Unit w;
    bool ok = true;
    // O (+)= P V of tile t, the first of the block's unit number `unit` if `first`
    auto pv = [&](int t, bool first, int unit) {
      const int vs = t % G::kNV;
      const bool go = bar_wait(smem_u32(&b.v_full[vs]), (t / G::kNV) & 1, &s_abort, p.err) &&
                      (!first || unit == 0 || bar_wait(smem_u32(&b.o_free), (unit - 1) & 1, &s_abort, p.err)) &&
                      bar_wait(smem_u32(&b.p_full[t & 1]), (t >> 1) & 1, &s_abort, p.err);
      if (!__all_sync(DC_FULL_MASK, go)) return false;
      tc_fence_after();
      const uint32_t sv = mn_major_lo(sbase + G::kV + vs * G::kTileBytes);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(tmem + kO, tmem + kP + (t & 1) * 64 + k * 8, sv + k * (2048 >> 4), kIdO, (!first || k > 0) ? 1u : 0u);
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
      ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.q_full[qb]), (live >> 1) & 1, &s_abort, p.err));
      for (int i = 0; ok && i < w.ntiles; ++i, ++g) {
        const int ks = g % G::kNK;
        ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.k_full[ks]), (g / G::kNK) & 1, &s_abort, p.err));
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
        prev_first = i == 0, prev_unit = live;
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
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const int row = tid;                          // row of the tile: node row / group, head row % group
    const int rnode = row / p.group;
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
      const bool met = bar_wait(smem_u32(&b.soft), syncs++ & 1, &s_abort, p.err);
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
        ok = bar_wait(smem_u32(&b.s_full[g & 1]), (g >> 1) & 1, &s_abort, p.err);
        if (valid < kTile || tree) {
          ok = ok && bar_wait(smem_u32(&b.v_full[g % G::kNV]), (g / G::kNV) & 1, &s_abort, p.err);
          ok = __all_sync(DC_FULL_MASK, ok);
          if (!ok) break;
          const bool bad = clean_v_row<D, F16>(smem + G::kV + (g % G::kNV) * G::kTileBytes + row * 128, row < valid, tree);
          if (tree) {
            const uint32_t bits = __ballot_sync(DC_FULL_MASK, bad);
            ok = meet();  // the previous tree tile's bits have been read
            if (lane == 0) s_odd[warp] = bits;
            ok = ok && meet();
          }
          fence_proxy_async();
        }
        if (g >= 2)  // P's columns are free
          ok = ok && bar_wait(smem_u32(&b.pv_done[g & 1]), ((g >> 1) - 1) & 1, &s_abort, p.err);
        ok = __all_sync(DC_FULL_MASK, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = trow + kS + (g & 1) * 128, tp = trow + kP + (g & 1) * 64;
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};  // tokens of the tile that this row sees
        const bool masked = valid < kTile || tree;
        if (masked) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int left = valid - q * 32;  // tokens of this word that exist
            see[q] = left >= 32 ? 0xFFFFFFFFu : left > 0 ? (1u << left) - 1u : 0u;
          }
          if (tree) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              see[q] &= tree_sees(p, w.n, w.len, live_row ? node : w.len, tok0 / 32 + q);
              const uint32_t o = see[q] & s_odd[q];
              if (tok0 == 0) odd[q] = o;
              else odd[4 + q] = o;
              any_odd |= o != 0;
            }
          }
        }
        // 64 scores at a time (all 128 would not fit the registers): the
        // maximum over both halves, then the weights of the second half, still
        // held, and of the first, read from TMEM again.
        float v[64];
        auto load = [&](int half) {
          tmem_ld64(ts + half * 64, v);
          if (flip | zero) {
#pragma unroll
            for (int k = 0; k < 64; ++k) v[k] = zero ? 0.f : -v[k];
          }
          if (masked) {
#pragma unroll
            for (int k = 0; k < 64; ++k) {
              const uint32_t word = half == 0 ? see[k >> 5] : see[2 + (k >> 5)];
              v[k] = (word >> (k & 31)) & 1u ? v[k] : -INFINITY;
            }
          }
        };
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          load(half);
#pragma unroll
          for (int k = 0; k < 64; ++k) m4[k & 3] = fmaxf(m4[k & 3], v[k]);
        }
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
        if (i == 0) {
          mref = mt;
        } else {
          const bool grow = mt > mref + kRescale;  // from -inf: any finite maximum
          if (__any_sync(DC_FULL_MASK, grow)) {
            const float f = grow ? ex2(mref - mt) : 1.f;
            if (grow) mref = mt, l *= f;
            ok = bar_wait(smem_u32(&b.pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, &s_abort, p.err);
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
        for (int q = 1; q >= 0; --q) {
          if (q == 0) load(0);
          uint32_t y[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float a = ex2(fmaf(v[2 * k], c, -mb)), d = ex2(fmaf(v[2 * k + 1], c, -mb));
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
      if (w.ntiles == 0) continue;
      ok = bar_wait(smem_u32(&b.pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, &s_abort, p.err);
      ok = __all_sync(DC_FULL_MASK, ok);
      if (!ok) break;
      tc_fence_after();
      const int64_t item = ((int64_t)w.n * p.kv_heads + w.h) * p.mtiles + w.mt;
      const int64_t slot = (item * p.max_chunks + w.chunk) * p.part_rows + row;
      float *part = reinterpret_cast<float *>(p.part_o) + slot * D;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float x[32];
        tmem_ld32(trow + kO + q * 32, x);
        if (used) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            reinterpret_cast<float4 *>(part)[q * 8 + k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
        __syncwarp();
      }
      if (used) p.part_ml[slot] = make_float2(mref == -INFINITY ? kNone : mref, l);
      if (any_odd) {
        // infinities and NaN of the nodes that the row sees
#pragma unroll 1
        for (int q = 0; q < 8; ++q)
          for (uint32_t r = odd[q]; r; r &= r - 1) {
            const uint16_t *vn = p.v_new + w.n * p.vn_sn + (q * 32 + __ffs(r) - 1) * p.vn_st + w.h * p.vn_sh;
#pragma unroll 1
            for (int k = 0; k < D; ++k) {
              const uint32_t e = vn[k];
              if (nonfinite2<F16>(e)) part[k] += unpack_lo<F16>(e);
            }
          }
      }
      __syncwarp();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&b.o_free));
      ++live;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_abort && warp >= kLoadWarp && lane == 0) drain_copies<G>(b, warp - kLoadWarp, g, live);
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The output of each row from its chunks: sum_k 2^(m_k - M) O_k / sum_k
// 2^(m_k - M) l_k, M = max m_k, in chunk order; zeros for a node past the
// tree's length and for one that saw nothing.  One warp a row, its elements
// over the lanes.  (Joining inside the attention kernel, by the last block of
// an item, took that block 7 us for 64 rows and four chunks, and some blocks
// had four items to join.)
template <int D, bool F16>
__global__ void __launch_bounds__(256) k_tree_join(const TreeAttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, heads = p.kv_heads * p.group;
  const int64_t orow = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (orow >= (int64_t)p.N * p.T * heads) return;
  const int hq = (int)(orow % heads), node = (int)(orow / heads % p.T), n = (int)(orow / heads / p.T);
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
#pragma unroll 8
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
  const int64_t rows = (int64_t)p.N * p.T * p.kv_heads * p.group;
  return launch_ex(k_tree_join<D, F16>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, true, 0, p);
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
cudaError_t launch(const TreeAttnParams &p, const TreeAttnMaps &maps, unsigned grid, cudaStream_t st) {
  const size_t smem = Geom<D>::kSmem + 1024;
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
