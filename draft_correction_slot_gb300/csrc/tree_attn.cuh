// tree_attn.cuh -- what the two tree-attention kernels share: units of work,
// TMEM and TMA helpers, the copies of a tile.
#pragma once

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
constexpr float kRescale = 8.f;       // log2 growth of a row's maximum before the output is rescaled

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// mbar_wait without its clock read on the way in: most waits here end within
// a few tries, and the chain of a tile passes through five of them.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *abort, int *err) {
  unsigned long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try(bar, parity)) return true;
    if ((it & 255u) == 0u) {
      if (*abort) return false;
      const unsigned long long t = global_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitNs) {
        *abort = 1;
        atomicOr(err, kErrTimeout);
        return false;
      }
    }
  }
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
// The tensor-core warp keeps its control flow and descriptors uniform (all
// lanes run the loop, one issues): from a branch of one lane every operand
// went through vector registers and a product's issue cost about 100 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// Shared-memory descriptors as two words.  High: 8-row (or 8-token) groups
// 1024 bytes apart, 128-byte swizzle.  Low: the address, and for a V tile
// (tokens along K, columns along M or N) the distance of 64-column blocks.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t k_major_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t mn_major_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (uint32_t)((kTile * 128) >> 4) << 16;
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "mov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 b;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "mov.b64 b, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// 32 lanes x C consecutive columns, C = 8, 16 or 32.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[C]) {
  if constexpr (C == 32) {
    tmem_ld32(addr, v);
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "r"(addr)
        : "memory");
  }
}
// A load in flight: 32 columns; its registers are the caller's only after
// tmem_ld_wait.
#define DC_R8(c, i) c(r[i]), c(r[i + 1]), c(r[i + 2]), c(r[i + 3]), c(r[i + 4]), c(r[i + 5]), c(r[i + 6]), c(r[i + 7])
#define DC_R32(c) DC_R8(c, 0), DC_R8(c, 8), DC_R8(c, 16), DC_R8(c, 24)
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : DC_R32("=r")
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : DC_R32("+r")::"memory");
}
#undef DC_R32
#undef DC_R8
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

// ---------------------------------------------------------------- units
struct Unit {
  int n, h, mt, chunk, nchunks;  // request, K/V head, row tile, chunk of the request's nchunks
  int ctx, len;                  // clamped lengths
  int tile0, ntiles, nctx;       // first tile, tiles (0: no live rows), context tiles of the request
};

// Lengths of request n, clamped, and its chunks (at least 1).
__device__ __forceinline__ int request_chunks(const TreeAttnParams &p, int n, int &ctx, int &len, bool flag = false) {
  const int capacity = p.max_pages << p.page_shift;
  ctx = p.ctx_len[n];
  len = p.tree_len ? p.tree_len[n] : p.T;
  if ((ctx < 0 || ctx > capacity || len < 0 || len > p.T) && flag) atomicOr(p.err, kErrBadLength);
  ctx = min(max(ctx, 0), capacity);
  len = len < 0 ? 0 : min(len, p.T);
  const int nt = len > 0 ? (ctx + kTile - 1) / kTile + (len + kTile - 1) / kTile : 0;
  const int per = tree_chunk_tiles(nt, p.items, p.sms, p.chunk_cap);
  return nt > 0 ? (nt + per - 1) / per : 1;
}

// This block's units, warp by warp without communication: 32 requests' lengths
// at a time in the lanes, those with the largest chunks first; units in the
// order (request, chunk, head, row tile), dealt to the blocks to and fro.
// (Dealt in request order and one way, the fullest of 152 blocks had 20 % more
// tiles than the mean for 32 requests of 1000 to 8000 tokens; now 13 %.)
struct UnitIter {
  const TreeAttnParams &p;
  int lane, base = 0, n0 = 0, round = 0, req = 0;
  int ctx = 0, len = 0, chunks = 0, before = 0, upto = 0, window = 0;
  __device__ UnitIter(const TreeAttnParams &p_, bool flag) : p(p_), lane(threadIdx.x & 31) { load(flag); }
  __device__ void load(bool flag) {
    req = n0 + lane;
    chunks = 0;
    if (req < p.N) chunks = request_chunks(p, req, ctx, len, flag);
    scan();
    if (p.N <= 32 && window <= (int)gridDim.x) return;  // one unit a block at most
    // sort the lanes by their tiles a chunk
    const int tiles = (ctx + kTile - 1) / kTile + (len + kTile - 1) / kTile;
    const int key = chunks > 0 ? len > 0 ? (tiles + chunks - 1) / chunks : 0 : -1;
    int rank = 0, src = 0;
#pragma unroll 8
    for (int o = 0; o < 32; ++o) {
      const int k = __shfl_sync(DC_FULL_MASK, key, o);
      rank += k > key || (k == key && o < lane);
    }
#pragma unroll 8
    for (int o = 0; o < 32; ++o)
      if (__shfl_sync(DC_FULL_MASK, rank, o) == lane) src = o;
    req = __shfl_sync(DC_FULL_MASK, req, src);
    ctx = __shfl_sync(DC_FULL_MASK, ctx, src);
    len = __shfl_sync(DC_FULL_MASK, len, src);
    chunks = __shfl_sync(DC_FULL_MASK, chunks, src);
    scan();
  }
  __device__ void scan() {  // units before and up to each lane's request, in the window
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
    const int u = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    while (u - base >= window) {
      base += window;
      n0 += 32;
      if (n0 >= p.N) return false;
      load(flag);
    }
    const int rel = u - base;
    const int src = __ffs(__ballot_sync(DC_FULL_MASK, upto > rel)) - 1;
    int i = rel - __shfl_sync(DC_FULL_MASK, before, src);
    w.n = __shfl_sync(DC_FULL_MASK, req, src);
    w.ctx = __shfl_sync(DC_FULL_MASK, ctx, src);
    w.len = __shfl_sync(DC_FULL_MASK, len, src);
    w.nchunks = __shfl_sync(DC_FULL_MASK, chunks, src);
    w.mt = i % p.mtiles, i /= p.mtiles;
    w.h = i % p.kv_heads, w.chunk = i / p.kv_heads;
    w.nctx = (w.ctx + kTile - 1) / kTile;
    const int nt = w.mt * p.tile_nodes < w.len ? w.nctx + (w.len + kTile - 1) / kTile : 0;
    w.tile0 = (int)((int64_t)nt * w.chunk / w.nchunks);  // chunks as even as they come
    w.ntiles = (int)((int64_t)nt * (w.chunk + 1) / w.nchunks) - w.tile0;
    ++round;
    return true;
  }
};


__device__ __forceinline__ void prefetch_maps(const TreeAttnMaps &maps) {
  const CUtensorMap *m[] = {&maps.q, &maps.k_cache, &maps.v_cache, &maps.k_new, &maps.v_new};
#pragma unroll
  for (int i = 0; i < 5; ++i)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m[i])) : "memory");
}

struct RingBars {
  unsigned long long q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4], v_empty[4];
};

// The two TMA warps: role 0 copies Q of every unit and K of every tile, role 1
// V; a page's tokens are a copy of their own.  G gives the shared-memory
// layout: kHalves 64-element column blocks, two Q buffers of kQBytes (a column
// block kQHalf) at kQ, kNK K and kNV V stages of kTileBytes (a column block
// kHalfBytes) at kK and kV.  g and live count the tiles and units begun.
constexpr int kLoadWarps = 2;
template <class G>
__device__ __forceinline__ void load_tiles(const TreeAttnParams &p, const TreeAttnMaps &maps, uint32_t sbase,
                                           RingBars &b, int role, volatile int *abort, int &g, int &live) {
  const int lane = threadIdx.x & 31;
  const bool is_v = role == 1;
  const int stages = is_v ? G::kNV : G::kNK;
  unsigned long long *full = is_v ? b.v_full : b.k_full, *empty = is_v ? b.v_empty : b.k_empty;
  const uint32_t ring = sbase + (is_v ? G::kV : G::kK);
  const CUtensorMap *cache = is_v ? &maps.v_cache : &maps.k_cache, *fresh = is_v ? &maps.v_new : &maps.k_new;
  UnitIter it(p, role == 0 && blockIdx.x == 0);
  Unit w;
  const int page_size = 1 << p.page_shift;
  const int box = min(page_size, kTile);  // tokens of one copy
  const int boxes = kTile / box;          // copies of a tile's column block
  bool ok = true;
  int stage = 0, round = 0;
  while (it.next(w, role == 0 && blockIdx.x == 0)) {
    if (w.ntiles == 0) continue;
    if (role == 0) {
      const int qb = live & 1;
      if (live >= 2) ok = bar_wait(smem_u32(&b.q_empty[qb]), ((live >> 1) - 1) & 1, abort, p.err);
      if (!__all_sync(DC_FULL_MASK, ok)) return;
      if (elect_one()) {
        mbar_arrive_expect_tx(smem_u32(&b.q_full[qb]), (uint32_t)(G::kHalves * p.tile_rows * 128));
        for (int c = 0; c < G::kHalves; ++c)
          tma_load_4d(sbase + G::kQ + qb * G::kQBytes + c * G::kQHalf, &maps.q, c * 64, w.h * p.group,
                      w.mt * p.tile_nodes, w.n, smem_u32(&b.q_full[qb]));
      }
    }
    ++live;
    for (int i = 0; i < w.ntiles; ++i, ++g) {
      const int tile = w.tile0 + i;
      const bool tree = tile >= w.nctx;
      const int tok0 = (tree ? tile - w.nctx : tile) * kTile;
      int page = 0, used = 1;  // copies of a column block; lane r holds copy r's page
      if (!tree) {
        used = min(boxes, (w.ctx - tok0 + box - 1) / box);
        if (lane < used) {
          page = __ldg(p.page_table + w.n * p.pt_stride + ((tok0 + lane * box) >> p.page_shift));
          if (page < 0 || page >= p.num_pages) {
            atomicOr(p.err, kErrBadPage);
            page = 0;
          }
        }
      }
      if (round > 0) ok = bar_wait(smem_u32(&empty[stage]), (round - 1) & 1, abort, p.err);
      if (!__all_sync(DC_FULL_MASK, ok)) return;
      const uint32_t dst = ring + stage * G::kTileBytes, bar = smem_u32(&full[stage]);
      if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(G::kHalves * 128 * (tree ? p.tree_box : used * box)));
      __syncwarp();
      for (int r = 0; r < used; ++r) {
        const int pg = __shfl_sync(DC_FULL_MASK, page, r);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < G::kHalves; ++c) {
            if (tree) tma_load_4d(dst + c * G::kHalfBytes, fresh, c * 64, tok0, w.h, w.n, bar);
            else tma_load_4d(dst + c * G::kHalfBytes + r * box * 128, cache, c * 64, tok0 & (page_size - 1), w.h, pg, bar);
          }
        }
        __syncwarp();
      }
      if (++stage == stages) stage = 0, ++round;
    }
  }
}

// After an expired wait: copies in flight land before the block gives its
// memory back.  Called by one thread of each TMA warp after the roles have
// met, with the tiles and units it began.
template <class G>
__device__ __forceinline__ void drain_copies(RingBars &b, int role, int g, int live) {
  const int stages = role == 1 ? G::kNV : G::kNK;
  unsigned long long *full = role == 1 ? b.v_full : b.k_full;
  for (int t = max(0, g - stages); t < g; ++t) mbar_drain(smem_u32(&full[t % stages]), (t / stages) & 1);
  if (role == 0)
    for (int t = max(0, live - 2); t < live; ++t) mbar_drain(smem_u32(&b.q_full[t & 1]), (t >> 1) & 1);
}

constexpr float kNone = -1e30f;  // reference of a row that has seen nothing: any score outgrows it

template <class G>
__device__ __forceinline__ void init_ring(RingBars &b) {
  for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&b.q_full[i]), 1), mbar_init(smem_u32(&b.q_empty[i]), 1);
  for (int i = 0; i < G::kNK; ++i) mbar_init(smem_u32(&b.k_full[i]), 1), mbar_init(smem_u32(&b.k_empty[i]), 1);
  for (int i = 0; i < G::kNV; ++i) mbar_init(smem_u32(&b.v_full[i]), 1), mbar_init(smem_u32(&b.v_empty[i]), 1);
}

// One token's row of a V tile before the product reads it.  Past the end
// (`there` false) lies what a page or a copy left: zeros in its place, since a
// zero weight does not cancel an infinity.  In the tree, a node's infinities
// and NaN stay out of the product (they would reach nodes that do not see it)
// and are added to the output of those that do.  Returns whether it had any.
template <int D, bool F16>
__device__ __forceinline__ bool clean_v_row(uint8_t *row, bool there, bool tree) {
  bool bad = false;
  if (!there) {
#pragma unroll
    for (int e = 0; e < D / 8; ++e)
      *reinterpret_cast<uint4 *>(row + (e >> 3) * (kTile * 128) + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
  } else if (tree) {
    for (int e = 0; e < D / 8; ++e) {
      uint4 *v = reinterpret_cast<uint4 *>(row + (e >> 3) * (kTile * 128) + (e & 7) * 16);
      const uint4 x = *v;
      uint32_t xs[4] = {x.x, x.y, x.z, x.w};
      bool any = false;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (nonfinite2<F16>(xs[k])) {
          const bool lo = nonfinite2<F16>(xs[k] & 0xFFFFu), hi = nonfinite2<F16>(xs[k] >> 16);
          xs[k] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
          any = true;
        }
      if (any) *v = make_uint4(xs[0], xs[1], xs[2], xs[3]);
      bad |= any;
    }
  }
  return bad;
}

// Word `word` of what node `node` sees of the tree's first len nodes.
__device__ __forceinline__ uint32_t tree_sees(const TreeAttnParams &p, int n, int len, int node, int word) {
  const int words = (p.T + 31) / 32, left = len - word * 32;
  if (left <= 0 || node >= len) return 0u;
  const uint32_t there = left >= 32 ? ~0u : (1u << left) - 1u;
  if (p.tree_mask) return there & (uint32_t)__ldg(p.tree_mask + n * p.mask_sn + (int64_t)node * words + word);
  const int upto = node + 1 - word * 32;  // nodes 0..node
  return there & (upto >= 32 ? ~0u : upto > 0 ? (1u << upto) - 1u : 0u);
}

}  // namespace
}  // namespace dc
