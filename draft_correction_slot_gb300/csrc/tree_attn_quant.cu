// tree_attn_quant.cu -- attention of a drafted tree's nodes (single tokens among
// them) over a paged cache held in 8 bits, and over the tree itself in 16.
//
//   out_i = sum_j e^{s_ij} v_j / sum_j e^{s_ij},  s_ij = scale q_i.k_j,
//   k_j = K8_j ks_b, v_j = V8_j vs_b with K8, V8 e4m3 and one scale for a block b of tokens.
//
// K8 and V8 go from the cache to the tensor core as they are: S^T = K8 Q^T (M =
// the tile's 128 tokens, N = the rows, up to 64) and O^T = V8^T P^T (M = the head's
// elements), products of 8-bit types, twice the rate of 16-bit ones.  (Widening
// a tile to 16 bits first would write and read 64 KB of shared memory for each 32
// KB of cache, more than the 23 bytes a cycle and SM that HBM delivers leave time
// for.)  The other operands are cut into 8-bit parts whose products add up:
//   Q: a row times a power of two that brings its largest element to 128..256,
//     then 2 parts of e4m3 (bf16: exact but for elements below 2^-10 of the
//     largest, whose error is below 2^-18 of it) or 3 (fp16); all into one S.
//   P: rounded to fp16 (2^-11 of a weight, or 2^-32 of its row's reference), then 3
//     parts of e5m2, N columns of their own: each the nearest to what is left, the
//     second times 2^4, the third times 2^8. Together they are that fp16 number, to the bit, for
//     any up to 2^15, its subnormals too (without the 2^4 a weight 2^-20 of its row's largest
//     kept 8 bits, one of 2^-25 three).
// The scales never touch an operand: ks multiplies a score (a thread has a
// token), log2(vs) is added to it, and the sum takes its weights divided by vs.
// So a row's reference is the largest log2 of weight x vs.  A token of a small vs
// may lie far below it and still be most of the sum, whose value lies anywhere
// between 1 / vs of the least and of the largest scale.  With scales of 2^-80 .. 2^80 it is
// 2^-73 .. 2^119, and a weight that ex2 flushes (below 2^-126 of the reference) is below
// 2^-25 of it if vs >= kSmallScale; below that a token's weights for the sum are exponentials of
// their own.  Where a reference moves by up to 2 x 80 octaves and more, sums follow by the
// factor's root, twice.
//
// The tree's own nodes are a unit of their own with 16-bit operands, 64 nodes a
// tile in a tile's place.  Units (request, K/V head, row tile, chunk of the
// context or tree) are dealt to one persistent block an SM; each leaves its rows'
// unnormalised output, reference and sum, and a last kernel joins them.  A first
// one makes the parts of Q.
//
// Softmax: four groups of four warps, 16 rows a thread (thread = token = TMEM
// lane); 64 rows take all four, 32 or 16 rows two or one, and the groups then
// are teams that take the tiles in turn, each with references, sums and O of its own.
// (Two groups of 32 rows a thread, with twice the registers: 669 us for 8 x 64 at 32000 where
// four took 528 on the same lengths.  The next tile's scores fetched under this one's
// exponentials: 542 for 484, registers spilled.)
//
// Every other role has a warp, so that each one's chain of waits and issues (200 cycles
// a wait, 60 a product or copy) runs beside the others': with S and O issued by one
// warp, that warp took 2050 cycles a tile of 16 rows.  A tile of 32 KB is due every 1400 cycles at
// HBM's rate.  It takes 1750 for 4 rows (48 requests of up to 24001 tokens: 288 us, 260 to 299), where the
// loading warp is what bounds it, and 2700 for 64 rows (32 x 16 to 8000: 133 us, 123 to 138; 8 x 64 to 32000: 536
// us, 457 to 589; mean and range of six draws of the lengths, L2 flushed before each call), where the softmax
// chain does: wait, scores, vote, exponentials and parts, store.  For 32 x 16 that is some 85 us of
// the kernel's 125; units' borders, the trees' units and the blocks' uneven ends are the rest.
//
// Roles: warps 0-15 softmax and output, 16 the products S, 17 the products O, 18
// TMA for K and V and the scales, 19 the list of the block's units and their Q.  A
// softmax group's warps vote on every unit and tile whether a wait has expired, and
// leave together, so that their barriers stay complete.
#include <type_traits>

#include "launch.h"
#include "quant.cuh"
#include "ring.h"
#include "tma_map.h"
#include "tree_attn.cuh"

namespace dc {
namespace {

constexpr int kGroup = 128;    // softmax threads of a group
constexpr int kTreeNodes = kQuantNodes;  // nodes of a tree tile
constexpr int kAhead = kAheadUnits, kUnits = 32;  // units whose row factors and odd nodes are kept; whose description is
constexpr float kTop = 7.f;     // log2 of a weight at its row's reference
constexpr float kSmallScale = -28.f;  // log2 of a V scale, see above
constexpr float kGrow = kTop + kRescale;  // log2 of the largest weight: 2^15 fits fp16 and e5m2

struct QuantMaps {
  CUtensorMap k, v, k_new, v_new;
};

template <int D, int R, int NP>
struct Geom8 {
  // Softmax groups and rows of one.  The groups are teams that take the tiles in turn, R rows of a tile each.
  static constexpr int kGroups = 4, kCols = 64 / kGroups;
  static constexpr int kTeams = 64 / R, kParts = R / kCols;  // teams, groups of a team
  static constexpr int kScoreWarp = 4 * kGroups, kOutWarp = kScoreWarp + 1, kLoadWarp = kScoreWarp + 2,
                       kPrepWarp = kScoreWarp + 3, kThreads = 32 * (kScoreWarp + 4);
  // Registers a thread: 96 at launch (65,536 / 640 in steps of 8), then 4 x 104 + 64 = 5 x 96.
  static constexpr int kSoftRegs = 104, kOtherRegs = 64;
  static constexpr int kNS = 2 * kTeams, kNP = kTeams > 2 ? kTeams : 2;   // buffers of S and of P
  static constexpr uint32_t kTileBytes = kTile * D;        // a context tile of K or V; a tree tile takes the same
  // K's products run ahead of V's, and a tile's V stays until its weights are there: V's ring is the longer one
  static constexpr int kNK = D == 64 ? 5 : R == 64 && NP == 3 ? 2 : 3, kNV = D == 64 ? 8 : R == 64 ? 5 : 7;
  static constexpr uint32_t kQPart = R * D, kQBytes = NP * kQPart, kQTree = 2 * kQPart;  // a unit's Q in parts, in 16 bits
  static constexpr int kPAtoms = (3 * R + 63) / 64;        // 64-byte column blocks of P
  static constexpr uint32_t kPAtom = kTile * 64, kPBytes = kPAtoms * kPAtom;
  // V before P: products over 64 elements read as many rows of M past a V stage,
  // which have to be shared memory of ours (their results are not used); so do the
  // tree's products over 64 nodes past a K stage
  static constexpr uint32_t kK = 0, kV = kK + kNK * kTileBytes, kP = kV + kNV * kTileBytes;
  static constexpr uint32_t kQ = kP + kNP * kPBytes, kSmem = kQ + 2 * kQBytes;
  // TMEM columns, all 512: S^T of kNS tiles, O^T of each team's even and odd units
  static constexpr uint32_t kTmem = 512, kS = 0, kO = kNS * R;
  static_assert(kO + kTeams * 6 * R == kTmem, "");
  static_assert(kSmem + 1024 + 9216 <= 232448, "");
  // descriptors' high words: D-byte swizzle for K8, V8, Q8, 64 for P8
  static constexpr uint32_t kHi = D == 128 ? (1024 >> 4) | 1u << 14 | 2u << 29 : (512 >> 4) | 1u << 14 | 4u << 29;
  static constexpr uint32_t kHiP = (512 >> 4) | 1u << 14 | 4u << 29;
};

struct Bars8 {
  unsigned long long q_full[2], q_empty[2], k_full[8], k_empty[8], v_full[8], v_empty[8];
  unsigned long long s_full[8], s_free[8], p_full[4], pv_done[4], o_free[4][2], units[kUnits], factors[kAhead], done[2];
};

// D[tmem] (+)= A[smem] B[smem], 8-bit operands
template <uint32_t kHiA, uint32_t kHiB>
__device__ __forceinline__ void mma8(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "mov.b64 a, {%1, %5};\nmov.b64 b, {%2, %6};\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kHiA), "n"(kHiB)
      : "memory");
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead = 16) { return ((saddr & 0x3FFFFu) >> 4) | (lead >> 4) << 16; }

// Contiguous bytes (16 at a time) from global to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
template <int C>
__device__ __forceinline__ void tmem_st(uint32_t addr, const float (&v)[C]) {
#pragma unroll
  for (int i = 0; i < C; i += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(v[i]), "f"(v[i + 1]),
                 "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]), "f"(v[i + 6]), "f"(v[i + 7]), "r"(addr + i)
                 : "memory");
  tmem_st_wait();
}
__device__ __forceinline__ void soft_sync(int group) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ bool soft_any(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, %2, 128, p;\n"
      "selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(1 + group)
      : "memory");
  return r != 0;
}
// Maximum over the warp by one integer reduction; NaN counts as -inf.
__device__ __forceinline__ float warp_fmax(float x) {
  const int b = __float_as_int(x != x ? -INFINITY : x);
  const int m = __reduce_max_sync(DC_FULL_MASK, b ^ ((b >> 31) & 0x7FFFFFFF));
  return __int_as_float(m ^ ((m >> 31) & 0x7FFFFFFF));
}
// dst[k] = sum of v[k] over the warp: at each step a lane hands half of its columns to its partner.
template <int N>
__device__ __forceinline__ void warp_col_sums(float (&v)[N], float *dst) {
  const int lane = threadIdx.x & 31;
  int col = 0;  // first column this lane still holds
#pragma unroll
  for (int o = 16, n = N / 2; o > 0; o >>= 1, n >>= 1) {
    if (n > 0) {
      const bool up = lane & o;
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const float mine = up ? v[n + k] : v[k], other = up ? v[k] : v[n + k];
        v[k] = mine + __shfl_xor_sync(DC_FULL_MASK, other, o);
      }
      if (up) col += n;
    } else {
      v[0] += __shfl_xor_sync(DC_FULL_MASK, v[0], o);
    }
  }
  constexpr int kLeft = N >= 32 ? N / 32 : 1;
#pragma unroll
  for (int k = 0; k < kLeft; ++k) dst[col + k] = v[k];
}

__device__ __forceinline__ float lg2(float x) {  // of normal numbers
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ float rcp(float x) {  // within an ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A value that all lanes have alike, in a uniform register: what loops, addresses and descriptors
// are made of then stays out of the vector registers (a product or copy whose operands come
// from those took 60 to 140 cycles to issue).
__device__ __forceinline__ int uni(int x) { return __reduce_max_sync(DC_FULL_MASK, x); }
// Two fp32 values in one register pair.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 both(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 apart(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// A load of C columns in flight: the registers are the caller's after tmem_wait.
template <int C>
__device__ __forceinline__ void tmem_start(uint32_t addr, uint32_t (&r)[C]) {
#pragma unroll
  for (int i = 0; i < C; i += 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]),
                   "=r"(r[i + 6]), "=r"(r[i + 7])
                 : "r"(addr + i)
                 : "memory");
}
template <int C>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[C]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < C; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7])::"memory");
}
// bar_wait for up to three barriers at once: their tries overlap.
__device__ __forceinline__ bool bar_wait3(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, uint32_t c, uint32_t pc,
                                          volatile int *abort, int *err) {
  unsigned long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    const bool x = mbar_try(a, pa), y = mbar_try(b, pb), z = mbar_try(c, pc);
    if (x & y & z) return true;
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

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two fp16 values to the nearest with three significant bits: e5m2 in their upper bytes.
__device__ __forceinline__ uint32_t top_bytes(uint32_t x) { return (x + 0x00800080u) & 0xFF00FF00u; }
// Four weights' three parts, a byte each.
__device__ __forceinline__ void split4(const float (&e)[4], uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  uint32_t h[2], m[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t p = pack2<true>(e[2 * i], e[2 * i + 1]);
    h[i] = top_bytes(p);
    const uint32_t r = hmul2(hsub2(p, h[i]), 0x4C004C00u);  // 2^4
    m[i] = top_bytes(r);
    l[i] = hmul2(hsub2(r, m[i]), 0x4C004C00u) + 0x00800080u;
  }
  hi = __byte_perm(h[0], h[1], 0x7531), mid = __byte_perm(m[0], m[1], 0x7531), lo = __byte_perm(l[0], l[1], 0x7531);
}

// ---------------------------------------------------------------- units
struct QuantUnit {
  int n, h, mt, slot;        // request, K/V head, row tile, chunk (the tree comes last)
  int ctx, len;              // clamped lengths
  int tile0, ntiles;         // tiles of 128 context tokens, or of 64 nodes (0: no live rows)
  bool tree;
};

// Lengths of request n, clamped, and the chunks of its context (0 without live nodes).
__device__ __forceinline__ int context_chunks(const QuantAttnParams &p, int n, int &ctx, int &len, bool flag = false) {
  const TreeAttnParams &t = p.t;
  const int capacity = t.max_pages << t.page_shift;
  ctx = t.ctx_len[n];
  len = t.tree_len ? t.tree_len[n] : t.T;
  if ((ctx < 0 || ctx > capacity || len < 0 || len > t.T) && flag) atomicOr(t.err, kErrBadLength);
  ctx = min(max(ctx, 0), capacity);
  len = len < 0 ? 0 : min(len, t.T);
  const int nt = len > 0 ? (ctx + kTile - 1) / kTile : 0;
  const int per = quant_chunk_tiles(nt, p.items, p.sms, p.chunk_cap);
  return (nt + per - 1) / per;
}

// This block's units, warp by warp without communication: first the contexts'
// chunks, 32 requests' at a time in the lanes and those with the largest chunks
// first, then the trees; dealt to the blocks to and fro.
struct QuantUnits {
  const QuantAttnParams &p;
  int lane, base = 0, n0 = 0, round = 0, req = 0;
  bool tree = false;
  int ctx = 0, len = 0, chunks = 0, before = 0, upto = 0, window = 0;
  __device__ QuantUnits(const QuantAttnParams &p_, bool flag) : p(p_), lane(threadIdx.x & 31) { load(flag); }
  __device__ void load(bool flag) {
    req = n0 + lane;
    chunks = ctx = len = 0;
    if (req < p.t.N) chunks = context_chunks(p, req, ctx, len, flag && !tree);
    scan();
    if (tree || (p.t.N <= 32 && window <= (int)gridDim.x)) return;  // units of one size, or one a block at most
    // sort the lanes by their tiles a chunk
    const int key = chunks > 0 ? ((ctx + kTile - 1) / kTile + chunks - 1) / chunks : req < p.t.N ? 0 : -1;
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
    const int count = (tree ? (len > 0 ? 1 : 0) : chunks) * p.t.kv_heads * p.mtiles;
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
  __device__ bool next(QuantUnit &w, bool flag = false) {
    const int u = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    while (u - base >= window) {
      base += window;
      n0 += 32;
      if (n0 >= p.t.N) {
        if (tree) return false;
        tree = true, n0 = 0;
      }
      load(flag);
    }
    const int rel = u - base;
    const int src = __ffs(__ballot_sync(DC_FULL_MASK, upto > rel)) - 1;
    int i = rel - __shfl_sync(DC_FULL_MASK, before, src);
    w.n = __shfl_sync(DC_FULL_MASK, req, src);
    w.ctx = __shfl_sync(DC_FULL_MASK, ctx, src);
    w.len = __shfl_sync(DC_FULL_MASK, len, src);
    const int nc = __shfl_sync(DC_FULL_MASK, chunks, src);
    w.tree = tree;
    w.mt = i % p.mtiles, i /= p.mtiles;
    w.h = i % p.t.kv_heads;
    const int chunk = i / p.t.kv_heads;
    w.slot = tree ? nc : chunk;
    if (w.mt * p.R >= w.len * p.t.group) {
      w.tile0 = w.ntiles = 0;
    } else if (tree) {
      w.tile0 = 0, w.ntiles = (w.len + kTreeNodes - 1) / kTreeNodes;
    } else {
      const int nt = (w.ctx + kTile - 1) / kTile;
      w.tile0 = (int)((int64_t)nt * chunk / nc);  // chunks as even as they come
      w.ntiles = (int)((int64_t)nt * (chunk + 1) / nc) - w.tile0;
    }
    ++round;
    return true;
  }
};

// A node's row of V before the product reads it: zeros past the tree's end; a
// node's infinities and NaN stay out of the product (they would reach nodes that do
// not see it) and are added to the output of those that do.  Returns whether it had any.
template <int D, bool F16>
__device__ __forceinline__ bool clean_node(uint8_t *row, bool there) {
  bool bad = false;
#pragma unroll 2
  for (int e = 0; e < D / 8; ++e) {
    uint4 *v = reinterpret_cast<uint4 *>(row + (e >> 3) * (kTreeNodes * 128) + (e & 7) * 16);
    if (!there) {
      *v = make_uint4(0, 0, 0, 0);
      continue;
    }
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
  return bad;
}

template <int D, int R, bool F16>
__global__ void __launch_bounds__(Geom8<D, R, F16 ? 3 : 2>::kThreads, 1)
k_quant_attn(const QuantAttnParams p, const __grid_constant__ QuantMaps maps) {
  constexpr int NP = F16 ? 3 : 2;
  using G = Geom8<D, R, NP>;
  const TreeAttnParams &t = p.t;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) Bars8 b;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(16) float s_factor[kAhead][R];      // score per unit of S, log2 (the row's power of two and p.scale)
  __shared__ QuantUnit s_unit[kUnits];                     // the block's units in turn; ntiles 0: the end
  __shared__ uint32_t s_odd[kAhead][8];                    // tree units: nodes whose V holds an infinity or NaN
  __shared__ float s_scale[G::kNV][2][8];                  // a V stage's tile: K and V scales of its blocks
  // of each group: kTop less its rows' references (what the scores are added to), rescale factors, and what
  // its warps put together
  __shared__ __align__(16) float s_nref[G::kGroups][G::kCols], s_f[G::kGroups][G::kCols], s_part[G::kGroups][4][G::kCols];
  const int tid = threadIdx.x, warp = __shfl_sync(DC_FULL_MASK, tid >> 5, 0), lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&b.q_full[i]), 1), mbar_init(smem_u32(&b.q_empty[i]), 1);
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&b.k_full[i]), 1), mbar_init(smem_u32(&b.k_empty[i]), 1);
      mbar_init(smem_u32(&b.v_full[i]), 33), mbar_init(smem_u32(&b.v_empty[i]), 1);
      mbar_init(smem_u32(&b.s_full[i]), 1), mbar_init(smem_u32(&b.s_free[i]), G::kParts * 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&b.p_full[i]), G::kParts * 4), mbar_init(smem_u32(&b.pv_done[i]), 1);
      for (int j = 0; j < 2; ++j) mbar_init(smem_u32(&b.o_free[i][j]), G::kParts * 4);
    }
    for (int i = 0; i < kAhead; ++i) mbar_init(smem_u32(&b.factors[i]), 1);
    for (int i = 0; i < kUnits; ++i) mbar_init(smem_u32(&b.units[i]), 1);
    mbar_init(smem_u32(&b.done[0]), 1), mbar_init(smem_u32(&b.done[1]), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 64) s_nref[tid / G::kCols][tid % G::kCols] = -kNone;
  if (warp == G::kLoadWarp && lane < 4)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k + lane)) : "memory");
  if (warp == G::kScoreWarp) tmem_alloc(smem_u32(&s_tmem), G::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(DC_FULL_MASK, s_tmem, 0);
  pdl_trigger();

  int g = 0;  // tiles that this role has begun (of the list's warp: units whose Q it has)
  // Unit number `unit` as the preparing warp has published it.
  const auto unit_at = [&](int unit) -> const QuantUnit & { return s_unit[unit & (kUnits - 1)]; };
  const auto units_bar = [&](int unit) { return smem_u32(&b.units[unit & (kUnits - 1)]); };
  const auto factors_bar = [&](int unit) { return smem_u32(&b.factors[unit & (kAhead - 1)]); };
  if (warp >= G::kScoreWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kOtherRegs));
    if (warp == G::kLoadWarp) {
      // ------------------------------------------------------------ TMA for K and V, the scales
      const int page_size = 1 << t.page_shift, box_shift = min(t.page_shift, 7), box = 1 << box_shift, boxes = kTile >> box_shift;
      const uint32_t box_bytes = box * D;
      // lanes 0-7 fetch K's scales of a tile, 8-15 V's: block j of the tile, in box box_j; its place in its
      // page is its place in the box where a box is a page
      const int j = lane & 7, tok_j = j << p.scale_shift, box_j = min(tok_j, kTile - 1) >> box_shift;
      const float *scale = lane < 8 ? p.k_scale : p.v_scale;
      const int64_t sp = lane < 8 ? p.ks_sp : p.vs_sp, sb = lane < 8 ? p.ks_sb : p.vs_sb, ss = lane < 8 ? p.ks_sh : p.vs_sh;
      scale += ((tok_j & (box - 1)) >> p.scale_shift) * sb;
      bool ok = true;
      int ks = 0, k_phase = 1, vs = 0, v_phase = 1;  // (a wait for phase 1 of a new barrier is over at once)
      for (int unit = 0; ok; ++unit) {
        ok = __all_sync(DC_FULL_MASK, bar_wait(units_bar(unit), (unit / kUnits) & 1, &s_abort, t.err));
        if (!ok) break;
        const QuantUnit &u = unit_at(unit);
        const int ntiles = uni(u.ntiles), n = uni(u.n), h = uni(u.h), tile0 = uni(u.tile0), ctx = uni(u.ctx);
        const bool tree = uni(u.tree);
        if (ntiles == 0) break;
        const float *scale_h = scale + h * ss;
        const int32_t *table = t.page_table + n * t.pt_stride;
        const int end = tree ? 0 : min(ctx, (tile0 + ntiles) * kTile);
        auto pages_from = [&](int tok) {  // lane l: page of the l-th box from token `tok` on
          tok += lane * box;
          int page = 0;
          if (tok < end) page = __ldg(table + (tok >> t.page_shift));
          return page;
        };
        int tok0 = tile0 * kTile, at = 0;
        int page = pages_from(tok0), page_next = pages_from(tok0 + 32 * box);
        for (int i = 0; i < ntiles; ++i, ++g, tok0 += kTile) {
          if (at == 32) {
            at = 0, page = page_next;
            page_next = pages_from(tok0 + 32 * box);
          }
          if (at == 0 && (page < 0 || page >= t.num_pages)) {
            atomicOr(t.err, kErrBadPage);
            page = 0;
          }
          const uint32_t k_bar = smem_u32(&b.k_full[ks]), v_bar = smem_u32(&b.v_full[vs]);
          const uint32_t k_empty = smem_u32(&b.k_empty[ks]);
          ok = __all_sync(DC_FULL_MASK, bar_wait3(k_empty, k_phase, smem_u32(&b.v_empty[vs]), v_phase, k_empty, k_phase,
                                                  &s_abort, t.err));
          if (!ok) break;
          const uint32_t k_dst = sbase + G::kK + ks * G::kTileBytes, v_dst = sbase + G::kV + vs * G::kTileBytes;
          if (tree) {
            const int bytes = (D / 64) * 128 * t.tree_box;
            if (elect_one()) {
              mbar_arrive_expect_tx(k_bar, bytes);
              asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(v_bar), "r"(bytes) : "memory");
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                tma_load_4d(k_dst + c * kTreeNodes * 128, &maps.k_new, c * 64, i * kTreeNodes, h, n, k_bar);
                tma_load_4d(v_dst + c * kTreeNodes * 128, &maps.v_new, c * 64, i * kTreeNodes, h, n, v_bar);
              }
              asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 33;" ::"r"(v_bar) : "memory");
            }
            __syncwarp();
          } else {
            const int used = min(boxes, (end - tok0 + box - 1) >> box_shift);  // copies of the tile
            const int slot = tok0 & (page_size - 1);
            // (the pages first, then all copies by one lane: a shuffle and an election between copies cost 130 cycles each)
            auto copies = [&](auto number) {
              constexpr int kBoxes = decltype(number)::value;
              int pg[kBoxes];
#pragma unroll
              for (int r = 0; r < kBoxes; ++r) pg[r] = uni(lane == at + r ? page : 0);
              if (elect_one()) {
                mbar_arrive_expect_tx(k_bar, used * box_bytes);
                mbar_arrive_expect_tx(v_bar, used * box_bytes);
                if (used == kBoxes) {
#pragma unroll
                  for (int r = 0; r < kBoxes; ++r) {
                    tma_load_4d(k_dst + r * (G::kTileBytes / kBoxes), &maps.k, 0, slot, h, pg[r], k_bar);
                    tma_load_4d(v_dst + r * (G::kTileBytes / kBoxes), &maps.v, 0, slot, h, pg[r], v_bar);
                  }
                } else {
#pragma unroll
                  for (int r = 0; r < kBoxes; ++r)
                    if (r < used) {
                      tma_load_4d(k_dst + r * (G::kTileBytes / kBoxes), &maps.k, 0, slot, h, pg[r], k_bar);
                      tma_load_4d(v_dst + r * (G::kTileBytes / kBoxes), &maps.v, 0, slot, h, pg[r], v_bar);
                    }
                }
              }
              __syncwarp();
            };
            if (boxes == 1) copies(std::integral_constant<int, 1>());
            else if (boxes == 2) copies(std::integral_constant<int, 2>());
            else if (boxes == 4) copies(std::integral_constant<int, 4>());
            else copies(std::integral_constant<int, 8>());
            const int pg_j = __shfl_sync(DC_FULL_MASK, page, at + box_j);
            if (lane < 16 && tok_j < kTile && tok0 + tok_j < end) {
              const float *src = scale_h + pg_j * sp;
              if (page_size > kTile) src += (slot >> p.scale_shift) * sb;
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&s_scale[vs][lane >> 3][j])), "l"(src)
                           : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(v_bar) : "memory");
            at += boxes;
          }
          if (++ks == G::kNK) ks = 0, k_phase ^= 1;
          if (++vs == G::kNV) vs = 0, v_phase ^= 1;
        }
      }
    } else if (warp == G::kPrepWarp) {
      // ------------------------------------------------------------ units, their Q
      const bool flag = blockIdx.x == 0;
      QuantUnits it(p, flag);
      QuantUnit w;
      bool ok = true, more = true;
      int made = 0;
      pdl_wait();  // k_quant_q's Q
      asm volatile("fence.proxy.async.global;" ::: "memory");
      for (int unit = 0; ok; ++unit) {
        const int qb = unit & 1, slot = unit & (kAhead - 1);
        // Units are published ahead of their Q, up to nine: the loads of short ones run that far ahead.
        for (int k = 0; k < 2 && more && made <= unit + 8; ++k) {
          do more = it.next(w, flag);
          while (more && w.ntiles == 0);
          if (!more) w.ntiles = 0;
          if (lane == 0) {
            s_unit[made & (kUnits - 1)] = w;
            mbar_arrive(units_bar(made));
          }
          ++made;
          __syncwarp();
        }
        if (unit >= 2) ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.q_empty[qb]), ((unit >> 1) - 1) & 1, &s_abort, t.err));
        if (!ok) break;
        const QuantUnit &u = unit_at(unit);
        if (u.ntiles == 0) {  // the end
          if (lane == 0) mbar_arrive(factors_bar(unit));
          break;
        }
        if (lane == 0) {
          const uint8_t *src = p.q_parts + (((int64_t)u.n * t.kv_heads + u.h) * p.mtiles + u.mt) * quant_q_bytes(NP, R, D);
          const uint32_t bytes = u.tree ? G::kQTree : G::kQBytes, q_bar = smem_u32(&b.q_full[qb]);
          mbar_arrive_expect_tx(q_bar, bytes);
          bulk_load(sbase + G::kQ + qb * G::kQBytes, src + (u.tree ? G::kQBytes : 0), bytes, q_bar);
          mbar_arrive_expect_tx(factors_bar(unit), R * 4);
          bulk_load(smem_u32(s_factor[slot]), src + G::kQBytes + G::kQTree + (u.tree ? R * 4 : 0), R * 4, factors_bar(unit));
        }
        ++g;
        __syncwarp();
      }
    } else if (warp == G::kScoreWarp) {
      // ------------------------------------------------------------ tensor core: S^T = K Q^T
      constexpr uint32_t kId = (1u << 4) | (8u << 24) | (uint32_t)(R >> 3) << 17;  // fp32 += e4m3 e4m3, M = 128, N = R
      constexpr uint32_t kId16 = F16 ? idesc_f16(128, R) : idesc_bf16(128, R);
      bool ok = true;
      int ks = 0, k_phase = 0;
      for (int unit = 0; ok; ++unit) {
        const int qb = unit & 1;
        ok = __all_sync(DC_FULL_MASK, bar_wait(units_bar(unit), (unit / kUnits) & 1, &s_abort, t.err));
        if (!ok) break;
        const int ntiles = uni(unit_at(unit).ntiles);
        const bool tree = uni(unit_at(unit).tree);
        if (ntiles == 0) break;
        ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.q_full[qb]), (unit >> 1) & 1, &s_abort, t.err));
        if (!ok) break;
        const uint32_t sq = desc_lo(sbase + G::kQ + qb * G::kQBytes);
        for (int i = 0; i < ntiles; ++i, ++g) {
          const int sb = g % G::kNS;
          const uint32_t k_bar = smem_u32(&b.k_full[ks]);
          ok = __all_sync(DC_FULL_MASK, bar_wait3(k_bar, k_phase, k_bar, k_phase, g >= G::kNS ? smem_u32(&b.s_free[sb]) : k_bar,
                                                  g >= G::kNS ? (g / G::kNS - 1) & 1 : k_phase, &s_abort, t.err));
          if (!ok) break;
          tc_fence_after();
          const uint32_t sk = desc_lo(sbase + G::kK + ks * G::kTileBytes), to = tmem + G::kS + sb * R;
          if (elect_one()) {
            if (tree) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                mma_ss(to, sk + (((k >> 2) * (kTreeNodes * 128) + (k & 3) * 32) >> 4),
                       sq + (((k >> 2) * (R * 128) + (k & 3) * 32) >> 4), kId16, k > 0 ? 1u : 0u);
            } else {
#pragma unroll
              for (int x = 0; x < NP; ++x)
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                  mma8<G::kHi, G::kHi>(to, sk + k * 2, sq + ((x * G::kQPart) >> 4) + k * 2, kId, (x > 0 || k > 0) ? 1u : 0u);
            }
            mma_commit(smem_u32(&b.s_full[sb]));
            mma_commit(smem_u32(&b.k_empty[ks]));
            if (i == ntiles - 1) mma_commit(smem_u32(&b.q_empty[qb]));
          }
          __syncwarp();
          if (++ks == G::kNK) ks = 0, k_phase ^= 1;
        }
      }
      if (elect_one()) {  // the lane that issued: nothing is in flight when the block frees its TMEM
        mma_commit(smem_u32(&b.done[0]));
        mbar_drain(smem_u32(&b.done[0]), 0);
      }
      __syncwarp();
    } else if (warp == G::kOutWarp) {
      // ------------------------------------------------------------ tensor core: O^T += V^T P^T
      constexpr uint32_t kId =  // B e5m2; both M- and N-major
          (1u << 4) | (8u << 24) | (1u << 10) | (1u << 15) | (1u << 16) | (uint32_t)(3 * R >> 3) << 17;
      constexpr uint32_t kId16 = (F16 ? idesc_f16(128, R) : idesc_bf16(128, R)) | (1u << 15) | (1u << 16);
      bool ok = true;
      int vs = 0, v_phase = 0;
      int begun[G::kTeams] = {};  // units that each team has begun
      for (int unit = 0; ok; ++unit) {
        ok = __all_sync(DC_FULL_MASK, bar_wait(units_bar(unit), (unit / kUnits) & 1, &s_abort, t.err));
        if (!ok) break;
        const int ntiles = uni(unit_at(unit).ntiles);
        const bool tree = uni(unit_at(unit).tree);
        if (ntiles == 0) break;
        for (int i = 0; i < ntiles; ++i, ++g) {
          const int team = g % G::kTeams, pb = g % G::kNP;
          const bool first = i < G::kTeams;
          int mine = 0;
#pragma unroll
          for (int k = 0; k < G::kTeams; ++k)
            if (k == team) mine = (begun[k] += first) - 1;
          const uint32_t v_bar = smem_u32(&b.v_full[vs]);
          const bool wait_o = first && mine >= 2;
          ok = __all_sync(DC_FULL_MASK, bar_wait3(v_bar, v_phase, smem_u32(&b.p_full[pb]), (g / G::kNP) & 1,
                                                  wait_o ? smem_u32(&b.o_free[team][mine & 1]) : v_bar,
                                                  wait_o ? ((mine >> 1) - 1) & 1 : v_phase, &s_abort, t.err));
          if (!ok) break;
          tc_fence_after();
          const uint32_t to = tmem + G::kO + (team * 2 + (mine & 1)) * 3 * R;
          const uint32_t sv = sbase + G::kV + vs * G::kTileBytes, sp = sbase + G::kP + pb * G::kPBytes;
          const uint32_t a = desc_lo(sv, tree ? kTreeNodes * 128 : G::kTileBytes), bd = desc_lo(sp, tree ? 16 : G::kPAtom);
          if (elect_one()) {
            if (tree) {
#pragma unroll
              for (int k = 0; k < kTreeNodes / 16; ++k)
                mma_ss(to, a + k * (2048 >> 4), bd + k * (2048 >> 4), kId16, (!first || k > 0) ? 1u : 0u);
            } else {
#pragma unroll
              for (int k = 0; k < kTile / 32; ++k)
                mma8<G::kHi, G::kHiP>(to, a + k * (32 * D >> 4), bd + k * (2048 >> 4), kId, (!first || k > 0) ? 1u : 0u);
            }
            mma_commit(smem_u32(&b.v_empty[vs]));
            mma_commit(smem_u32(&b.pv_done[pb]));
          }
          __syncwarp();
          if (++vs == G::kNV) vs = 0, v_phase ^= 1;
        }
      }
      if (elect_one()) {
        mma_commit(smem_u32(&b.done[1]));
        mbar_drain(smem_u32(&b.done[1]), 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kSoftRegs));
    // ------------------------------------------------------------ softmax, output
    // Each team of groups takes every kTeams-th tile, with references, sums and O of its own; a unit's
    // tiles i, i + kTeams, ... make a partial result of their own, whichever team has them.
    constexpr int C = G::kCols;
    const int group = warp >> 2, quad = warp & 3, tok = tid & (kGroup - 1);
    const int team = group / G::kParts, col0 = group % G::kParts * C;  // this group's rows: columns col0 .. col0 + C - 1
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + col0;
    float *const nref_of = s_nref[group], *const f_of = s_f[group];
    uint32_t(*const s_word)[C] = reinterpret_cast<uint32_t(*)[C]>(s_part[group]);  // mask words (a tile's step between uses of s_part)
    bool ok = true;
    auto wait = [&](unsigned long long *bar, int phase) {
      if (ok) ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(bar), phase & 1, &s_abort, t.err));
    };
    // rows of partial result j of a unit
    auto slot_of = [&](const QuantUnit &u, int j) {
      return (((((int64_t)u.n * t.kv_heads + u.h) * p.mtiles + u.mt) * p.slots + u.slot) * G::kTeams + j) * R + col0;
    };
    // A unit's output, unnormalised, leaves for the join after the team's first tile of
    // the unit that follows, whose products go to the other half of its O, so that the
    // tensor core and the copies go on meanwhile.
    int done_g = -1, done_unit = 0, done_i = 0;  // that unit's last tile of this team (-1: none), its number, the team's first tile of it
    int begun = 0;                               // units that this team has begun
    auto finish = [&](int par) {
      // (with a P buffer a team the tile after it has waited for that product already)
      if (G::kNP > G::kTeams) wait(&b.pv_done[done_g % G::kNP], done_g / G::kNP);
      tc_fence_after();
      const QuantUnit &u = unit_at(done_unit);
      const uint32_t from = trow + G::kO + (team * 2 + par) * 3 * R;
      float *part = p.part_o + slot_of(u, done_i) * D + tok;  // [row][D]
      const bool tree = u.tree;
#pragma unroll 1
      for (int k0 = 0; k0 < C; k0 += 8) {
        uint32_t x[8], y[8], z[8];
        tmem_start<8>(from + k0, x);
        if (!tree) tmem_start<8>(from + R + k0, y), tmem_start<8>(from + 2 * R + k0, z);
        tmem_wait<8>(x);
        if (!tree) {
          tmem_wait<8>(y), tmem_wait<8>(z);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            x[k] = __float_as_uint(fmaf(__uint_as_float(z[k]), 0.00390625f,
                                        fmaf(__uint_as_float(y[k]), 0.0625f, __uint_as_float(x[k]))));
        }
        if (tok < D && ok) {
#pragma unroll
          for (int k = 0; k < 8; ++k) part[(k0 + k) * D] = __uint_as_float(x[k]);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&b.o_free[team][par]));
      if (tok < D && ok && tree) {
        // infinities and NaN of this team's nodes that a row sees
#pragma unroll 1
        for (int q = done_i * 2; q < (u.len + 31) / 32; q += (q & 1) ? 2 * G::kTeams - 1 : 1)
#pragma unroll 1
          for (uint32_t r = s_odd[done_unit & (kAhead - 1)][q]; r; r &= r - 1) {
              const int nd = __ffs(r) - 1;
              const uint32_t e = t.v_new[u.n * t.vn_sn + (q * 32 + nd) * t.vn_st + u.h * t.vn_sh + tok];
              if (!nonfinite2<F16>(e)) continue;
#pragma unroll 1
              for (int k = 0; k < C; ++k)
                if ((tree_sees(t, u.n, u.len, (u.mt * R + col0 + k) / t.group, q) >> nd) & 1u) part[k * D] += unpack_lo<F16>(e);
            }
      }
      __syncwarp();
      done_g = -1;
    };
    for (int unit = 0;; ++unit) {
      if (ok) ok = __all_sync(DC_FULL_MASK, bar_wait(factors_bar(unit), (unit / kAhead) & 1, &s_abort, t.err));
      // the group's warps leave together when a wait has expired
      if (soft_any(group, !ok)) {
        ok = false;
        break;
      }
      const QuantUnit &u = unit_at(unit);
      const int ntiles = uni(u.ntiles), tile0 = uni(u.tile0);
      const bool tree = uni(u.tree);
      const int end = uni(tree ? u.len : u.ctx);
      if (ntiles == 0) break;
      const int first = (team + G::kTeams - g % G::kTeams) % G::kTeams;  // the team's first tile of the unit
      if (first >= ntiles) {  // none: an empty partial result
        if (tok < C) p.part_ml[slot_of(u, first) + tok] = make_float2(kNone, 0.f);
        g += ntiles;
        continue;
      }
      const float *factor = s_factor[unit & (kAhead - 1)] + col0;
      const uint32_t to_o = trow + G::kO + (team * 2 + (begun & 1)) * 3 * R;
      f32x2 l[C / 2];  // the rows' sums over this thread's tokens
#pragma unroll
      for (int k = 0; k < C / 2; ++k) l[k] = 0ull;
      bool leave = false;
      int x_g = 0;  // this tile
      for (int i = first; i < ntiles; i += G::kTeams) {
        x_g = g + i;
        const int vs = x_g % G::kNV, sb = x_g % G::kNS, pb = x_g % G::kNP;
        const int width = tree ? kTreeNodes : kTile, tok0 = (tile0 + i) * width, valid = min(width, end - tok0);
        {
          // S; V with its scales (and the tree's odd nodes); P's buffer is free
          const uint32_t s_bar = smem_u32(&b.s_full[sb]), s_phase = (x_g / G::kNS) & 1;
          const bool used = x_g >= G::kNP;
          if (ok)
            ok = __all_sync(DC_FULL_MASK,
                            bar_wait3(s_bar, s_phase, smem_u32(&b.v_full[vs]), (x_g / G::kNV) & 1,
                                      used ? smem_u32(&b.pv_done[pb]) : s_bar, used ? (x_g / G::kNP - 1) & 1 : s_phase,
                                      &s_abort, t.err));
        }
        tc_fence_after();
        uint32_t raw[C];
        tmem_start<C>(trow + G::kS + sb * R, raw);  // in flight under the scales
        float ks = 1.f, lvs = 0.f, inv = 1.f;
        if (!tree) {
          if (tok < valid) {
            const int blk = tok >> p.scale_shift;
            ks = s_scale[vs][0][blk];
            const float f = s_scale[vs][1][blk];
            lvs = lg2(f), inv = lvs < kSmallScale ? 0.f : rcp(f);
          } else if (col0 == 0 && ok) {
            // past the end lies what a page or a copy left: zeros in its place, since a zero weight does not cancel NaN
            uint4 *row = reinterpret_cast<uint4 *>(smem + G::kV + vs * G::kTileBytes + tok * D);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) row[e] = make_uint4(0, 0, 0, 0);
          }
        } else {
          if (col0 == 0 && quad < kTreeNodes / 32) {
            bool bad = false;
            if (ok) bad = clean_node<D, F16>(smem + G::kV + vs * G::kTileBytes + tok * 128, tok < valid);
            const uint32_t bits = __ballot_sync(DC_FULL_MASK, bad);
            if (lane == 0) s_odd[unit & (kAhead - 1)][i * 2 + quad] = bits;
          }
          // this warp's 32 nodes are one word of each row's mask: lane k fetches row k's
          if (lane < C)
            s_word[quad][lane] = quad < kTreeNodes / 32 ? tree_sees(t, u.n, u.len, (u.mt * R + col0 + lane) / t.group, tok0 / 32 + quad) : 0u;
          __syncwarp();
        }
        const bool mask = tree || valid < kTile;
        const f32x2 ks2 = both(ks, ks), lvs2 = both(lvs, lvs);
        f32x2 x[C / 2];
        // log2 of weight x vs
        auto scaled = [&] {
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(factor + k);
            x[k / 2] = fma2(mul2(both(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1])), ks2), both(f.x, f.y), lvs2);
            x[k / 2 + 1] = fma2(mul2(both(__uint_as_float(raw[k + 2]), __uint_as_float(raw[k + 3])), ks2), both(f.z, f.w), lvs2);
          }
          if (!mask) return;
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const uint4 word = *reinterpret_cast<const uint4 *>(&s_word[quad][k]);
            const bool in = tree || tok < valid;  // (the words are of the tree alone)
            const float2 a = apart(x[k / 2]), c = apart(x[k / 2 + 1]);
            auto sees = [&](uint32_t m) { return tree ? (m >> lane) & 1u : (uint32_t)in; };
            x[k / 2] = both(sees(word.x) ? a.x : -INFINITY, sees(word.y) ? a.y : -INFINITY);
            x[k / 2 + 1] = both(sees(word.z) ? c.x : -INFINITY, sees(word.w) ? c.y : -INFINITY);
          }
        };
        float grow;
        auto against = [&] {  // the exponents against the references, in x's place
          float g0 = -INFINITY, g1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const float4 r = *reinterpret_cast<const float4 *>(nref_of + k);
            x[k / 2] = add2(x[k / 2], both(r.x, r.y)), x[k / 2 + 1] = add2(x[k / 2 + 1], both(r.z, r.w));
            const float2 a = apart(x[k / 2]), c = apart(x[k / 2 + 1]);
            g0 = max3(g0, a.x, a.y), g1 = max3(g1, c.x, c.y);
          }
          grow = fmaxf(g0, g1);
        };
        tmem_wait<C>(raw);
        scaled();
        // The group's warps vote on every tile but a unit's first, which gives the references: whether a
        // score has outgrown its row's reference, or a wait has expired, when all leave together.
        bool renew = i == first;
        if (!renew) {
          against();
          if (soft_any(group, grow > kGrow || !ok)) {
            if (soft_any(group, !ok)) {
              leave = true, ok = false;
              break;
            }
            renew = true;
            tmem_start<C>(trow + G::kS + sb * R, raw);
            tmem_wait<C>(raw);
            scaled();
          }
        }
        if (renew) {
          // references from the rows' maxima over the tile; l and O^T follow
          __syncwarp();  // (the mask's words have been read)
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const float2 a = apart(x[k / 2]), c = apart(x[k / 2 + 1]);
            const float m0 = warp_fmax(a.x), m1 = warp_fmax(a.y), m2 = warp_fmax(c.x), m3 = warp_fmax(c.y);
            if (lane == 0) *reinterpret_cast<float4 *>(&s_part[group][quad][k]) = make_float4(m0, m1, m2, m3);
          }
          soft_sync(group);
          if (tok < C) {
            const float m = fmaxf(fmaxf(s_part[group][0][tok], s_part[group][1][tok]),
                                  fmaxf(s_part[group][2][tok], s_part[group][3][tok]));
            const float old = nref_of[tok];
            const bool grown = m + old > kGrow;  // (the others stay: a row's result hangs on its own scores)
            nref_of[tok] = grown ? kTop - m : old;
            f_of[tok] = grown ? ex2(0.5f * (kTop - m - old)) : 1.f;  // (the factor's root)
          }
          soft_sync(group);
          if (i > first) {
#pragma unroll
            for (int k = 0; k < C / 2; ++k) {
              const f32x2 f = both(f_of[2 * k], f_of[2 * k + 1]);
              l[k] = mul2(mul2(l[k], f), f);
            }
            // this team's last product
            wait(&b.pv_done[(x_g - G::kTeams) % G::kNP], (x_g - G::kTeams) / G::kNP);
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < (tree ? 1 : 3); ++part)
#pragma unroll 1
              for (int k0 = 0; k0 < C; k0 += 8) {
                float o[8];
                tmem_ld<8>(to_o + part * R + k0, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= f_of[k0 + k] * f_of[k0 + k];
                tmem_st<8>(to_o + part * R + k0, o);
              }
          }
          // (the words anew: s_part took their place)
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const float4 r = *reinterpret_cast<const float4 *>(nref_of + k);
            x[k / 2] = add2(x[k / 2], both(r.x, r.y)), x[k / 2 + 1] = add2(x[k / 2 + 1], both(r.z, r.w));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&b.s_free[sb]));
        uint8_t *pbuf = smem + G::kP + pb * G::kPBytes;
        const f32x2 inv2 = both(inv, inv);
        if (lvs < kSmallScale) {  // (rare: V below 2^-19, blocks of zeros; inv is 0)
#pragma unroll
          for (int k = 0; k < C / 2; ++k) {
            const float2 v = apart(x[k]);
            l[k] = add2(l[k], both(ex2(v.x - lvs), ex2(v.y - lvs)));
          }
        }
        if (tree) {
#pragma unroll
          for (int k = 0; k < C; k += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int y = 0; y < 8; y += 2) {
              const float2 v = apart(x[(k + y) / 2]);
              const float e0 = ex2(v.x), e1 = ex2(v.y);
              l[(k + y) / 2] = add2(l[(k + y) / 2], both(e0, e1));
              pk[y / 2] = pack2<F16>(e0, e1);
            }
            if (tok < kTreeNodes)
              *reinterpret_cast<uint4 *>(pbuf + tok * 128 + ((((col0 + k) >> 3) ^ (tok & 7)) << 4)) =
                  make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        } else {
#pragma unroll
          for (int k0 = 0; k0 < C; k0 += 16) {  // rows of a store
            uint32_t parts[3][4];
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              float e[4];
#pragma unroll
              for (int z = 0; z < 4; z += 2) {
                const int at = (k0 + k + z) / 2;
                const float2 v = apart(x[at]);
                e[z] = ex2(v.x), e[z + 1] = ex2(v.y);
                l[at] = fma2(both(e[z], e[z + 1]), inv2, l[at]);
              }
              split4(e, parts[0][k / 4], parts[1][k / 4], parts[2][k / 4]);
            }
#pragma unroll
            for (int y = 0; y < 3; ++y) {
              const int col = y * R + col0 + k0;  // of the parts side by side
              *reinterpret_cast<uint4 *>(pbuf + (col >> 6) * G::kPAtom + tok * 64 + ((((col & 63) >> 4) ^ ((tok >> 1) & 3)) << 4)) =
                  make_uint4(parts[y][0], parts[y][1], parts[y][2], parts[y][3]);
            }
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&b.p_full[pb]));
        if (i == first && done_g >= 0) finish((begun - 1) & 1);
      }
      if (leave) break;
      float sum[C];
#pragma unroll
      for (int k = 0; k < C / 2; ++k) {
        const float2 v = apart(l[k]);
        sum[2 * k] = v.x, sum[2 * k + 1] = v.y;
      }
      warp_col_sums<C>(sum, s_part[group][quad]);
      soft_sync(group);
      if (tok < C) {
        const float *s4 = s_part[group][0] + tok;
        if (ok) p.part_ml[slot_of(u, first) + tok] = make_float2(-nref_of[tok], (s4[0] + s4[C]) + (s4[2 * C] + s4[3 * C]));
        nref_of[tok] = -kNone;  // no reference yet: any score outgrows it
      }
      soft_sync(group);
      done_g = x_g, done_unit = unit, done_i = first, ++begun;
      g += ntiles;
    }
    if (done_g >= 0 && ok) {  // (after an expired wait there is no output)
      // (nothing has waited for this product yet)
      wait(&b.pv_done[done_g % G::kNP], done_g / G::kNP);
      if (ok) finish((begun - 1) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == G::kLoadWarp) asm volatile("cp.async.wait_all;" ::: "memory");
  // after an expired wait: copies in flight land before the block gives its memory back
  if (s_abort && warp == G::kPrepWarp && lane == 0)
    unit_copies(g, [&](int i, int parity) { mbar_drain(smem_u32(&b.q_full[i]), parity); },
                [&](int i, int parity) { mbar_drain(smem_u32(&b.factors[i]), parity); });
  if (s_abort && warp == G::kLoadWarp && lane == 0) {
    last_uses(g, G::kNK, [&](int i, int parity) { mbar_drain(smem_u32(&b.k_full[i]), parity); });
    last_uses(g, G::kNV, [&](int i, int parity) { mbar_drain(smem_u32(&b.v_full[i]), parity); });
  }
  if (warp == G::kScoreWarp) tmem_dealloc(tmem, G::kTmem);
}

// Q as the units' products take it: of each row tile of a K/V head the rows' parts of
// e4m3 (NP of R x D bytes), the rows in 16 bits ([64-element block][row]), both swizzled as
// shared memory has them, then the rows' factors, of either form.  A warp a row.
// (Once for each row tile, in a kernel of its own: by a warp of the attention's blocks a
// unit's Q took up to 30,000 cycles, more than its tiles.)  Bound by latency: 16,384 rows some 5 us, of
// which the attention's start hides a part.
template <int D, bool F16>
__global__ void __launch_bounds__(256) k_quant_q(const QuantAttnParams p) {
  constexpr int NP = F16 ? 3 : 2, E = D / 32;
  const TreeAttnParams &t = p.t;
  pdl_trigger();
  const int lane = threadIdx.x & 31, R = p.R, shift = R == 64 ? 6 : R == 32 ? 5 : 4;
  const uint32_t i = blockIdx.x * 8u + (threadIdx.x >> 5);  // row of all row tiles (at most 2^30; whole blocks)
  const uint32_t item = i >> shift, pair = item / (uint32_t)p.mtiles;
  const int row = (int)(i & (uint32_t)(R - 1)), mt = (int)(item - pair * p.mtiles);
  const int n = (int)(pair / (uint32_t)t.kv_heads), h = (int)(pair - (uint32_t)n * t.kv_heads);
  const int r = mt * R + row, node = r / t.group;
  const int len = t.tree_len ? min(max(t.tree_len[n], 0), t.T) : t.T;
  uint32_t x[E / 2];
#pragma unroll
  for (int k = 0; k < E / 2; ++k) x[k] = 0u;
  if (node < len) {
    const uint16_t *q = t.q + n * t.q_sn + node * t.q_st + (h * t.group + r - node * t.group) * t.q_sh + lane * E;
#pragma unroll
    for (int k = 0; k < E / 2; ++k) x[k] = __ldg(reinterpret_cast<const uint32_t *>(q) + k);
  }
  float most = 0.f;
#pragma unroll
  for (int k = 0; k < E / 2; ++k) most = fmaxf(most, fmaxf(fabsf(unpack_lo<F16>(x[k])), fabsf(unpack_lo<F16>(x[k] >> 16))));
  most = warp_max(most);
  // the power of two that brings the row's largest to 128..256 (rows below 2^-100 count as of that size; a
  // row with an infinity becomes NaN)
  const int e = max((int)(__float_as_uint(most) >> 23), 27);
  const float mul = __uint_as_float(e < 255 ? (uint32_t)(261 - e) << 23 : 0x7FC00000u);
  // (the factors too: products with the 16-bit form, the tree's, may all be -inf, and the row would pass for empty)
  const float c = e < 255 ? t.scale * kLog2e : mul;
  uint8_t *dst = p.q_parts + (int64_t)item * quant_q_bytes(NP, R, D);
  const int at = lane * E;
  const int off = row * D + (((at >> 4) ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4) + (at & 15);
  uint16_t part[NP][E / 2];
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    // (fp16 holds either type's elements of that size but for what lies below 2^-24)
    uint32_t f = pack2<true>(unpack_lo<F16>(x[k]) * mul, unpack_lo<F16>(x[k] >> 16) * mul);
#pragma unroll
    for (int y = 0; y < NP; ++y) {
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(part[y][k]) : "r"(f));
      uint32_t back;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(part[y][k]));
      f = hsub2(f, back);
    }
  }
#pragma unroll
  for (int y = 0; y < NP; ++y) {
    if constexpr (E == 4) *reinterpret_cast<uint32_t *>(dst + y * R * D + off) = part[y][0] | (uint32_t)part[y][1] << 16;
    else *reinterpret_cast<uint16_t *>(dst + y * R * D + off) = part[y][0];
  }
  dst += NP * R * D;
  uint8_t *wide = dst + (at >> 6) * (R * 128) + row * 128 + ((((at & 63) >> 3) ^ (row & 7)) << 4) + (at & 7) * 2;
  if constexpr (E == 4) *reinterpret_cast<uint2 *>(wide) = make_uint2(x[0], x[1]);
  else *reinterpret_cast<uint32_t *>(wide) = x[0];
  if (lane == 0) {
    float *factor = reinterpret_cast<float *>(dst + 2 * R * D);
    factor[row] = c * __uint_as_float((uint32_t)min(e - 7, 254) << 23);
    factor[R + row] = c;
  }
}

// The output of each row from its units: sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M)
// l_k, M = max m_k, chunks in order and the tree last; zeros for a node past the
// tree's length and for one that saw nothing.  One warp a row, its elements over the lanes.
template <int D, bool F16>
__global__ void __launch_bounds__(256, 6) k_quant_join(const QuantAttnParams p) {
  constexpr int E = D / 32;
  const TreeAttnParams &t = p.t;
  const int lane = threadIdx.x & 31, heads = t.kv_heads * t.group;
  const int n = blockIdx.x, of_n = blockIdx.y * 8 + (threadIdx.x >> 5);  // request, row of it
  if (of_n >= t.T * heads) return;
  const int node = of_n / heads, hq = of_n - node * heads;
  const int64_t orow = (int64_t)n * t.T * heads + of_n;
  int ctx, len;
  const int nc = context_chunks(p, n, ctx, len);
  const int h = hq / t.group, r = node * t.group + hq - h * t.group, mt = r / p.R, row = r - mt * p.R;
  const int teams = kQuantRows / p.R;  // partial results of a unit
  const int64_t first = (((int64_t)n * t.kv_heads + h) * p.mtiles + mt) * p.slots * teams * p.R + row;
  const float *po = p.part_o + first * D + lane * E;
  const float2 *ml = p.part_ml + first;
  pdl_wait();
  const int live = node < len ? (nc + 1) * teams : 0;
  float M = kNone, L = 0.f, acc[E] = {};
  // 32 partial results at a time, one a lane
  for (int k0 = 0; k0 < live; k0 += 32) {
    const float2 a = k0 + lane < live ? __ldcg(&ml[(int64_t)(k0 + lane) * p.R]) : make_float2(kNone, 0.f);
    // factors' roots: a sum is multiplied by them one after the other (see the top of this file)
    const float top = fmaxf(M, warp_max(a.x)), r0 = ex2(0.5f * (M - top)), f0 = r0 * r0;
    const float rk = a.y != 0.f ? ex2(0.5f * (a.x - top)) : 0.f, wk = rk * rk;
    M = top, L = L * r0 * r0 + warp_sum(a.y * rk * rk);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f0;
    const int k1 = min(live - k0, 32);
    const uint32_t holds = __ballot_sync(DC_FULL_MASK, a.y != 0.f);  // (an empty one was not written)
#pragma unroll 4
    for (int k = 0; k < k1; ++k) {
      const float f = __shfl_sync(DC_FULL_MASK, wk, k);
      if (!((holds >> k) & 1u)) continue;  // by its sum, not by f: a NaN counts however little its tokens weigh
      const float *src = po + (int64_t)(k0 + k) * p.R * D;
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
  uint32_t *out = reinterpret_cast<uint32_t *>(t.out + orow * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = some ? pack2<F16>(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  if (t.lse && lane == 0) t.lse[orow] = some ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

// A 4D map (element, token of a page, head, page) of one cache; a copy is a
// page's tokens (up to a tile) of one head.
bool encode_cache(CUtensorMap *map, const QuantAttnParams &p, const void *base, int64_t st, int64_t sh, int64_t sp) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int page = 1 << p.t.page_shift, D = p.t.head_dim;
  const auto bytes = [&](int n, int64_t s) { return (cuuint64_t)(n > 1 ? s : D); };
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)p.t.kv_heads, (cuuint64_t)p.t.num_pages};
  const cuuint64_t strides[3] = {bytes(page, st), bytes(p.t.kv_heads, sh), bytes(p.t.num_pages, sp)};
  const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)(page < kTile ? page : kTile), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same of the tree's own K or V: (64 elements, nodes, head, request) of a 16-bit type.
bool encode_nodes(CUtensorMap *map, const TreeAttnParams &t, const void *base, int64_t st, int64_t sh, int64_t sn) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const auto bytes = [&](int n, int64_t s) { return (cuuint64_t)(n > 1 ? s * 2 : t.head_dim * 2); };
  const cuuint64_t dims[4] = {(cuuint64_t)t.head_dim, (cuuint64_t)t.T, (cuuint64_t)t.kv_heads, (cuuint64_t)t.N};
  const cuuint64_t strides[3] = {bytes(t.T, st), bytes(t.kv_heads, sh), bytes(t.N, sn)};
  const cuuint32_t box[4] = {64, (cuuint32_t)t.tree_box, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, t.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int R, bool F16>
cudaError_t launch(const QuantAttnParams &p, const QuantMaps &maps, unsigned grid, cudaStream_t st) {
  const size_t smem = Geom8<D, R, F16 ? 3 : 2>::kSmem + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(k_quant_attn<D, R, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_ex(k_quant_attn<D, R, F16>, dim3(grid), dim3(Geom8<D, R, F16 ? 3 : 2>::kThreads), smem, st, true, 0, p, maps);
}

template <int D, bool F16>
cudaError_t launch_all(const QuantAttnParams &p, const QuantMaps &maps, unsigned grid, cudaStream_t st) {
  const int64_t q_rows = (int64_t)p.t.N * p.t.kv_heads * p.mtiles * p.R;
  k_quant_q<D, F16><<<(unsigned)(q_rows / 8), 256, 0, st>>>(p);  // (R is a multiple of 8)
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = p.R == 16   ? launch<D, 16, F16>(p, maps, grid, st)
                        : p.R == 32 ? launch<D, 32, F16>(p, maps, grid, st)
                                    : launch<D, 64, F16>(p, maps, grid, st);
  if (e != cudaSuccess) return e;
  const int rows = p.t.T * p.t.kv_heads * p.t.group;  // at most 256 x 1024 a request
  return launch_ex(k_quant_join<D, F16>, dim3((unsigned)p.t.N, (unsigned)((rows + 7) / 8)), dim3(256), 0, st, true, 0, p);
}

}  // namespace

cudaError_t launch_quant_attention(const QuantAttnParams &p, cudaStream_t st) {
  QuantMaps maps;
  if (!encode_cache(&maps.k, p, p.k_cache, p.kc_st, p.kc_sh, p.kc_sp) ||
      !encode_cache(&maps.v, p, p.v_cache, p.vc_st, p.vc_sh, p.vc_sp) ||
      !encode_nodes(&maps.k_new, p.t, p.t.k_new, p.t.kn_st, p.t.kn_sh, p.t.kn_sn) ||
      !encode_nodes(&maps.v_new, p.t, p.t.v_new, p.t.vn_st, p.t.vn_sh, p.t.vn_sn))
    return cudaErrorInvalidValue;
  const int64_t most = (int64_t)p.t.N * p.t.kv_heads * p.mtiles * p.slots;
  const unsigned grid = (unsigned)(most < p.sms ? most : p.sms);
  if (p.t.head_dim == 128) return p.t.f16 ? launch_all<128, true>(p, maps, grid, st) : launch_all<128, false>(p, maps, grid, st);
  return p.t.f16 ? launch_all<64, true>(p, maps, grid, st) : launch_all<64, false>(p, maps, grid, st);
}

}  // namespace dc
