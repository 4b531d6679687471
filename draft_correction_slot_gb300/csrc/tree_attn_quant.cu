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
//   P: rounded to fp16 (2^-11), then 3 parts of e5m2, N columns of their own: the
//     first two to nearest, each leaving its error to the next, so that 2^-11 of
//     a weight is lost once more; the third times 2^7, below whose least step lies
//     nothing that fp16 kept.
// The scales never touch an operand: ks multiplies a score (a thread has a
// token), log2(vs) is added to it, and the sum takes its weights divided by vs.
// So a row's reference is the largest log2 of weight x vs.
//
// The tree's own nodes are a unit of their own with 16-bit operands, 64 nodes a
// tile in a tile's place.  Units (request, K/V head, row tile, chunk of the
// context or tree) are dealt to one persistent block an SM; each leaves its rows'
// unnormalised output, reference and sum, and a second kernel joins them.
//
// Roles: warps 0-7 softmax and output (two groups of four, half of the rows each;
// thread = token = TMEM lane), 8 the tensor core, 9 and 10 TMA for K and V with the
// scales, 12-15 the units' Q parts and the tree's K and V.  After an expired wait the
// softmax and preparing warps run their loops to the end without waiting or
// storing, so that their barriers stay complete.
#include "launch.h"
#include "quant.cuh"
#include "tma_map.h"
#include "tree_attn.cuh"

namespace dc {
namespace {

constexpr int kGroup = 128, kSoft = 2 * kGroup;  // softmax threads of a group, of both
constexpr int kMmaWarp = 8, kLoadWarp = 9, kPrepWarp = 12;
constexpr int kThreads = 512;  // four warpgroups; warp 11 only completes the third
// Registers a thread: 128 at launch (65,536 / 512), then 2 x 168 + 2 x 88 = 4 x 128.
constexpr int kSoftRegs = 168, kOtherRegs = 88;
constexpr int kTreeNodes = 64;  // nodes of a tree tile
constexpr int kAhead = 8;       // units whose row factors and odd nodes are kept
constexpr float kTop = 7.f;     // log2 of a weight at its row's reference
constexpr float kGrow = kTop + kRescale;  // log2 of the largest weight: 2^15 fits fp16 and e5m2

struct QuantMaps {
  CUtensorMap k, v;
};

template <int D, int R, int NP>
struct Geom8 {
  static constexpr uint32_t kTileBytes = kTile * D;        // a context tile of K or V; a tree tile takes the same
  static constexpr int kNK = D == 64 ? 6 : NP == 3 ? 3 : 4, kNV = D == 64 ? 6 : 4;
  static constexpr uint32_t kQPart = R * D, kQBytes = NP * kQPart;
  static constexpr int kPAtoms = (3 * R + 63) / 64;        // 64-byte column blocks of P
  static constexpr uint32_t kPAtom = kTile * 64, kPBytes = kPAtoms * kPAtom;
  // V before P: products over 64 elements read as many rows of M past a V stage,
  // which have to be shared memory of ours (their results are not used); so do the
  // tree's products over 64 nodes past a K stage
  static constexpr uint32_t kK = 0, kV = kK + kNK * kTileBytes, kP = kV + kNV * kTileBytes;
  static constexpr uint32_t kQ = kP + 2 * kPBytes, kSmem = kQ + 2 * kQBytes;
  static constexpr uint32_t kTmem = 8 * R;                 // columns: S^T of even and odd tiles, O^T of even and odd units
  static constexpr uint32_t kS = 0, kO = 2 * R;
  // descriptors' high words: D-byte swizzle for K8, V8, Q8, 64 for P8
  static constexpr uint32_t kHi = D == 128 ? (1024 >> 4) | 1u << 14 | 2u << 29 : (512 >> 4) | 1u << 14 | 4u << 29;
  static constexpr uint32_t kHiP = (512 >> 4) | 1u << 14 | 4u << 29;
};

struct Bars8 {
  unsigned long long q_full[2], q_empty[2], k_full[8], k_empty[8], v_full[8], v_empty[8];
  unsigned long long s_full[2], p_full[2], pv_done[2], o_free[2], factors[kAhead], done;
};

constexpr int kVFull = 33;  // arrivals that fill a V stage: TMA's and each lane's scales

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
__device__ __forceinline__ void prep_sync() { asm volatile("barrier.cta.sync 3, 128;" ::: "memory"); }
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
    const uint32_t r = hsub2(p, h[i]);
    m[i] = top_bytes(r);
    l[i] = top_bytes(hmul2(hsub2(r, m[i]), 0x58005800u));  // 2^7
  }
  hi = __byte_perm(h[0], h[1], 0x7531), mid = __byte_perm(m[0], m[1], 0x7531), lo = __byte_perm(l[0], l[1], 0x7531);
}

// ---------------------------------------------------------------- units
struct QuantUnit {
  int n, h, mt, slot;        // request, K/V head, row tile, place among the partial results
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

template <int D, int R, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
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
  __shared__ uint32_t s_odd[kAhead][8];                    // tree units: nodes whose V holds an infinity or NaN
  __shared__ float s_scale[G::kNV][2][8];                  // a V stage's tile: K and V scales of its blocks
  __shared__ __align__(16) float s_mb[R], s_f[R];          // the rows' references less kTop, and rescale factors
  __shared__ __align__(16) float s_part[4][R];
  uint32_t(*const s_word)[R] = reinterpret_cast<uint32_t(*)[R]>(s_part);  // mask words (a tile's step between uses of s_part)
  const int tid = threadIdx.x, warp = __shfl_sync(DC_FULL_MASK, tid >> 5, 0), lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b.q_full[i]), 4), mbar_init(smem_u32(&b.q_empty[i]), 1);
      mbar_init(smem_u32(&b.s_full[i]), 1), mbar_init(smem_u32(&b.p_full[i]), kSoft / 32);
      mbar_init(smem_u32(&b.pv_done[i]), 1), mbar_init(smem_u32(&b.o_free[i]), kSoft / 32);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&b.k_full[i]), 1), mbar_init(smem_u32(&b.k_empty[i]), 1);
      mbar_init(smem_u32(&b.v_full[i]), kVFull), mbar_init(smem_u32(&b.v_empty[i]), 1);
      mbar_init(smem_u32(&b.factors[i]), 4);
    }
    mbar_init(smem_u32(&b.done), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kLoadWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), G::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(DC_FULL_MASK, s_tmem, 0);
  int g = 0, live = 0;  // tiles and units with tiles that this role has begun

  pdl_trigger();

  QuantUnit w;
  if (warp >= kMmaWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp >= kPrepWarp) {
    // ------------------------------------------------------------ Q parts, the tree's K and V
    QuantUnits it(p, false);
    const int pt = tid - kPrepWarp * 32;
    constexpr int kPer = 128 / R;              // threads of a row
    constexpr int kVecs = D / kPer / 8;        // 16-byte vectors of a thread
    const int row = pt / kPer, e0 = (pt % kPer) * (D / kPer);
    const float c = t.scale * kLog2e;
    bool ok = true;
    auto wait = [&](unsigned long long *bar, int phase) {
      if (ok) ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(bar), phase & 1, &s_abort, t.err));
    };
    while (it.next(w)) {
      if (w.ntiles == 0) continue;
      const int qb = live & 1, r = w.mt * R + row, node = r / t.group;
      const bool there = node < w.len;
      const uint4 *q = reinterpret_cast<const uint4 *>(t.q + w.n * t.q_sn + (there ? node : 0) * t.q_st +
                                                       (w.h * t.group + r - node * t.group) * t.q_sh + e0);
      float most = 0.f;
      if (!w.tree && there) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const uint4 x = __ldg(q + i);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            most = fmaxf(most, fmaxf(fabsf(unpack_lo<F16>(u[j])), fabsf(unpack_lo<F16>(u[j] >> 16))));
        }
      }
#pragma unroll
      for (int o = 1; o < kPer; o <<= 1) most = fmaxf(most, __shfl_xor_sync(DC_FULL_MASK, most, o));
      // the power of two that brings the row's largest to 128..256 (rows below 2^-100 count as of that size)
      const int e = max((int)(__float_as_uint(most) >> 23), 27);
      const float mul = __uint_as_float((uint32_t)(261 - e) << 23);
      const float factor = w.tree ? c : c * __uint_as_float((uint32_t)min(e - 7, 254) << 23);
      if (live >= 2) wait(&b.q_empty[qb], (live >> 1) - 1);
      uint8_t *dst = smem + G::kQ + qb * G::kQBytes;
#pragma unroll 1
      for (int i = 0; i < kVecs; ++i) {  // (one at a time: the elements are at hand in L1, registers are not)
        const uint4 x = there ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
        const int at = e0 + i * 8;
        if (w.tree) {
          if (ok)
            *reinterpret_cast<uint4 *>(dst + (at >> 6) * (R * 128) + row * 128 + ((((at & 63) >> 3) ^ (row & 7)) << 4)) = x;
          continue;
        }
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[2 * j] = unpack_lo<F16>(u[j]) * mul, f[2 * j + 1] = unpack_lo<F16>(u[j] >> 16) * mul;
        uint8_t *d = dst + row * D + (((at >> 4) ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4) + (at & 8);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[j] = to_e4m3x2(f[2 * j], f[2 * j + 1]);
            const float2 y = from_e4m3x2(h[j]);
            f[2 * j] -= y.x, f[2 * j + 1] -= y.y;
          }
          if (ok) *reinterpret_cast<uint2 *>(d + k * G::kQPart) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        }
      }
      if (pt % kPer == 0 && ok) s_factor[live & (kAhead - 1)][row] = factor;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0 && ok) {
        mbar_arrive(smem_u32(&b.q_full[qb]));
        mbar_arrive(smem_u32(&b.factors[live & (kAhead - 1)]));
      }
      for (int i = 0; w.tree && i < w.ntiles; ++i) {
        const int gt = g + i, ks = gt % G::kNK, vs = gt % G::kNV;
        const int nd = i * kTreeNodes + (pt >> 1), k0 = (pt & 1) * (D / 2);  // a node's half a thread
        const bool in = nd < w.len;
        const uint16_t *src[2] = {t.k_new + w.n * t.kn_sn + nd * t.kn_st + w.h * t.kn_sh + k0,
                                  t.v_new + w.n * t.vn_sn + nd * t.vn_st + w.h * t.vn_sh + k0};
        uint8_t *dst[2] = {smem + G::kK + ks * G::kTileBytes + (pt >> 1) * 128, smem + G::kV + vs * G::kTileBytes + (pt >> 1) * 128};
        bool bad = false;
        if (in) asm volatile("prefetch.global.L2 [%0];" ::"l"(src[1]) : "memory");  // (V's first sectors, under the wait for K)
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          uint4 x[D / 16];
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            x[j] = in ? __ldg(reinterpret_cast<const uint4 *>(kv ? src[1] : src[0]) + j) : make_uint4(0, 0, 0, 0);
          // A stage is free when its last tile's product is done.  The products of the unit before come
          // first: past them the stage's barrier is at most one phase behind, and a parity tells.
          if (kv == 0 && i == 0 && live > 0) wait(&b.q_empty[(live - 1) & 1], (live - 1) >> 1);
          if (kv == 0 && gt >= G::kNK) wait(&b.k_empty[ks], gt / G::kNK - 1);
          if (kv == 1 && gt >= G::kNV) wait(&b.v_empty[vs], gt / G::kNV - 1);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t xs[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
            // a node's infinities and NaN in V stay out of the product (they would reach
            // nodes that do not see it) and are added to the output of those that do
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (kv == 1 && nonfinite2<F16>(xs[k])) {
                const bool lo = nonfinite2<F16>(xs[k] & 0xFFFFu), hi = nonfinite2<F16>(xs[k] >> 16);
                xs[k] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
                bad = true;
              }
            const int e = k0 + j * 8;
            if (ok)
              *reinterpret_cast<uint4 *>((kv ? dst[1] : dst[0]) + (e >> 6) * (kTreeNodes * 128) +
                                         ((((e & 63) >> 3) ^ ((pt >> 1) & 7)) << 4)) = make_uint4(xs[0], xs[1], xs[2], xs[3]);
          }
        }
        // (__ballot: two bits a node, gathered to one)
        uint32_t bits = __ballot_sync(DC_FULL_MASK, bad);
        bits = (bits | bits >> 1) & 0x55555555u;
        bits = (bits | bits >> 1) & 0x33333333u, bits = (bits | bits >> 2) & 0x0F0F0F0Fu;
        bits = (bits | bits >> 4) & 0x00FF00FFu, bits = (bits | bits >> 8) & 0xFFFFu;
        if (lane == 0 && ok) reinterpret_cast<uint16_t *>(s_odd[live & (kAhead - 1)])[i * 4 + (pt >> 5)] = (uint16_t)bits;
        fence_proxy_async();
        prep_sync();
        if (pt == 0 && ok) {
          mbar_arrive(smem_u32(&b.k_full[ks]));
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&b.v_full[vs])), "n"(kVFull) : "memory");
        }
      }
      g += w.ntiles;
      ++live;
    }
  } else if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ------------------------------------------------------------ TMA: the context's K; V and the scales
    const bool is_v = warp != kLoadWarp, flag = !is_v && blockIdx.x == 0;
    const int stages = is_v ? G::kNV : G::kNK;
    unsigned long long *full = is_v ? b.v_full : b.k_full, *empty = is_v ? b.v_empty : b.k_empty;
    const uint32_t ring = sbase + (is_v ? G::kV : G::kK);
    const CUtensorMap *map = is_v ? &maps.v : &maps.k;
    const int page_size = 1 << t.page_shift, box = min(page_size, kTile), boxes = kTile / box, per = 32 / boxes;
    // lanes 0-7 fetch K's scales of a tile, 8-15 V's; block j of the tile
    const int j = lane & 7, tok_j = j << p.scale_shift;
    const float *scale = lane < 8 ? p.k_scale : p.v_scale;
    const int64_t sp = lane < 8 ? p.ks_sp : p.vs_sp, sb = lane < 8 ? p.ks_sb : p.vs_sb, ss = lane < 8 ? p.ks_sh : p.vs_sh;
    QuantUnits it(p, flag);
    bool ok = true;
    while (ok && it.next(w, flag)) {
      if (w.tree) {
        g += w.ntiles;
        continue;
      }
      int page = 0;  // lane l: page of box l of the tiles at hand
      for (int i = 0; ok && i < w.ntiles; ++i, ++g) {
        const int tok0 = (w.tile0 + i) * kTile, at = i % per * boxes, stage = g % stages;
        if (at == 0) {
          const int tok = tok0 + lane * box;
          page = 0;
          if (tok < w.ctx && lane < (w.ntiles - i) * boxes) {
            page = __ldg(t.page_table + w.n * t.pt_stride + (tok >> t.page_shift));
            if (page < 0 || page >= t.num_pages) {
              atomicOr(t.err, kErrBadPage);
              page = 0;
            }
          }
        }
        if (g >= stages) ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&empty[stage]), (g / stages - 1) & 1, &s_abort, t.err));
        if (!ok) break;
        const int used = min(boxes, (w.ctx - tok0 + box - 1) / box);  // copies of the tile
        const uint32_t dst = ring + stage * G::kTileBytes, bar = smem_u32(&full[stage]);
        if (is_v) {
          const int pg = __shfl_sync(DC_FULL_MASK, page, at + min(tok_j, kTile - 1) / box);
          if (lane < 16 && tok_j < kTile && tok0 + tok_j < w.ctx) {
            const float *src = scale + pg * sp + (((tok0 + tok_j) & (page_size - 1)) >> p.scale_shift) * sb + w.h * ss;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&s_scale[stage][lane >> 3][j])), "l"(src)
                         : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        }
        if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(used * box * D));
        __syncwarp();
        for (int r = 0; r < used; ++r) {
          const int pg = __shfl_sync(DC_FULL_MASK, page, at + r);
          if (elect_one()) tma_load_4d(dst + r * box * D, map, 0, tok0 & (page_size - 1), w.h, pg, bar);
          __syncwarp();
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ tensor core
    constexpr uint32_t kId8 = (1u << 4) | (8u << 24);                              // fp32 += e4m3 e4m3, M = 128
    constexpr uint32_t kIdS = kId8 | (uint32_t)(R >> 3) << 17;
    constexpr uint32_t kIdO = kId8 | (1u << 10) | (1u << 15) | (1u << 16) | (uint32_t)(3 * R >> 3) << 17;  // B e5m2; both M- and N-major
    constexpr uint32_t kIdS16 = F16 ? idesc_f16(128, R) : idesc_bf16(128, R);
    constexpr uint32_t kIdO16 = kIdS16 | (1u << 15) | (1u << 16);
    QuantUnits it(p, false);
    bool ok = true;
    // O^T (+)= V^T P^T of tile x, the first of the block's unit number `unit` if `first`
    auto pv = [&](int x, bool first, int unit, bool tree) {
      const int vs = x % G::kNV;
      const bool go = bar_wait(smem_u32(&b.v_full[vs]), (x / G::kNV) & 1, &s_abort, t.err) &&
                      (!first || unit < 2 || bar_wait(smem_u32(&b.o_free[unit & 1]), ((unit >> 1) - 1) & 1, &s_abort, t.err)) &&
                      bar_wait(smem_u32(&b.p_full[x & 1]), (x >> 1) & 1, &s_abort, t.err);
      if (!__all_sync(DC_FULL_MASK, go)) return false;
      tc_fence_after();
      const uint32_t to = tmem + G::kO + (unit & 1) * 3 * R;
      const uint32_t sv = sbase + G::kV + vs * G::kTileBytes, sp = sbase + G::kP + (x & 1) * G::kPBytes;
      if (tree) {
        const uint32_t a = desc_lo(sv, kTreeNodes * 128), pb = desc_lo(sp);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTreeNodes / 16; ++k)
            mma_ss(to, a + k * (2048 >> 4), pb + k * (2048 >> 4), kIdO16, (!first || k > 0) ? 1u : 0u);
          mma_commit(smem_u32(&b.v_empty[vs]));
          mma_commit(smem_u32(&b.pv_done[x & 1]));
        }
      } else {
        const uint32_t a = desc_lo(sv, G::kTileBytes), pb = desc_lo(sp, G::kPAtom);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            mma8<G::kHi, G::kHiP>(to, a + k * (32 * D >> 4), pb + k * (2048 >> 4), kIdO, (!first || k > 0) ? 1u : 0u);
          mma_commit(smem_u32(&b.v_empty[vs]));
          mma_commit(smem_u32(&b.pv_done[x & 1]));
        }
      }
      __syncwarp();
      return true;
    };
    bool prev_first = false, prev_tree = false;
    int prev_unit = 0;
    while (ok && it.next(w)) {
      if (w.ntiles == 0) continue;
      const int qb = live & 1;
      ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.q_full[qb]), (live >> 1) & 1, &s_abort, t.err));
      for (int i = 0; ok && i < w.ntiles; ++i, ++g) {
        const int ks = g % G::kNK;
        ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(&b.k_full[ks]), (g / G::kNK) & 1, &s_abort, t.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sq = desc_lo(sbase + G::kQ + qb * G::kQBytes), sk = desc_lo(sbase + G::kK + ks * G::kTileBytes);
        const uint32_t to = tmem + G::kS + (g & 1) * R;
        if (elect_one()) {
          if (w.tree) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(to, sk + (((k >> 2) * (kTreeNodes * 128) + (k & 3) * 32) >> 4),
                     sq + (((k >> 2) * (R * 128) + (k & 3) * 32) >> 4), kIdS16, k > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int x = 0; x < NP; ++x)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                mma8<G::kHi, G::kHi>(to, sk + k * 2, sq + ((x * G::kQPart) >> 4) + k * 2, kIdS, (x > 0 || k > 0) ? 1u : 0u);
          }
          mma_commit(smem_u32(&b.s_full[g & 1]));
          mma_commit(smem_u32(&b.k_empty[ks]));
          if (i == w.ntiles - 1) mma_commit(smem_u32(&b.q_empty[qb]));
        }
        __syncwarp();
        if (g > 0) ok = pv(g - 1, prev_first, prev_unit, prev_tree);
        prev_first = i == 0, prev_unit = live, prev_tree = w.tree;
      }
      ++live;
    }
    if (ok && g > 0) pv(g - 1, prev_first, prev_unit, prev_tree);
    if (elect_one()) {  // the lane that issued: nothing is in flight when the block frees its TMEM
      mma_commit(smem_u32(&b.done));
      mbar_drain(smem_u32(&b.done), 0);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------------------ softmax, output
    QuantUnits it(p, false);
    constexpr int C = R / 2;  // this group's rows: columns col0 .. col0 + C - 1
    const int group = warp >> 2, quad = warp & 3, tok = tid & (kGroup - 1), col0 = group * C;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + col0;
    bool ok = true;
    auto wait = [&](unsigned long long *bar, int phase) {
      if (ok) ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(bar), phase & 1, &s_abort, t.err));
    };
    // A unit's output, unnormalised, leaves for the join after the first tile of
    // the unit that follows, whose products go to the other half of O, so that the
    // tensor core and the copies go on meanwhile.
    QuantUnit done = {};
    int done_g = -1, done_unit = 0;  // that unit's last tile (-1: none), its number
    auto slot_of = [&](const QuantUnit &u) {  // the unit's rows among the partial results
      return ((((int64_t)u.n * t.kv_heads + u.h) * p.mtiles + u.mt) * p.slots + u.slot) * R;
    };
    auto finish = [&] {
      const int par = done_unit & 1;
      wait(&b.pv_done[done_g & 1], done_g >> 1);
      tc_fence_after();
      const uint32_t from = trow + G::kO + par * 3 * R;
      float o[C];
      tmem_ld<C>(from, o);
      if (!done.tree) {
        float x[C];
        tmem_ld<C>(from + R, x);
#pragma unroll
        for (int k = 0; k < C; ++k) o[k] += x[k];
        tmem_ld<C>(from + 2 * R, x);
#pragma unroll
        for (int k = 0; k < C; ++k) o[k] = fmaf(x[k], 0.0078125f, o[k]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&b.o_free[par]));
      float *part = p.part_o + (slot_of(done) + col0) * D + tok;  // [row][D]
      if (tok < D && ok) {
#pragma unroll
        for (int k = 0; k < C; ++k) part[k * D] = o[k];
        if (done.tree) {
          // infinities and NaN of the nodes that a row sees
#pragma unroll 1
          for (int q = 0; q < (done.len + 31) / 32; ++q)
#pragma unroll 1
            for (uint32_t r = s_odd[done_unit & (kAhead - 1)][q]; r; r &= r - 1) {
              const int x = __ffs(r) - 1;
              const uint32_t e = t.v_new[done.n * t.vn_sn + (q * 32 + x) * t.vn_st + done.h * t.vn_sh + tok];
              if (!nonfinite2<F16>(e)) continue;
#pragma unroll 1
              for (int k = 0; k < C; ++k)
                if ((tree_sees(t, done.n, done.len, (done.mt * R + col0 + k) / t.group, q) >> x) & 1u)
                  part[k * D] += unpack_lo<F16>(e);
            }
        }
      }
      __syncwarp();
      done_g = -1;
    };
    while (it.next(w)) {
      if (w.ntiles == 0) continue;
      const float *factor = s_factor[live & (kAhead - 1)] + col0;
      wait(&b.factors[live & (kAhead - 1)], live / kAhead);
      ++live;
      float l[C];  // the rows' sums over this thread's tokens
#pragma unroll
      for (int k = 0; k < C; ++k) l[k] = 0.f;
      for (int i = 0; i < w.ntiles; ++i, ++g) {
        const int tok0 = (w.tile0 + i) * (w.tree ? kTreeNodes : kTile), vs = g % G::kNV;
        const int valid = w.tree ? min(kTreeNodes, w.len - tok0) : min(kTile, w.ctx - tok0);
        wait(&b.v_full[vs], g / G::kNV);  // the scales, and the tree's odd nodes
        float ks = 1.f, lvs = 0.f, inv = 1.f;
        if (!w.tree && tok < valid) {
          const int blk = tok >> p.scale_shift;
          ks = s_scale[vs][0][blk];
          const float x = s_scale[vs][1][blk];
          lvs = __log2f(x), inv = __frcp_rn(x);
        }
        if (!w.tree && valid < kTile && group == 0) {
          // past the end lies what a page or a copy left: zeros in its place, since a zero weight does not cancel NaN
          if (ok && tok >= valid) {
            uint4 *row = reinterpret_cast<uint4 *>(smem + G::kV + vs * G::kTileBytes + tok * D);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) row[e] = make_uint4(0, 0, 0, 0);
          }
        }
        wait(&b.s_full[g & 1], g >> 1);
        if (g >= 2) wait(&b.pv_done[g & 1], (g >> 1) - 1);  // P's buffer is free
        tc_fence_after();
        float v[C];
        // once, or once more when a score has outgrown its row's reference
        for (bool renew = false;;) {
          // log2 of weight x vs
          tmem_ld<C>(trow + G::kS + (g & 1) * R, v);
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(factor + k);
            v[k] = fmaf(v[k] * ks, f.x, lvs), v[k + 1] = fmaf(v[k + 1] * ks, f.y, lvs);
            v[k + 2] = fmaf(v[k + 2] * ks, f.z, lvs), v[k + 3] = fmaf(v[k + 3] * ks, f.w, lvs);
          }
          if (w.tree) {
            // this warp's 32 nodes are one word of each row's mask: lane k fetches row k's
            if (lane < C)
              s_word[quad][col0 + lane] =
                  quad < kTreeNodes / 32 ? tree_sees(t, w.n, w.len, (w.mt * R + col0 + lane) / t.group, tok0 / 32 + quad) : 0u;
            __syncwarp();
#pragma unroll
            for (int k = 0; k < C; k += 4) {
              const uint4 word = *reinterpret_cast<const uint4 *>(&s_word[quad][col0 + k]);
              v[k] = (word.x >> lane) & 1u ? v[k] : -INFINITY;
              v[k + 1] = (word.y >> lane) & 1u ? v[k + 1] : -INFINITY;
              v[k + 2] = (word.z >> lane) & 1u ? v[k + 2] : -INFINITY;
              v[k + 3] = (word.w >> lane) & 1u ? v[k + 3] : -INFINITY;
            }
            __syncwarp();
          } else if (tok >= valid) {
#pragma unroll
            for (int k = 0; k < C; ++k) v[k] = -INFINITY;
          }
          if (renew) {
            // references from the rows' maxima over the tile; l and O^T follow
#pragma unroll
            for (int k = 0; k < C; ++k) {
              const float m = warp_fmax(v[k]);
              if (lane == k) s_part[quad][col0 + k] = m;
            }
            soft_sync(group);
            if (tok < C) {
              const int k = col0 + tok;
              const float m = fmaxf(fmaxf(s_part[0][k], s_part[1][k]), fmaxf(s_part[2][k], s_part[3][k]));
              const float old = s_mb[k];
              const bool grown = m - old > kGrow;  // (the others stay: a row's result hangs on its own scores)
              s_mb[k] = grown ? m - kTop : old;
              s_f[k] = grown ? ex2(old - m + kTop) : 1.f;
            }
            soft_sync(group);
#pragma unroll
            for (int k = 0; k < C; ++k) l[k] *= s_f[col0 + k];
            if (i > 0) {
              wait(&b.pv_done[(g - 1) & 1], (g - 1) >> 1);
              tc_fence_after();
              const uint32_t to = trow + G::kO + ((live - 1) & 1) * 3 * R;
#pragma unroll 1
              for (int x = 0; x < (w.tree ? 1 : 3); ++x) {
                float o[C];
                tmem_ld<C>(to + x * R, o);
#pragma unroll
                for (int k = 0; k < C; ++k) o[k] *= s_f[col0 + k];
                tmem_st<C>(to + x * R, o);
              }
            }
          } else if (i == 0) {
            // a unit begins with the best of four tokens' scores as the references
            if (lane == 0) {
#pragma unroll
              for (int k = 0; k < C; k += 4)
                *reinterpret_cast<float4 *>(&s_part[quad][col0 + k]) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
            soft_sync(group);
            if (tok < C) {
              const int k = col0 + tok;
              const float m = fmaxf(fmaxf(s_part[0][k], s_part[1][k]), fmaxf(s_part[2][k], s_part[3][k])) - kTop;
              s_mb[k] = fabsf(m) < INFINITY ? m : kNone;
            }
            soft_sync(group);
          }
          // exponents against the references, in v's place
          float grow[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const float4 mb = *reinterpret_cast<const float4 *>(&s_mb[col0 + k]);
            v[k] -= mb.x, v[k + 1] -= mb.y, v[k + 2] -= mb.z, v[k + 3] -= mb.w;
            grow[0] = fmaxf(grow[0], v[k]), grow[1] = fmaxf(grow[1], v[k + 1]);
            grow[2] = fmaxf(grow[2], v[k + 2]), grow[3] = fmaxf(grow[3], v[k + 3]);
          }
          if (renew || !soft_any(group, fmaxf(fmaxf(grow[0], grow[1]), fmaxf(grow[2], grow[3])) > kGrow)) break;
          renew = true;
        }
        uint8_t *pbuf = smem + G::kP + (g & 1) * G::kPBytes;
        if (w.tree) {
#pragma unroll
          for (int k = 0; k < C; k += 8) {
            float e[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              e[x] = ex2(v[k + x]);
              l[k + x] += e[x];
            }
            if (tok < kTreeNodes)
              *reinterpret_cast<uint4 *>(pbuf + tok * 128 + ((((col0 + k) >> 3) ^ (tok & 7)) << 4)) =
                  make_uint4(pack2<F16>(e[0], e[1]), pack2<F16>(e[2], e[3]), pack2<F16>(e[4], e[5]), pack2<F16>(e[6], e[7]));
          }
        } else {
          constexpr int kStep = C < 16 ? C : 16;  // rows of a store
#pragma unroll
          for (int k = 0; k < C; k += kStep) {
            uint32_t parts[3][kStep / 4];
#pragma unroll
            for (int x = 0; x < kStep; x += 4) {
              float e[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                e[y] = ex2(v[k + x + y]);
                l[k + x + y] = fmaf(e[y], inv, l[k + x + y]);
              }
              split4(e, parts[0][x / 4], parts[1][x / 4], parts[2][x / 4]);
            }
#pragma unroll
            for (int x = 0; x < 3; ++x) {
              const int col = x * R + col0 + k;  // of the parts side by side
              uint8_t *d = pbuf + (col >> 6) * G::kPAtom + tok * 64 + ((((col & 63) >> 4) ^ ((tok >> 1) & 3)) << 4) + (col & 15);
              if constexpr (kStep == 16) *reinterpret_cast<uint4 *>(d) = make_uint4(parts[x][0], parts[x][1], parts[x][2], parts[x][3]);
              else *reinterpret_cast<uint2 *>(d) = make_uint2(parts[x][0], parts[x][1]);
            }
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&b.p_full[g & 1]));
        if (i == 0 && done_g >= 0) finish();
      }
      warp_col_sums<C>(l, s_part[quad] + col0);
      soft_sync(group);
      if (tok < C && ok) {
        const int k = col0 + tok;
        p.part_ml[slot_of(w) + k] = make_float2(s_mb[k], (s_part[0][k] + s_part[1][k]) + (s_part[2][k] + s_part[3][k]));
      }
      soft_sync(group);
      done = w, done_g = g - 1, done_unit = live - 1;
    }
    if (done_g >= 0) finish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kLoadWarp + 1) asm volatile("cp.async.wait_all;" ::: "memory");
  if (s_abort && lane == 0 && (warp == kLoadWarp || warp == kLoadWarp + 1)) {
    // after an expired wait: copies in flight land before the block gives its memory back
    const int stages = warp == kLoadWarp ? G::kNK : G::kNV;
    unsigned long long *full = warp == kLoadWarp ? b.k_full : b.v_full;
    for (int x = max(0, g - stages); x < g; ++x) mbar_drain(smem_u32(&full[x % stages]), (x / stages) & 1);
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem, G::kTmem);
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
  const int64_t first = (((int64_t)n * t.kv_heads + h) * p.mtiles + mt) * p.slots * p.R + row;
  const float *po = p.part_o + first * D + lane * E;
  const float2 *ml = p.part_ml + first;
  pdl_wait();
  float2 a[2];  // partial results lane and 32 + lane (at most kTreeMaxChunks)
  const int live = node < len ? nc + 1 : 0;
  for (int q = 0; q < 2; ++q) a[q] = q * 32 + lane < live ? __ldcg(&ml[(q * 32 + lane) * p.R]) : make_float2(kNone, 0.f);
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
      const float *src = po + (int64_t)k * p.R * D;
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

template <int D, int R, bool F16>
cudaError_t launch(const QuantAttnParams &p, const QuantMaps &maps, unsigned grid, cudaStream_t st) {
  const size_t smem = Geom8<D, R, F16 ? 3 : 2>::kSmem + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(k_quant_attn<D, R, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k_quant_attn<D, R, F16><<<grid, kThreads, smem, st>>>(p, maps);
  return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t launch_all(const QuantAttnParams &p, const QuantMaps &maps, unsigned grid, cudaStream_t st) {
  const cudaError_t e = p.R == 16   ? launch<D, 16, F16>(p, maps, grid, st)
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
      !encode_cache(&maps.v, p, p.v_cache, p.vc_st, p.vc_sh, p.vc_sp))
    return cudaErrorInvalidValue;
  const int64_t most = (int64_t)p.t.N * p.t.kv_heads * p.mtiles * p.slots;
  const unsigned grid = (unsigned)(most < p.sms ? most : p.sms);
  if (p.t.head_dim == 128) return p.t.f16 ? launch_all<128, true>(p, maps, grid, st) : launch_all<128, false>(p, maps, grid, st);
  return p.t.f16 ? launch_all<64, true>(p, maps, grid, st) : launch_all<64, false>(p, maps, grid, st);
}

}  // namespace dc
