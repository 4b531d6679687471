// tree_attn_few.cu -- tree attention when a K/V head has at most 64 query
// rows (nodes x group), single-token decoding among them.
//
// The products are turned round: S^T = K Q^T (M = the tile's 128 tokens, N =
// the rows, padded to 16, 32 or 64) and O^T += V^T P^T (M = the head's
// elements, N = the rows).  So a tile costs 128 x rows exponentials, where
// rows in M cost 128 x 128 whatever their number.  Two softmax groups of four
// warps have half of the rows each, and each of their warps 32 tokens of every
// row of its group: two warps a scheduler hide each other's latencies (with
// one group a tile's step took 2800 cycles, as long as its 64 KB take to
// arrive, and nothing was left to make up for the unit borders).  P^T goes to shared memory, a
// token's row of N weights the 128 bytes of a swizzle row.
//
// A row's reference (the maximum when last taken) is common to its group's
// warps; its sum is kept per thread, over the thread's tokens, until the
// unit's end.  A unit's first references are the best of four tokens' scores; per
// tile a group's warps only vote whether any score has outgrown its row's reference
// by 2^8, and only then the references are taken anew (the maxima across the
// group) and the rows' O^T is rescaled.
//
// Every unit leaves its result to the join kernel (tree_attn.cu).  32 requests
// of up to 8000 tokens, 16 nodes x 4 heads: 132 us with it, 613 MB (floor 91);
// inside a unit a 64 KB tile takes 2865 cycles, HBM's rate.
//
// Roles: warps 0-7 softmax (thread = token = TMEM lane) and output (thread =
// element), warp 8 the tensor core, warps 9-10 TMA.  After an expired wait the
// softmax warps run their loops to the end without waiting or storing, so
// that their block barriers stay complete.
#include "tree_attn.cuh"

namespace dc {
namespace {

constexpr int kGroup = 128, kSoft = 2 * kGroup;  // softmax threads of a group, of both
constexpr int kMmaWarp = kSoft / 32, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);

template <int D, int N>
struct GeomFew {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kHalfBytes = kTile * 128;
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  static constexpr int kNK = D == 128 ? 2 : 4, kNV = D == 128 ? 3 : 4;
  static constexpr uint32_t kQHalf = N * 128, kQBytes = kHalves * kQHalf;
  static constexpr uint32_t kPBytes = kTile * 128;
  // V before P: for head_dim 64 the product reads 64 rows of M past each V
  // stage (their results are not used), which have to be shared memory of ours
  static constexpr uint32_t kK = 0, kV = kK + kNK * kTileBytes, kP = kV + kNV * kTileBytes;
  static constexpr uint32_t kQ = kP + 2 * kPBytes;
  static constexpr uint32_t kSmem = kQ + 2 * kQBytes;
  static constexpr uint32_t kTmem = N == 16 ? 64 : N == 32 ? 128 : 256;
  static constexpr uint32_t kS = 0, kO = 2 * N;  // TMEM columns: S^T of even and odd tiles, O^T of even and odd units
};

struct BarsFew : RingBars {
  unsigned long long s_full[2], p_full[2], pv_done[2], o_free[2], done;
};

template <int C>
__device__ __forceinline__ void tmem_st(uint32_t addr, const float (&v)[C]) {
#pragma unroll
  for (int i = 0; i < C; i += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(v[i]), "f"(v[i + 1]),
                 "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]), "f"(v[i + 6]), "f"(v[i + 7]), "r"(addr + i)
                 : "memory");
  tmem_st_wait();
}

// The threads of a softmax group meet; the softmax threads of both.
__device__ __forceinline__ void soft_sync(int group) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ void both_sync() { asm volatile("barrier.cta.sync 3, 256;" ::: "memory"); }
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

// dst[k] = sum of v[k] over the warp: at each step a lane hands half of its
// columns to its partner (31 shuffles for 32 columns instead of 160).
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

template <int D, int N, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
k_tree_attn_few(const TreeAttnParams p, const __grid_constant__ TreeAttnMaps maps) {
  using G = GeomFew<D, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) BarsFew b;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_odd[2][8];           // nodes whose V holds an infinity or NaN, of even and odd units
  __shared__ __align__(16) float s_mb[N];  // the rows' references (log2 units)
  __shared__ __align__(16) float s_f[N];   // rescale factors
  __shared__ __align__(16) float s_part[4][N];
  uint32_t(*const s_word)[N] = reinterpret_cast<uint32_t(*)[N]>(s_part);  // mask words (a tile's step between uses of s_part)
  const int tid = threadIdx.x, warp = __shfl_sync(DC_FULL_MASK, tid >> 5, 0), lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);

  if (tid == 0) {
    init_ring<G>(b);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b.s_full[i]), 1);
      mbar_init(smem_u32(&b.p_full[i]), kSoft / 32);
      mbar_init(smem_u32(&b.pv_done[i]), 1);
      mbar_init(smem_u32(&b.o_free[i]), kSoft / 32);
    }
    mbar_init(smem_u32(&b.done), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows past the unit's are zeros: their scores are 0 and outgrow nothing
  for (uint32_t i = tid * 16; i < 2 * G::kQBytes; i += kThreads * 16)
    *reinterpret_cast<uint4 *>(smem + G::kQ + i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (warp == kLoadWarp && lane == 0) prefetch_maps(maps);
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), G::kTmem);
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
    constexpr uint32_t kIdS = F16 ? idesc_f16(128, N) : idesc_bf16(128, N);
    constexpr uint32_t kIdO = kIdS | (1u << 15) | (1u << 16);  // A is M-major, B is N-major
    UnitIter it(p, false);
    Unit w;
    bool ok = true;
    // O^T (+)= V^T P^T of tile t, the first of the block's unit number `unit` if `first`
    auto pv = [&](int t, bool first, int unit) {
      const int vs = t % G::kNV;
      const bool go = bar_wait(smem_u32(&b.v_full[vs]), (t / G::kNV) & 1, &s_abort, p.err) &&
                      (!first || unit < 2 || bar_wait(smem_u32(&b.o_free[unit & 1]), ((unit >> 1) - 1) & 1, &s_abort, p.err)) &&
                      bar_wait(smem_u32(&b.p_full[t & 1]), (t >> 1) & 1, &s_abort, p.err);
      if (!__all_sync(DC_FULL_MASK, go)) return false;
      tc_fence_after();
      const uint32_t sv = mn_major_lo(sbase + G::kV + vs * G::kTileBytes);
      const uint32_t sp = mn_major_lo(sbase + G::kP + (t & 1) * G::kPBytes);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ss(tmem + G::kO + (unit & 1) * N, sv + k * (2048 >> 4), sp + k * (2048 >> 4), kIdO, (!first || k > 0) ? 1u : 0u);
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
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tmem + G::kS + (g & 1) * N, sk + (((k >> 2) * G::kHalfBytes + (k & 3) * 32) >> 4),
                   sq + (((k >> 2) * G::kQHalf + (k & 3) * 32) >> 4), kIdS, k > 0 ? 1u : 0u);
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
    constexpr int C = N / 2;  // this group's rows: columns col0 .. col0 + C - 1
    const int group = warp >> 2, quad = warp & 3, t = tid & (kGroup - 1), col0 = group * C;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + col0;
    const int R = p.tile_rows;
    float c = p.scale * kLog2e;
    const bool flip = c < 0.f, zero = c == 0.f;
    c = zero ? 1.f : fabsf(c);
    bool ok = true;
    auto wait = [&](unsigned long long *bar, int phase) {
      if (ok) ok = __all_sync(DC_FULL_MASK, bar_wait(smem_u32(bar), phase & 1, &s_abort, p.err));
    };
    // A unit's output, unnormalised, leaves for the join after the first tile
    // of the unit that follows, whose products go to the other half of O, so
    // that the tensor core and the copies go on meanwhile.
    Unit done = {};
    int done_g = -1, done_unit = 0;                  // that unit's last tile (-1: none), its number
    bool seen_tree = false, done_tree = false;       // the unit has tree tiles: its s_odd holds
    auto slot_of = [&](const Unit &u) {              // the unit's rows among the partial results
      const int64_t item = ((int64_t)u.n * p.kv_heads + u.h) * p.mtiles + u.mt;
      return (item * p.max_chunks + u.chunk) * N;
    };
    auto finish = [&] {
      const int par = done_unit & 1;
      wait(&b.pv_done[done_g & 1], done_g >> 1);
      tc_fence_after();
      float o[C];
      tmem_ld<C>(trow + G::kO + par * N, o);
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&b.o_free[par]));
      float *part = reinterpret_cast<float *>(p.part_o) + (slot_of(done) + col0) * D + t;  // [row][D]
      if (t < D && ok) {
#pragma unroll
        for (int k = 0; k < C; ++k) part[k * D] = o[k];
        if (done_tree) {
          // infinities and NaN of the nodes that a row sees
#pragma unroll 1
          for (int q = 0; q < (p.T + 31) / 32; ++q)
#pragma unroll 1
            for (uint32_t r = s_odd[par][q]; r; r &= r - 1) {
              const int j = __ffs(r) - 1;
              const uint32_t e = p.v_new[done.n * p.vn_sn + (q * 32 + j) * p.vn_st + done.h * p.vn_sh + t];
              if (!nonfinite2<F16>(e)) continue;
#pragma unroll 1
              for (int k = 0; k < C && col0 + k < R; ++k)
                if ((tree_sees(p, done.n, done.len, done.mt * p.tile_nodes + (col0 + k) / p.group, q) >> j) & 1u)
                  part[k * D] += unpack_lo<F16>(e);
            }
        }
      }
      __syncwarp();
      done_g = -1;
    };
    while (it.next(w)) {
      if (w.ntiles == 0) continue;
      const int node0 = w.mt * p.tile_nodes;
      ++live;
      float l[C];  // the rows' sums over this thread's tokens
#pragma unroll
      for (int k = 0; k < C; ++k) l[k] = 0.f;
      seen_tree = false;
      for (int i = 0; i < w.ntiles; ++i, ++g) {
        const int tile = w.tile0 + i;
        const bool tree = tile >= w.nctx;
        const int tok0 = (tree ? tile - w.nctx : tile) * kTile;
        const int valid = min(kTile, (tree ? w.len : w.ctx) - tok0);
        wait(&b.s_full[g & 1], g >> 1);
        if (valid < kTile || tree) {
          if (group == 0) {  // the first group cleans V for both
            wait(&b.v_full[g % G::kNV], g / G::kNV);
            bool bad = false;
            if (ok) bad = clean_v_row<D, F16>(smem + G::kV + (g % G::kNV) * G::kTileBytes + t * 128, t < valid, tree);
            if (tree) {
              const uint32_t bits = __ballot_sync(DC_FULL_MASK, bad);
              both_sync();  // the words' last readers (two units back) are done
              if (lane == 0) s_odd[(live - 1) & 1][tok0 / 32 + warp] = bits;
            }
          } else if (tree) {
            both_sync();
          }
          if (tree) both_sync();
          seen_tree |= tree;
        }
        if (g >= 2) wait(&b.pv_done[g & 1], (g >> 1) - 1);  // P's buffer is free
        tc_fence_after();
        float v[C];
        // once, or once more when a score has outgrown its row's reference
        for (bool renew = false;;) {
          tmem_ld<C>(trow + G::kS + (g & 1) * N, v);
          if (flip | zero) {
#pragma unroll
            for (int k = 0; k < C; ++k) v[k] = zero ? 0.f : -v[k];
          }
          if (tree) {
            // this warp's 32 nodes are one word of each row's mask: lane k fetches row k's
            if (lane < C) {
              const int row = col0 + lane;
              s_word[quad][row] = row < R ? tree_sees(p, w.n, w.len, node0 + row / p.group, tok0 / 32 + quad) : 0u;
            }
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
          } else if (t >= valid) {
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
            if (t < C) {
              const int k = col0 + t;
              const float m = fmaxf(fmaxf(s_part[0][k], s_part[1][k]), fmaxf(s_part[2][k], s_part[3][k])) * c;
              const float old = s_mb[k];
              s_mb[k] = fmaxf(old, m);
              s_f[k] = m > old ? ex2(old - m) : 1.f;
            }
            soft_sync(group);
#pragma unroll
            for (int k = 0; k < C; ++k) l[k] *= s_f[col0 + k];
            if (i > 0) {
              wait(&b.pv_done[(g - 1) & 1], (g - 1) >> 1);
              tc_fence_after();
              float o[C];
              const uint32_t to = trow + G::kO + ((live - 1) & 1) * N;
              tmem_ld<C>(to, o);
#pragma unroll
              for (int k = 0; k < C; ++k) o[k] *= s_f[col0 + k];
              tmem_st<C>(to, o);
            }
          } else if (i == 0) {
            // a unit begins with the best of four tokens' scores as the references
            if (lane == 0) {
#pragma unroll
              for (int k = 0; k < C; k += 4)
                *reinterpret_cast<float4 *>(&s_part[quad][col0 + k]) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
            soft_sync(group);
            if (t < C) {
              const int k = col0 + t;
              const float m = fmaxf(fmaxf(s_part[0][k], s_part[1][k]), fmaxf(s_part[2][k], s_part[3][k])) * c;
              s_mb[k] = fabsf(m) < INFINITY ? m : kNone;
            }
            soft_sync(group);
          }
          // exponents against the references, in v's place
          float grow[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            const float4 mb = *reinterpret_cast<const float4 *>(&s_mb[col0 + k]);
            v[k] = fmaf(v[k], c, -mb.x), v[k + 1] = fmaf(v[k + 1], c, -mb.y);
            v[k + 2] = fmaf(v[k + 2], c, -mb.z), v[k + 3] = fmaf(v[k + 3], c, -mb.w);
            grow[0] = fmaxf(grow[0], v[k]), grow[1] = fmaxf(grow[1], v[k + 1]);
            grow[2] = fmaxf(grow[2], v[k + 2]), grow[3] = fmaxf(grow[3], v[k + 3]);
          }
          if (renew || !soft_any(group, fmaxf(fmaxf(grow[0], grow[1]), fmaxf(grow[2], grow[3])) > kRescale)) break;
          renew = true;
        }
        uint8_t *prow = smem + G::kP + (g & 1) * G::kPBytes + t * 128;
#pragma unroll
        for (int k = 0; k < C; k += 8) {
          float e[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            e[x] = ex2(v[k + x]);
            l[k + x] += e[x];
          }
          *reinterpret_cast<uint4 *>(prow + ((((col0 + k) >> 3) ^ (t & 7)) * 16)) =
              make_uint4(pack2<F16>(e[0], e[1]), pack2<F16>(e[2], e[3]), pack2<F16>(e[4], e[5]), pack2<F16>(e[6], e[7]));
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&b.p_full[g & 1]));
        if (i == 0 && done_g >= 0) finish();
      }
      warp_col_sums<C>(l, s_part[quad] + col0);
      soft_sync(group);
      if (t < C && ok) {
        const int k = col0 + t;
        p.part_ml[slot_of(w) + k] = make_float2(s_mb[k], (s_part[0][k] + s_part[1][k]) + (s_part[2][k] + s_part[3][k]));
      }
      soft_sync(group);
      done = w, done_g = g - 1, done_unit = live - 1, done_tree = seen_tree;
    }
    if (done_g >= 0) finish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_abort && warp >= kLoadWarp && lane == 0) drain_copies<G>(b, warp - kLoadWarp, g, live);
  if (warp == kMmaWarp) tmem_dealloc(tmem, G::kTmem);
}

template <int D, int N, bool F16>
cudaError_t launch(const TreeAttnParams &p, const TreeAttnMaps &maps, unsigned grid, cudaStream_t st) {
  const size_t smem = GeomFew<D, N>::kSmem + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(k_tree_attn_few<D, N, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k_tree_attn_few<D, N, F16><<<grid, kThreads, smem, st>>>(p, maps);
  return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t launch_n(const TreeAttnParams &p, const TreeAttnMaps &maps, unsigned grid, cudaStream_t st) {
  return p.part_rows == 16   ? launch<D, 16, F16>(p, maps, grid, st)
         : p.part_rows == 32 ? launch<D, 32, F16>(p, maps, grid, st)
                             : launch<D, 64, F16>(p, maps, grid, st);
}

}  // namespace

cudaError_t launch_tree_attention_few(const TreeAttnParams &p, const TreeAttnMaps &maps, unsigned grid,
                                      cudaStream_t st) {
  if (p.head_dim == 128) return p.f16 ? launch_n<128, true>(p, maps, grid, st) : launch_n<128, false>(p, maps, grid, st);
  return p.f16 ? launch_n<64, true>(p, maps, grid, st) : launch_n<64, false>(p, maps, grid, st);
}

}  // namespace dc
