// sample.cu -- one token per row: temperature, top-k, top-p, min-p, and the
// draw from a given uniform.
//
// With d_v = max x - x_v and w_v = e^{-d_v / t}: the kept set of top-k and
// top-p is a prefix of the order (value descending, id ascending), so it is
// given by its last value and, among the tokens of that value, its last id;
// min-p is a bound on d.  The token is the smallest id whose cumulative kept
// weight exceeds u times the kept total.
//
// One cluster of blocks a row.  Its blocks bring their slices of the row into
// shared memory once (DRAM sees every logit once) and take from there:
//   the maximum;
//   a histogram of d, its linear bins a 2048th of the row's range, merged
//     over the cluster: of each 16-byte vector's best token for top-k (the
//     k-th best vector bounds the k-th best token from below), of all tokens
//     for top-p;
//   the few candidates around the border, collected in the first block;
//   and, unless top-k leaves only those, the weights: summed over all tokens,
//     over those surely kept, and per 512 tokens for the draw.
// The first block sorts the candidates, finds the border exactly, and draws:
// the 512 tokens by their sums, then the token in them.
// What this does not cover the first block does alone, in about eight passes
// over the row: top_k over kTopkMost, or over the row's 16-byte vectors, of a
// larger vocabulary; borders with more tokens around them than the list holds;
// an infinite maximum, one near the type's lowest value, or one that over the
// temperature is past 10^38.  The bins follow the least vector maximum, so a
// vector of tokens masked with a finite value far below the others leaves the
// live ones in a few bins, and such rows go there too (-inf does not count).
//
// Weights are summed as 64-bit integers in units of 2^-40 (V <= 2^20 of them
// stay below 2^60), up to 16 of one thread's first in fp32: the same sums
// whatever the cluster's size and the blocks' timing.  A token below half a
// unit counts as far as its thread's 16 reach one.  e^{-d / t} is taken as
// 2^-z with z = d / (t ln 2) carried with its rounding error: a row's border
// can lie where a token has 10^-6 of the mass, and a bias of 10^-7 common to
// all weights beyond it would move it.
//
// 512 rows of 151936 bf16 logits (155 MB, 23 us of bytes), in a graph: 172 us
// with rows of all kinds, 200 with top-p alone, 135 with top-k alone, 97 with neither.  Half of the issue slots are used; the rest
// goes to steps that only the first block takes (the decision 8,000 cycles,
// sort and draw 16,000 of a top-p row's 140,000), to shared atomics of the
// histogram that meet in a bank (27,000) and to blocks that end at different
// times (2.25 waves).  16 rows: 27 us, all of it latency between the phases.
// The first block alone: 0.32 ms for 16 rows with top_k 1000, 1.0 ms for 512;
// 0.95 ms for 16 rows whose top-p border more than kList tokens share.  With
// 272 tokens masked at -1e4, 16 rows of top_p 0.9 take 0.69 ms (30 us without),
// 512 rows 2.3 ms (0.23).
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace dc {
namespace {

typedef unsigned long long u64;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBins = 2048;      // histogram bins
constexpr int kList = 1088;      // candidates the list holds (its 8704 bytes also hold the histogram)
constexpr int kTopkMost = 512;   // largest top_k of the candidate path
constexpr int kChunk = 512;      // tokens of a partial sum (one warp)
constexpr int kMostBlocks = 8;   // blocks of a cluster
// Bytes of a slice held in shared memory.  Three blocks an SM leave about 62 KB
// beside the list; 40 KB is what a thread loads at once (kAtOnce vectors).  An
// eighth of 151936 bf16 logits fits, of 200008 not: 16 rows with top_p 0.9 take
// 30 and 50 us.
constexpr size_t kMostSlice = 40 * 1024;

// Larger key <=> larger value; -0 and +0 share a key, NaN counts as -inf.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return x != x ? 0x007FFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Sum over the block; s: kWarps entries.
__device__ __forceinline__ u64 block_sum(u64 v, u64 *s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(DC_FULL_MASK, v, o);
  __syncthreads();
  if (lane == 0) s[warp] = v;
  __syncthreads();
  u64 r = 0;
  for (int w = 0; w < kWarps; ++w) r += s[w];
  return r;
}

template <bool F32>
struct SampleRow {
  const void *x;
  float mx, ch, cl, dmax;
  uint32_t key;  // kept: order key above `key`, or equal and id <= last
  int last;
  __device__ float value(int v) const {
    const float f = F32 ? static_cast<const float *>(x)[v]
                        : bf16_bits_to_float(static_cast<const uint16_t *>(x)[v]);
    return f != f ? -INFINITY : f;
  }
  // e^{-d / t}; 0 below 2^-64.  d / (t ln 2) as a product with its rounding
  // error, so that weights of large d keep fp32's relative accuracy and carry
  // no common bias.
  __device__ float share(float v) const {
    const float d = v == mx ? 0.f : mx - v;
    const float zh = d * ch;
    if (!(zh < 64.f)) return 0.f;
    const float zl = fmaf(d, cl, fmaf(d, ch, -zh));
    const float w = exp2f(-zh);
    return fmaf(-w * 0.693147180559945f, zl, w);
  }
  // In units of 2^-40, and of 2^-54 (512 of these stay below 2^64).
  __device__ u64 weight(float v) const { return __float2ull_rn(share(v) * 1099511627776.f); }
  __device__ u64 fine_weight(float v) const { return __float2ull_rn(share(v) * 18014398509481984.f); }
  __device__ bool kept(float v, int i) const {
    const uint32_t k = order_key(v);
    return (k > key || (k == key && i <= last)) && (v == mx || mx - v <= dmax);
  }
};

// ---------------------------------------------------------------- clusters
// (relaxed: publishes nothing)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Address of this block's shared `p` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void *p, int rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return d;
}
__device__ __forceinline__ void put32(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void put64(uint32_t at, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t get32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add32(uint32_t at, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(at), "r"(v) : "memory");
  return old;
}

// Inclusive scan over the block (T: u64, double or int); s: kWarps entries.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(DC_FULL_MASK, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += s[w];
  return v;
}
// The lowest thread with `hit`, and its values; -1 if none.
__device__ __forceinline__ int block_first(bool hit, int *s) {
  __syncthreads();
  if (threadIdx.x == 0) *s = kThreads;
  __syncthreads();
  if (hit) atomicMin(s, (int)threadIdx.x);
  __syncthreads();
  return *s == kThreads ? -1 : *s;
}

// Sorts list[0, n) descending, the whole block.  A bitonic network whose
// merges begin with mirrored pairs, so that every exchange puts the larger
// entry first: what a power of two above n would add are least entries that
// never move, and pairs that reach past n are left out.  Pairs closer than 64
// stay within a warp's 64 entries: those steps need no block barrier.
__device__ __forceinline__ void sort_desc(u64 *list, int n) {
  __syncthreads();
  int pairs = 1;
  while (2 * pairs < n) pairs <<= 1;
  for (int k = 2; k <= 2 * pairs; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      const int to = 2 * j == k ? k - 1 : j;  // the partner's distance, in bits: mirrored or plain
      for (int i = threadIdx.x; i < pairs; i += kThreads) {
        const int a = ((i & ~(j - 1)) << 1) | (i & (j - 1)), b = a ^ to;
        if (b >= n) continue;
        const u64 x = list[a], y = list[b];
        if (x < y) list[a] = y, list[b] = x;
      }
      if (j > 32 || (j == 1 && k >= 64)) __syncthreads();
      else __syncwarp();
    }
  __syncthreads();
}

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats in a register pair, one instruction for both.
__device__ __forceinline__ u64 two(float a, float b) {
  u64 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 of_two(u64 x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
__device__ __forceinline__ u64 fma_two(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ u64 mul_two(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 add_two(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum_two(u64 x) {
  const float2 f = of_two(x);
  return f.x + f.y;
}
// 1 where a >= b, else 0.
__device__ __forceinline__ float at_least(float a, float b) {
  float d;
  asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// What a block is told by the first one.
struct Orders {
  int step;        // kCollect, kWeigh (and collect), kStop
  float from, to;  // distances from the maximum: collect [from, to), weigh as surely kept what is nearer than `from`
};
enum { kStop, kCollect, kWeigh };

// The least integer that is at least p * mass; what the uniform u is of the
// mass, below it.  (By one thread: a block's 256 would keep the SM's few
// 64-bit units busy for some 700 cycles.)
__device__ __forceinline__ u64 target_of(float u, u64 mass) {
  const u64 target = (u64)((double)u * (double)mass);
  return target >= mass ? mass - 1 : target;
}
__device__ __forceinline__ u64 share_of(float p, u64 mass) {
  return (u64)ceil((double)fmaxf(p, 0.f) * (double)mass);
}

struct SampleShared {
  u64 red[kWarps];
  float redf[kWarps];
  int redi[kWarps];
  int first;
  float mx[kMostBlocks], low[kMostBlocks];
  uint32_t arg[kMostBlocks];
  u64 sure[kMostBlocks], all[kMostBlocks];
  u64 need, target;     // (first block)
  uint32_t listed;      // (first block) candidates of the cluster
  uint32_t mine, base;  // candidates of this block, and where they go in the first block's list
  float dmax;
  Orders orders;
  int again;            // by mass, after a try: the border was not among the candidates
};

// Maxima that a NaN goes through.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The vector at `at` that reaches past the row's V logits: -inf there.
template <bool F32>
__device__ __noinline__ uint4 fetch_tail(const uint8_t *row, int at, int V) {
  uint32_t x[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (F32) {
      x[q] = at + q < V ? reinterpret_cast<const uint32_t *>(row)[at + q] : 0xFF800000u;
    } else {
      const uint32_t a = at + 2 * q < V ? reinterpret_cast<const uint16_t *>(row)[at + 2 * q] : 0xFF80u;
      const uint32_t b = at + 2 * q + 1 < V ? reinterpret_cast<const uint16_t *>(row)[at + 2 * q + 1] : 0xFF80u;
      x[q] = a | b << 16;
    }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}
// NaN to -inf.
template <bool F32>
__device__ __noinline__ uint4 without_nan(uint4 w) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (F32) {
      if ((x[q] & 0x7FFFFFFFu) > 0x7F800000u) x[q] = 0xFF800000u;
    } else {
      if ((x[q] & 0x7FFFu) > 0x7F80u) x[q] = (x[q] & 0xFFFF0000u) | 0xFF80u;
      if ((x[q] & 0x7FFF0000u) > 0x7F800000u) x[q] = (x[q] & 0xFFFFu) | 0xFF800000u;
    }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// E logits of a 16-byte vector as floats.
template <bool F32>
__device__ __forceinline__ void unpack(const uint4 &w, float (&f)[F32 ? 4 : 8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) f[i] = __uint_as_float(x[i]);
    else f[2 * i] = __uint_as_float(x[i] << 16), f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
}

// The general path, one block, for what the candidate list does not hold: the
// border's key a byte at a time by histograms (of counts for top-k, of masses
// for top-p), its id and the drawn token by sums of kChunk tokens.  The
// tokens of a key have one weight, so how many of them are kept follows by a
// division.  About eight passes over the row.
template <bool F32>
struct General {
  SampleRow<F32> r;
  int V;
  uint32_t *hist;  // [2][4][256]
  u64 *chunk_all;  // [chunks]
  SampleShared &s;

  static constexpr int E = F32 ? 4 : 8;
  __device__ uint4 load(int i) const {  // vector i of the row; -inf past its end
    const uint8_t *row = static_cast<const uint8_t *>(r.x);
    return (i + 1) * E <= V ? __ldg(reinterpret_cast<const uint4 *>(row) + i) : fetch_tail<F32>(row, i * E, V);
  }
  __device__ void values(const uint4 &w, float (&f)[E]) const {
    unpack<F32>(w, f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = f[e] != f[e] ? -INFINITY : f[e];
  }
  // f(value, id) of this thread's tokens, four vectors in flight
  template <typename F>
  __device__ void pass(F f) const {
    const int vecs = (V + E - 1) / E;
    for (int i0 = threadIdx.x; i0 < vecs; i0 += 4 * kThreads) {
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = load(min(i0 + q * kThreads, vecs - 1));
#pragma unroll 1
      for (int q = 0; q < 4 && i0 + q * kThreads < vecs; ++q) {
        float x[E];
        values(q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : w[3], x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int v = (i0 + q * kThreads) * E + e;
          if (v < V) f(x[e], v);
        }
      }
    }
  }
  // The largest key whose tokens and those of larger keys reach `need` (> 0)
  // together; `of` a token's share (LIMBS: 1 if below 2^11, 4 if below 2^44).
  // before: the share of larger keys.  A bin is summed in limbs of 11 bits (2^20
  // tokens of one stay below 2^31): 32-bit atomics on shared memory are the fast ones.
  template <int LIMBS, typename F>
  __device__ uint32_t border(u64 need, F of, u64 &before) const {
    const int tid = threadIdx.x;
    uint32_t *h = hist + (tid >> 5 & 1) * 1024;  // two copies: half as many warps meet in a bin
    uint32_t key = 0;
    before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int i = tid; i < 2048; i += kThreads) hist[i] = 0;
      __syncthreads();
      pass([&](float x, int v) {
        const uint32_t q = order_key(x);
        if (shift == 24 || q >> (shift + 8) == key) {
          const u64 n = of(x, v);
#pragma unroll
          for (int l = 0; l < LIMBS; ++l) {
            const uint32_t part = (uint32_t)(n >> (11 * l)) & 2047u;
            if (part) atomicAdd(&h[l * 256 + (q >> shift & 255u)], part);
          }
        }
      });
      __syncthreads();
      u64 n = 0;
#pragma unroll
      for (int l = 0; l < LIMBS; ++l)
        n += ((u64)hist[l * 256 + 255 - tid] + hist[1024 + l * 256 + 255 - tid]) << (11 * l);
      const u64 upto = block_scan(n, s.red);
      const int who = block_first(before + upto >= need, &s.first);
      if (tid == max(who, 0)) s.target = upto - n;
      __syncthreads();
      before += s.target;
      key = key << 8 | (uint32_t)(255 - max(who, 0));
    }
    return key;
  }
  // The smallest id up to which the tokens' shares are more than aim(total).
  template <typename F, typename A>
  __device__ int find(F of, A aim, u64 &total) const {
    const int tid = threadIdx.x, lane = tid & 31, chunks = (V + kChunk - 1) / kChunk;
    __syncthreads();
    for (int ch = tid >> 5; ch < chunks; ch += kWarps) {
      constexpr int kVecs = kChunk / E / 32;
      const int i = ch * (kChunk / E) + lane, last = (V - 1) / E;
      uint4 w[kVecs];
      u64 n = 0;
#pragma unroll
      for (int q = 0; q < kVecs; ++q) w[q] = load(min(i + q * 32, last));
#pragma unroll
      for (int q = 0; q < kVecs; ++q) {
        float x[E];
        values(w[q], x);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((i + q * 32) * E + e < V) n += of(x[e], (i + q * 32) * E + e);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(DC_FULL_MASK, n, o);
      if (lane == 0) chunk_all[ch] = n;
    }
    __syncthreads();
    const int per = (chunks + kThreads - 1) / kThreads;
    u64 mine = 0;
    for (int i = tid * per; i < min(chunks, (tid + 1) * per); ++i) mine += chunk_all[i];
    const u64 upto = block_scan(mine, s.red);
    __syncthreads();
    if (tid == kThreads - 1) s.red[0] = upto, s.target = aim(upto);
    __syncthreads();
    total = s.red[0];
    u64 target = s.target, cum = upto - mine;
    int at = -1;
    for (int i = tid * per; i < min(chunks, (tid + 1) * per) && at < 0; ++i) {
      if (cum + chunk_all[i] > target) at = i;
      else cum += chunk_all[i];
    }
    int who = block_first(at >= 0, &s.first);
    if (tid == max(who, 0)) s.redi[0] = max(at, 0), s.target = target - cum;
    __syncthreads();
    const int v = s.redi[0] * kChunk + tid * (kChunk / kThreads);
    target = s.target;
    u64 n[kChunk / kThreads], sum = 0;
#pragma unroll
    for (int q = 0; q < kChunk / kThreads; ++q) {
      n[q] = v + q < V ? of(r.value(v + q), v + q) : 0;
      sum += n[q];
    }
    u64 before = block_scan(sum, s.red) - sum;
    at = -1;
#pragma unroll
    for (int q = 0; q < kChunk / kThreads; ++q) {
      before += n[q];
      if (at < 0 && before > target) at = v + q;
    }
    who = block_first(at >= 0, &s.first);
    if (tid == max(who, 0)) s.redi[0] = max(at, 0);
    __syncthreads();
    return s.redi[0];
  }
  __device__ int operator()(int k, float tp, float u, u64 &total) {
    u64 before, n;
    auto count = [](float, int) -> u64 { return 1; };
    if (k < V) {
      const uint32_t key = border<1>((u64)k, count, before);
      r.last = find([&](float x, int) -> u64 { return order_key(x) == key; }, [&](u64) { return (u64)k - before - 1; }, n);
      r.key = key;
    }
    if (tp < 1.f) {
      const SampleRow<F32> top = r;  // what top-k left
      auto in = [&](float x, int v) { return order_key(x) > top.key || (order_key(x) == top.key && v <= top.last); };
      auto mass = [&](float x, int v) -> u64 { return in(x, v) ? top.weight(x) : 0; };
      u64 all = 0;
      pass([&](float x, int v) { all += mass(x, v); });
      all = block_sum(all, s.red);
      __syncthreads();
      if (threadIdx.x == 0) s.need = max(share_of(tp, all), (u64)1);
      __syncthreads();
      const u64 need = s.need;
      const uint32_t key = border<4>(need, mass, before);
      const u64 w = top.weight(key_value(key));
      const u64 more = (need - before + w - 1) / w;  // tokens of the border's key; w > 0, its mass is
      r.last = find([&](float x, int v) -> u64 { return order_key(x) == key && in(x, v); }, [&](u64) { return more - 1; }, n);
      r.key = key;
    }
    return find([&](float x, int v) -> u64 { return r.kept(x, v) ? r.weight(x) : 0; },
                [&](u64 all) { return target_of(u, all); }, total);
  }
};
// (s.need: the kept total)
template <bool F32>
__device__ __noinline__ int sample_general(SampleRow<F32> r, int V, int k, float tp, float u, uint32_t *hist,
                                           u64 *chunk_all, SampleShared &s) {
  General<F32> g{r, V, hist, chunk_all, s};
  u64 total;
  const int token = g(k, tp, u, total);
  if (threadIdx.x == 0) s.need = total;
  return token;
}

template <bool F32, bool HELD>
__global__ void __launch_bounds__(kThreads, 3)
k_sample(const SampleParams p, int blocks, int slice, int chunks_all) {
  constexpr int E = F32 ? 4 : 8, kSize = F32 ? 4 : 2;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ SampleShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.z, V = p.V;
  u64 *list = reinterpret_cast<u64 *>(smem);                 // [kList]; before the candidates: the histogram
  uint32_t *hist = reinterpret_cast<uint32_t *>(smem);       // [kBins]
  u64 *chunk_all = list + kList;                             // [chunks_all], the first block's: kept weight a chunk
  const int share = kBins / blocks;                          // merged bins that each block holds
  uint32_t *merged = reinterpret_cast<uint32_t *>(chunk_all + (chunks_all + 1) / 2 * 2);  // (16-byte steps: `data` is read in vectors)
  uint8_t *data = reinterpret_cast<uint8_t *>(merged + share);
  const int64_t row = blockIdx.x;
  const uint8_t *src = static_cast<const uint8_t *>(p.logits) + row * p.stride * kSize;
  const int v0 = rank * slice, v1 = min(V, v0 + slice), nv = max(0, v1 - v0);
  const int nch = (nv + kChunk - 1) / kChunk, vecs = nch * (kChunk / E);
  float t = p.temperature ? p.temperature[row] : 1.f, tp = p.top_p ? p.top_p[row] : 1.f, u = p.u[row];
  const float mp = p.min_p ? p.min_p[row] : 0.f;
  int k = p.top_k ? p.top_k[row] : 0;
  cluster_arrive_relaxed();  // this block is there

  bool nan = false;  // (not held) this thread's block met a NaN
  // A vector of the slice; past the vocabulary's end: -inf.
  auto fetch = [&](int i) {
    const int at = v0 + i * E;
    return at + E <= V ? ld_stream_v4(src + (int64_t)at * kSize) : fetch_tail<F32>(src, at, V);
  };
  auto vec = [&](int i) {
    if constexpr (HELD) return reinterpret_cast<const uint4 *>(data)[i];
    else return nan ? without_nan<F32>(fetch(i)) : fetch(i);
  };
  // a vector's largest logit; NaN if it has one
  auto best_of = [&](const uint4 &w) {
    float a, b;
    if constexpr (F32) {
      a = max_nan(__uint_as_float(w.x), __uint_as_float(w.y)), b = max_nan(__uint_as_float(w.z), __uint_as_float(w.w));
    } else {
      const uint32_t m = bf16x2_max_nan(bf16x2_max_nan(w.x, w.y), bf16x2_max_nan(w.z, w.w));
      a = __uint_as_float(m << 16), b = __uint_as_float(m & 0xFFFF0000u);
    }
    return max_nan(a, b);
  };

  // ---------------------------------------------------------------- the maximum
  // `low`: the least of the vectors' maxima, which sets the histogram's range
  float mx = -INFINITY, low = INFINITY;
  constexpr int kAtOnce = 10;  // vectors a thread has in flight: a 40 KB slice at once
  for (int i0 = tid; i0 < vecs; i0 += kAtOnce * kThreads) {
    uint4 w[kAtOnce];
    if (v0 + vecs * E <= V) {
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (i0 + q * kThreads < vecs) w[q] = ld_stream_v4(src + (int64_t)(v0 + (i0 + q * kThreads) * E) * kSize);
    } else {
#pragma unroll 1
      for (int q = 0; q < kAtOnce; ++q)
        if (i0 + q * kThreads < vecs) {
          const uint4 x = fetch(i0 + q * kThreads);
          if constexpr (HELD) reinterpret_cast<uint4 *>(data)[i0 + q * kThreads] = x;
        }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (i0 + q * kThreads < vecs) w[q] = HELD ? reinterpret_cast<uint4 *>(data)[i0 + q * kThreads] : fetch(i0 + q * kThreads);
    }
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      if (i0 + q * kThreads >= vecs) continue;
      float m = best_of(w[q]);
      if (m != m) {
        nan = true;
        w[q] = without_nan<F32>(w[q]);
        m = best_of(w[q]);
      }
      if constexpr (HELD) reinterpret_cast<uint4 *>(data)[i0 + q * kThreads] = w[q];
      mx = fmaxf(mx, m);
      low = fminf(low, m == -INFINITY ? INFINITY : m);
    }
  }
  mx = warp_max(mx), low = -warp_max(-low);
  if (lane == 0) s.redf[warp] = mx, s.redi[warp] = __float_as_int(low);
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  if (t != t) t = 1.f;
  if (k <= 0 || k > V) k = V;
  if (tp != tp) tp = 1.f;
  if (!(u > 0.f)) u = 0.f;
  if (tid == 0) {  // (one thread: 256 would keep the few 64-bit units busy for 6 us)
    s.listed = s.mine = 0;
    s.dmax = mp > 0.f ? __double2float_rd(fmax(0.0, -(double)t * log((double)fminf(mp, 1.f)))) : INFINITY;
  }
  nan = __syncthreads_or(nan);
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s.redf[w]), low = fminf(low, __int_as_float(s.redi[w]));
  cluster_wait();  // every block of the cluster is there
  if (tid < blocks) {
    put32(peer(&s.mx[rank], tid), __float_as_uint(mx));
    put32(peer(&s.low[rank], tid), __float_as_uint(low));
  }
  cluster_sync();
  for (int b = 0; b < blocks; ++b) mx = fmaxf(mx, s.mx[b]), low = fminf(low, s.low[b]);

  if (mx == -INFINITY) {
    if (rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      if (p.logprob) p.logprob[row] = -INFINITY;
    }
    return;
  }
  if (t <= 0.f) {
    // the lowest id of the maximum
    uint32_t arg = 0xFFFFFFFFu;
    for (int i = tid; i < vecs; i += kThreads) {
      float f[E];
      unpack<F32>(vec(i), f);
#pragma unroll
      for (int e = E - 1; e >= 0; --e)
        if (f[e] == mx) arg = min(arg, (uint32_t)(v0 + i * E + e));
    }
    arg = __reduce_min_sync(DC_FULL_MASK, arg);
    __syncthreads();
    if (lane == 0) s.redi[warp] = (int)arg;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) arg = min(arg, (uint32_t)s.redi[w]);
    if (tid == 0) put32(peer(&s.arg[rank], 0), arg);
    cluster_sync();
    if (rank == 0 && tid == 0) {
      for (int b = 0; b < blocks; ++b) arg = min(arg, s.arg[b]);
      p.tokens[row] = (int)arg;
      if (p.logprob) p.logprob[row] = 0.f;
    }
    return;
  }
  SampleRow<F32> r;
  r.x = src;
  r.mx = mx;
  // log2 e / t in two floats: the quotient, and the quotient of what it leaves
  const float ts = fmaxf(t, 1e-30f);
  r.ch = __fdiv_rn(1.44269502f, ts);
  r.cl = __fdiv_rn(fmaf(-r.ch, ts, 1.44269502f) + 1.92596303e-8f, ts);
  if (!(ts < 3e38f)) r.ch = r.cl = 0.f;
  r.dmax = s.dmax;
  r.key = 0, r.last = V;

  // ---------------------------------------------------------------- which way
  const bool small = V <= kList;                       // everything is a candidate
  const bool by_list = small || (k < V && k <= kTopkMost);
  const bool by_mass = !by_list && k == V && tp < 1.f;
  const bool whole = k == V && tp >= 1.f && !small;    // min-p at most
  bool general = !(by_list || by_mass || whole) || mx == INFINITY || mx < -3e38f || ts > 1e30f;
  // bins of d, 1.5 times the range down to the least vector maximum
  const float range = 1.5f * fmaxf(mx - low, 1e-6f), scale = (float)kBins / range;
  if (!small && !whole && !(range < 1e30f)) general = true;
  // (the weighing pass takes distances of up to a step of the logits' type below
  // the maximum: over t they have to stay finite)
  if (!by_list && !(r.ch * fabsf(mx) < 1e38f)) general = true;
  if (!general && (by_mass || (by_list && !small))) {
    // histogram: the bin is the integer below 2^23 + d scale, by the addition's own rounding
    const float dtop = (float)(kBins - 1) / scale;
    auto bin_of = [&](float x) { return __float_as_uint(fmaf(fminf(mx - x, dtop), scale, 8388608.f)) & (2 * kBins - 1); };
    auto count = [&](const uint4 &w) {
      if (by_list) {
        const float m = best_of(w);
        if (m > -INFINITY) atomicAdd(&hist[min(bin_of(m), (uint32_t)kBins - 1)], 1u);
      } else {
        float f[E];
        unpack<F32>(w, f);
#pragma unroll
        for (int e = 0; e < E; ++e) atomicAdd(&hist[bin_of(f[e])], 1u);  // (-inf: the last bin)
      }
    };
    for (int i0 = tid; i0 < vecs; i0 += 4 * kThreads) {  // four loads in flight
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i0 + q * kThreads < vecs) w[q] = vec(i0 + q * kThreads);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i0 + q * kThreads < vecs) count(w[q]);
    }
  }
  if (!general && (by_mass || (by_list && !small))) {
    cluster_sync();
    for (int i = tid; i < share; i += kThreads) {
      uint32_t n = 0;
      for (int b = 0; b < blocks; ++b) n += get32(peer(&hist[rank * share + i], b));
      merged[i] = n;
    }
    cluster_sync();
  }

  // The first block decides; the others do as told, any number of times.
  constexpr int kPer = kBins / kThreads;
  u64 sure_all = 0, all_all = 0;  // (first block) weight surely kept, and of all tokens
  int tries = 0;
  int b1 = 0, b2 = kBins;         // (first block) bins collected: [b1, b2)
  int edge = 0;                   // (first block) after a try: the end of [b1, b2) that the border lies beyond,
  u64 edge_mass = 0;              // and the exact mass before it
  while (true) {
    if (rank == 0) {
      Orders o{kStop, 0.f, 0.f};
      if (general) {
      } else if (whole) {
        o = Orders{kWeigh, INFINITY, INFINITY};
      } else if (small) {
        o = Orders{kCollect, 0.f, INFINITY};
      } else {
        // this thread's bins
        int n[kPer], sum = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const int bin = tid * kPer + q;
          n[q] = (int)get32(peer(&merged[bin % share], bin / share));
          sum += n[q];
        }
        if (by_list) {
          // the bin where the vectors' count reaches k: its tokens and the better ones hold the k best
          int upto = block_scan(sum, s.redi) - sum, bin = kBins - 1;
          bool hit = false;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            if (!hit && upto < k && upto + n[q] >= k) hit = true, bin = tid * kPer + q;
            upto += n[q];
          }
          const int who = block_first(hit, &s.first);
          if (tid == max(who, 0)) s.redi[0] = who < 0 ? kBins : bin + 1;
          __syncthreads();
          const int to = s.redi[0];
          o = Orders{kCollect, 0.f, to >= kBins ? INFINITY : ((float)to + 0.5f) / scale};  // (half a bin to spare)
        } else {
          const float per_bin = range / (float)kBins * r.ch;
          // masses by the bins' middles; after a first try, from its exact masses on
          float m[kPer], mass = 0.f;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            m[q] = n[q] ? (float)n[q] * ex2_approx(-(float)(tid * kPer + q) * per_bin) : 0.f;
            mass += m[q];
          }
          const float cum = block_scan(mass, s.redf);
          __syncthreads();
          if (tid == kThreads - 1) s.redf[0] = cum;
          if (tries && tid == edge / kPer) {  // what the exact mass says the middles' are off by
            float before = cum - mass;
            for (int q = 0; q < edge % kPer; ++q) before += m[q];
            s.redf[1] = __ull2float_rn(edge_mass) * 0x1p-40f - before;
          }
          __syncthreads();
          const float need = fmaxf(tp, 0.f) * (tries ? __ull2float_rn(all_all) * 0x1p-40f : s.redf[0]);
          float before = cum - mass + (tries ? s.redf[1] : 0.f);
          int bin = kBins - 1;
          bool hit = false;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            if (!hit && before + m[q] >= need) hit = true, bin = tid * kPer + q;
            before += m[q];
          }
          const int who = block_first(hit, &s.first);
          __syncthreads();
          if (tid == max(who, 0)) s.redi[0] = who < 0 ? kBins - 1 : bin;
          __syncthreads();
          bin = s.redi[0];
          // as many bins around it as an eighth of the list takes (the first
          // try then finds the border in all but 2 rows of a hundred; with
          // half of the list in one more, but the pass and the sort take 2 to
          // 7 us longer); the counts before each bin go where the candidates
          // will be
          int upto = block_scan(sum, s.redi) - sum;
          uint32_t *cnt = reinterpret_cast<uint32_t *>(list);  // [kBins + 1] (the histogram is merged)
          static_assert(kList * 8 >= (kBins + 1) * 4, "");
          __syncthreads();
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            cnt[tid * kPer + q] = (uint32_t)upto;
            upto += n[q];
          }
          if (tid == kThreads - 1) cnt[kBins] = (uint32_t)upto;
          __syncthreads();
          int wide = 0;  // the widest 2^i - 1 bins to both sides that fit
          for (int x = 1; x < kBins; x = 2 * x + 1) {
            if (cnt[min(kBins, bin + x + 1)] - cnt[max(0, bin - x)] > kList / 8) break;
            wide = x;
          }
          b1 = max(0, bin - wide), b2 = min(kBins, bin + wide + 1);
          const uint32_t inside = cnt[b2] - cnt[b1];
          __syncthreads();
          if (inside > kList || tries == 4 || edge >= kBins) general = true;
          else o = Orders{kWeigh, ((float)b1 - 0.5f) / scale, b2 >= kBins ? INFINITY : ((float)b2 - 0.5f) / scale};
        }
      }
      if (tid == 0) s.listed = 0;
      if (tid < blocks) {
        put32(peer(&s.mine, tid), 0u);
        put32(peer(&s.orders.step, tid), (uint32_t)o.step);
        put32(peer(&s.orders.from, tid), __float_as_uint(o.from));
        put32(peer(&s.orders.to, tid), __float_as_uint(o.to));
      }
    }
    cluster_sync();
    const Orders o = s.orders;
    if (o.step == kStop) {
      if (rank != 0) return;
      break;
    }
    // ---------------------------------------------------------------- the pass over the tokens
    // candidates gather in this block's list, then go to the first one's (one
    // by one, each would wait for the reply from the other block's memory)
    uint32_t *count = rank == 0 ? &s.listed : &s.mine;
    // the tokens of vector i, logits f, whose bits are set (from registers: a
    // second read of the row costs a warp a wait on L2; a held one is near)
    auto collect = [&](int i, uint32_t bits, const float (&f)[E]) {
      uint32_t at = atomicAdd(count, (uint32_t)__popc(bits));
      auto put = [&](int e, float x) {
        if (at < kList) list[at] = (u64)order_key(x) << 32 | (0xFFFFFFFFu - (uint32_t)(v0 + i * E + e));
        ++at;
      };
      if constexpr (HELD) {
        for (; bits; bits &= bits - 1) {
          const int e = __ffs(bits) - 1;
          put(e, F32 ? reinterpret_cast<const float *>(data)[i * E + e]
                     : bf16_bits_to_float(reinterpret_cast<const uint16_t *>(data)[i * E + e]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (bits >> e & 1u) put(e, f[e]);
      }
    };
    if (o.step == kCollect) {
      for (int i0 = tid; i0 < vecs; i0 += 4 * kThreads) {
        uint4 w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (i0 + q * kThreads < vecs) w[q] = vec(i0 + q * kThreads);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (i0 + q * kThreads >= vecs) continue;
          const float m = best_of(w[q]);
          if (m > -INFINITY && mx - m < o.to) {
            float f[E];
            unpack<F32>(w[q], f);
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) bits |= f[e] > -INFINITY && mx - f[e] < o.to ? 1u << e : 0u;
            collect(i0 + q * kThreads, bits, f);
          }
        }
      }
    } else {
      // a weight of 2^-100 stands for the lesser ones and for -inf: logits are
      // raised to `least`, below the maximum however small 100 / ch
      float least = fminf(mx - 100.f / r.ch, key_value(order_key(mx) - 1));
      uint32_t least2 = __float_as_uint(least);
      if constexpr (!F32) {  // the next bf16 below it, twice
        least2 = (least2 + (least < 0.f ? 0xFFFFu : 0u)) >> 16;
        least = __uint_as_float(least2 << 16);
        least2 |= least2 << 16;
      }
      const bool min_p = r.dmax < INFINITY;
      const u64 nmx2 = two(-mx, -mx), ch2 = two(r.ch, r.ch), nch2 = two(-r.ch, -r.ch), ncl2 = two(-r.cl, -r.cl),
                nln2 = two(-0.693147180559945f, -0.693147180559945f), minus2 = two(-1.f, -1.f);
      // y > -from as y >= the next float
      const float nearest = key_value(order_key(-o.from) + 1);
      // what the weights beyond the border's candidates stay below
      const float w_to = ex2_approx(-fminf(o.to, mx - least) * r.ch) * (1.f - 0x1p-12f);
      u64 sure = 0, all = 0;
      // a lane's sum (at most 16) in units of 2^-40, as 2^22 hi + lo
      auto fixed = [](float x, uint32_t &hi, uint32_t &lo) {
        const float y = x * 262144.f, f = floorf(y);
        hi = (uint32_t)f;
        lo = __float2uint_rn((y - f) * 4194304.f);
      };
      constexpr int kVecs = kChunk / E / 32;  // of a lane in a chunk
      uint4 ahead[kVecs];                     // (not held) the next chunk's
      if (!HELD && warp < nch) {
#pragma unroll
        for (int q = 0; q < kVecs; ++q) ahead[q] = vec(warp * (kChunk / E) + q * 32 + lane);
      }
      for (int ch = warp; ch < nch; ch += kWarps) {
        u64 kept2 = 0, certain2 = 0, total2 = 0;  // of this lane's 16 tokens
#pragma unroll
        for (int q = 0; q < kVecs; ++q) {
          const int i = ch * (kChunk / E) + q * 32 + lane;
          if (HELD) ahead[q] = vec(i);
          const uint32_t x[4] = {ahead[q].x, ahead[q].y, ahead[q].z, ahead[q].w};
          if (!HELD && ch + kWarps < nch) ahead[q] = vec(i + kWarps * (kChunk / E));
          float y[E];
          u64 w[E / 2];
#pragma unroll
          for (int h = 0; h < E / 2; ++h) {
            u64 pair;
            if constexpr (F32) {
              pair = two(fmaxf(__uint_as_float(x[2 * h]), least), fmaxf(__uint_as_float(x[2 * h + 1]), least));
            } else {
              const uint32_t v = bf16x2_max(x[h], least2);
              pair = two(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
            }
            // with y = -d: 2^-z, z = d (ch + cl) = zh + zl
            const u64 y2 = add_two(pair, nmx2), nzh = mul_two(y2, ch2), zl = fma_two(y2, ncl2, fma_two(y2, nch2, nzh));
            const float2 z = of_two(nzh);
            const u64 w0 = two(ex2_approx(z.x), ex2_approx(z.y));
            w[h] = fma_two(mul_two(w0, nln2), zl, w0);
            const float2 f = of_two(y2);
            y[2 * h] = f.x, y[2 * h + 1] = f.y;
          }
          if (by_mass) {
            float most = 0.f;  // the largest weight not surely kept
#pragma unroll
            for (int h = 0; h < E / 2; ++h) {
              total2 = add_two(total2, w[h]);
              const u64 in = two(at_least(y[2 * h], nearest), at_least(y[2 * h + 1], nearest));
              const u64 wk = mul_two(w[h], in);
              const float2 out = of_two(fma_two(wk, minus2, w[h]));
              most = fmaxf(most, fmaxf(out.x, out.y));
              w[h] = wk;
            }
            if (most >= w_to) {
              uint32_t bits = 0;
              float v[E];
              unpack<F32>(make_uint4(x[0], x[1], x[2], x[3]), v);
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const float far = mx - v[e];
                bits |= far >= o.from && far < o.to && v[e] > -INFINITY ? 1u << e : 0u;
              }
              if (bits) collect(i, bits, v);
            }
          }
          if (min_p) {  // the draw leaves out what min-p does; the border counts it
#pragma unroll
            for (int h = 0; h < E / 2; ++h) {
              certain2 = add_two(certain2, w[h]);
              w[h] = mul_two(w[h], two(at_least(y[2 * h], -r.dmax), at_least(y[2 * h + 1], -r.dmax)));
            }
          }
#pragma unroll
          for (int h = 0; h < E / 2; ++h) kept2 = add_two(kept2, w[h]);
        }
        const float kept = sum_two(kept2), certain = sum_two(certain2), total = sum_two(total2);
        uint32_t hi, lo;
        fixed(kept, hi, lo);
        const u64 x = ((u64)__reduce_add_sync(DC_FULL_MASK, hi) << 22) + __reduce_add_sync(DC_FULL_MASK, lo);
        if (lane == 0) put64(peer(&chunk_all[v0 / kChunk + ch], 0), x);
        if (by_mass) {
          if (min_p) fixed(certain, hi, lo);
          sure += ((u64)hi << 22) + lo;
          fixed(total, hi, lo);
          all += ((u64)hi << 22) + lo;
        }
      }
      if (by_mass) {
        sure = block_sum(sure, s.red);
        all = block_sum(all, s.red);
        if (tid == 0) {
          put64(peer(&s.sure[rank], 0), sure);
          put64(peer(&s.all[rank], 0), all);
        }
      }
    }
    if (!whole && rank != 0) {
      __syncthreads();
      if (tid == 0) s.base = s.mine > 0 ? add32(peer(&s.listed, 0), s.mine <= kList ? s.mine : kList + 1u) : 0;
      __syncthreads();
      if (s.mine <= kList) {
        const uint32_t list0 = peer(list, 0);
        for (uint32_t i = tid; i < s.mine; i += kThreads)
          if (s.base + i < kList) put64(list0 + (s.base + i) * 8, list[i]);
      }
    }
    cluster_sync();
    if (by_list || whole) {
      if (rank != 0) return;
      break;
    }
    // by mass: is the border among the candidates?
    ++tries;
    if (rank == 0) {
      sure_all = all_all = 0;
      for (int b = 0; b < blocks; ++b) sure_all += s.sure[b], all_all += s.all[b];
      const int n = (int)min(s.listed, (uint32_t)kList);
      u64 m = 0;
      for (int i = tid; i < n; i += kThreads) m += r.weight(key_value((uint32_t)(list[i] >> 32)));
      m = block_sum(m, s.red);
      if (tid == 0) s.need = share_of(tp, all_all);
      __syncthreads();
      const u64 need = s.need;
      const bool in = s.listed <= kList && (sure_all < need || sure_all == 0) && sure_all + m >= need;
      if (sure_all >= need) edge = b1, edge_mass = sure_all;
      else edge = b2, edge_mass = sure_all + m;
      __syncthreads();
      // (not in `orders`: the next ones may be written while a block still reads this,
      // and a block that took their kStop for this one would leave under the writes)
      if (tid < blocks) put32(peer(&s.again, tid), in ? 0u : 1u);
    }
    cluster_sync();
    if (!s.again) {  // the others are done
      if (rank != 0) return;
      break;
    }
    __syncthreads();
  }

  // ---------------------------------------------------------------- the draw (first block)
  int token = -1;
  u64 total = 0;
  if (!general && by_list && s.listed > kList) general = true;
  if (general) {
    token = sample_general<F32>(r, V, k, tp, u, hist, chunk_all, s);
    total = s.need;  // (thread 0 uses it)
  } else {
    // candidates in order
    const int n = whole ? 0 : (int)s.listed;
    if (n > 0) sort_desc(list, n);
    const auto weight_at = [&](int i) { return r.weight(key_value((uint32_t)(list[i] >> 32))); };
    // the first `m` of them stay: the shortest prefix with mass `need`
    int m = n;
    if (by_list) m = min(n, k);
    const int per = (n + kThreads - 1) / kThreads;
    if (n > 0 && tp < 1.f) {
      u64 mine = 0;
      for (int q = 0; q < per; ++q) {
        const int i = tid * per + q;
        if (i < m) mine += weight_at(i);
      }
      const u64 upto = block_scan(mine, s.red);
      __syncthreads();
      if (tid == kThreads - 1) s.need = share_of(tp, by_list ? upto : all_all);
      __syncthreads();
      const u64 need = s.need;
      u64 cum = (by_list ? 0 : sure_all) + upto - mine;
      int at = -1;
      for (int q = 0; q < per && at < 0; ++q) {
        const int i = tid * per + q;
        if (i >= m) break;
        cum += weight_at(i);
        if (cum >= need) at = i + 1;
      }
      const int who = block_first(at > 0, &s.first);
      __syncthreads();
      if (tid == max(who, 0)) s.redi[0] = who < 0 ? m : at;
      __syncthreads();
      m = s.redi[0];
    }
    if (by_list) {
      // the kept ones, by id, and the draw among them
      for (int i = tid; i < n; i += kThreads) {
        const u64 e = list[i];
        const float x = key_value((uint32_t)(e >> 32));
        const bool keep = i < m && (x == mx || mx - x <= r.dmax);
        list[i] = keep ? (e & 0xFFFFFFFFull) << 32 | (e >> 32) : 0;  // ids are stored complemented: descending is by id
      }
      sort_desc(list, n);
      const auto by_id = [&](int i) { return list[i] ? r.weight(key_value((uint32_t)list[i])) : 0; };
      u64 mine = 0;
      for (int q = 0; q < per; ++q)
        if (tid * per + q < n) mine += by_id(tid * per + q);
      const u64 upto = block_scan(mine, s.red);
      __syncthreads();
      if (tid == kThreads - 1) s.red[0] = upto, s.target = target_of(u, upto);
      __syncthreads();
      total = s.red[0];
      u64 target = s.target;
      u64 cum = upto - mine;
      int at = -1;
      for (int q = 0; q < per && at < 0; ++q) {
        const int i = tid * per + q;
        if (i >= n) break;
        cum += by_id(i);
        if (cum > target) at = i;
      }
      const int who = block_first(at >= 0, &s.first);
      if (tid == who) s.redi[0] = (int)(0xFFFFFFFFu - (uint32_t)(list[at] >> 32));
      __syncthreads();
      token = s.redi[0];
    } else {
      if (by_mass) {
        // the kept candidates join their chunks; the border as a rule for any token
        for (int i = tid; i < m; i += kThreads) {
          const float x = key_value((uint32_t)(list[i] >> 32));
          if (x == mx || mx - x <= r.dmax) atomicAdd(&chunk_all[(0xFFFFFFFFu - (uint32_t)list[i]) / kChunk], weight_at(i));
        }
        r.key = (uint32_t)(list[m - 1] >> 32), r.last = (int)(0xFFFFFFFFu - (uint32_t)list[m - 1]);
        __syncthreads();
      }
      u64 mine = 0;
      const int cper = (chunks_all + kThreads - 1) / kThreads;
      for (int q = 0; q < cper; ++q)
        if (tid * cper + q < chunks_all) mine += chunk_all[tid * cper + q];
      const u64 upto = block_scan(mine, s.red);
      __syncthreads();
      if (tid == kThreads - 1) s.red[0] = upto, s.target = target_of(u, upto);
      __syncthreads();
      total = s.red[0];
      u64 target = s.target;
      u64 cum = upto - mine;
      int at = -1;
      for (int q = 0; q < cper && at < 0; ++q) {
        const int i = tid * cper + q;
        if (i >= chunks_all) break;
        if (cum + chunk_all[i] > target) at = i;
        else cum += chunk_all[i];
      }
      const int who = block_first(at >= 0, &s.first);
      if (tid == who) s.redi[0] = at, s.red[0] = target - cum;
      __syncthreads();
      const int v = s.redi[0] * kChunk + tid * (kChunk / kThreads);
      target = s.red[0] << 14;
      // in the chunk: in finer units, since the chunk's sum, rounded 16 tokens
      // at a time, may have mass where each token alone rounds to none
      u64 w[kChunk / kThreads], sum = 0;
#pragma unroll
      for (int q = 0; q < kChunk / kThreads; ++q) {
        const float x = v + q < V ? r.value(v + q) : -INFINITY;
        w[q] = v + q < V && x > -INFINITY && r.kept(x, v + q) ? r.fine_weight(x) : 0;
        sum += w[q];
      }
      u64 before = block_scan(sum, s.red) - sum;
      int found = -1, last = -1;
#pragma unroll
      for (int q = 0; q < kChunk / kThreads; ++q) {
        before += w[q];
        if (w[q] > 0) {
          last = v + q;
          if (found < 0 && before > target) found = v + q;
        }
      }
      const int got = block_first(found >= 0, &s.first);
      if (got >= 0) {
        if (tid == got) s.redi[0] = found;
      } else {
        // the chunk's sum was above its tokens': the last one
        if (tid == 0) s.redi[0] = -1;
        __syncthreads();
        if (last >= 0) atomicMax(&s.redi[0], last);
      }
      __syncthreads();
      token = s.redi[0];
    }
  }
  if (tid == 0) {
    p.tokens[row] = token;
    const float x = r.value(min(max(token, 0), V - 1)), d = x == mx ? 0.f : mx - x;
    if (p.logprob) p.logprob[row] = -(d / ts) - logf(__ull2float_rn(total) * 0x1p-40f);
  }
}

template <bool F32>
cudaError_t launch(const SampleParams &p, cudaStream_t st) {
  constexpr int kSize = F32 ? 4 : 2, kSms = 152;
  // Blocks of a cluster: as many as keep the launch within the three blocks an
  // SM holds and a slice at 16 KB or more, and two at least.  A block's fixed
  // steps cost as much as some 10,000 tokens, so many rows want few blocks, but
  // one block alone waits too long on its own loads.  512 rows of 151936 bf16
  // logits: 200 / 168 / 181 / 218 us with 1 / 2 / 4 / 8 blocks; 100 rows: 82 /
  // 58 / 62 us with 2 / 4 / 8; 16 rows: 52 / 37 / 26 us with 2 / 4 / 8.
  int blocks = kMostBlocks;
  while (blocks > 2 && (int64_t)p.rows * blocks > 3 * kSms) blocks /= 2;
  while (blocks > 1 && (int64_t)p.V * kSize < (int64_t)blocks << 14) blocks /= 2;
  const int chunks = (p.V + kChunk - 1) / kChunk, slice = (chunks + blocks - 1) / blocks * kChunk;
  const bool held = (size_t)slice * kSize <= kMostSlice;
  const size_t smem = kList * 8 + (size_t)(chunks + 1) / 2 * 16 + kBins / blocks * 4 + (held ? (size_t)slice * kSize : 0);
  const auto kernel = held ? k_sample<F32, true> : k_sample<F32, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_ex(kernel, dim3((unsigned)p.rows, 1, (unsigned)blocks), dim3(kThreads), smem, st, false, (unsigned)blocks,
                   p, blocks, slice, chunks);
}

}  // namespace

cudaError_t launch_sample(const SampleParams &p, bool f32, cudaStream_t st) {
  return f32 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace dc
