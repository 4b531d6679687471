// sample.cu -- one token per row: temperature, top-k, top-p, min-p, and the
// draw from a given uniform.
//
// With d_v = max x - x_v and w_v = e^{-d_v / t}: the kept set of top-k and
// top-p is a prefix of the order (value descending, id ascending), so it is
// given by its last value and, among the tokens of that value, its last id;
// min-p is a bound on d.  The token is the smallest id whose cumulative kept
// weight exceeds u times the kept total.
//
// Weights are summed as 64-bit integers in units of 2^-40 (V <= 2^20 of them
// stay below 2^60): the sums are exact, so neither the threads' order nor
// how a row is split over them can change a token.
// One block a row; the last value and id are found by bisection, a pass over
// the row each step.
#include "common.cuh"
#include "kernels.h"

namespace dc {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
typedef unsigned long long u64;

// Larger key <=> larger value; -0 and +0 share a key, NaN counts as -inf.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return x != x ? 0x007FFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

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
  // e^{-d / t} in units of 2^-40.  d / (t ln 2) as a product with its
  // rounding error, so that weights of large d keep fp32's relative
  // accuracy and carry no common bias.
  __device__ u64 weight(float v) const {
    const float d = v == mx ? 0.f : mx - v;
    const float zh = d * ch;
    if (!(zh < 64.f)) return 0;
    const float zl = fmaf(d, cl, fmaf(d, ch, -zh));
    const float w = exp2f(-zh);
    return __float2ull_rn(fmaf(-w * 0.693147180559945f, zl, w) * 1099511627776.f);
  }
  __device__ bool kept(float v, int i) const {
    const uint32_t k = order_key(v);
    return (k > key || (k == key && i <= last)) && (v == mx || mx - v <= dmax);
  }
};

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleParams p) {
  __shared__ u64 s_red[kWarps];
  const int row = blockIdx.x, tid = threadIdx.x, V = p.V;
  SampleRow<F32> r;
  r.x = static_cast<const char *>(p.logits) + row * p.stride * (F32 ? 4 : 2);
  // the maximum and its lowest id, as one integer
  u64 best = 0;
  for (int v = tid; v < V; v += kThreads) {
    const u64 k = (u64)order_key(r.value(v)) << 32 | (uint32_t)(V - v);
    best = k > best ? k : best;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 k = __shfl_xor_sync(DC_FULL_MASK, best, o);
    best = k > best ? k : best;
  }
  if ((tid & 31) == 0) s_red[tid >> 5] = best;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) best = s_red[w] > best ? s_red[w] : best;
  const int arg = V - (int)(uint32_t)best;
  r.mx = r.value(arg);
  float t = p.temperature ? p.temperature[row] : 1.f;
  if (t != t) t = 1.f;
  if (r.mx == -INFINITY || t <= 0.f) {
    if (tid == 0) {
      p.tokens[row] = r.mx == -INFINITY ? -1 : arg;
      if (p.logprob) p.logprob[row] = r.mx == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }
  const double c = 1.4426950408889634 / fmax((double)t, 1e-30);
  r.ch = (float)c, r.cl = (float)(c - (double)r.ch);
  int k = p.top_k ? p.top_k[row] : 0;
  if (k <= 0 || k > V) k = V;
  float tp = p.top_p ? p.top_p[row] : 1.f, mp = p.min_p ? p.min_p[row] : 0.f;
  if (tp != tp) tp = 1.f;
  r.dmax = mp > 0.f ? __double2float_rd(fmax(0.0, -(double)t * log((double)fminf(mp, 1.f)))) : INFINITY;
  r.key = 0, r.last = V;

  // The shortest prefix of the order for which `over` (monotone in the
  // prefix) of its count and mass holds: its last value by bisection on the
  // key, then its last id.
  auto shortest = [&](auto over) {
    const uint32_t key0 = r.key;
    const int last0 = r.last;
    auto measure = [&](uint32_t key, int last) {
      u64 n = 0, m = 0;
      for (int v = tid; v < V; v += kThreads) {
        const float f = r.value(v);
        const uint32_t q = order_key(f);
        if ((q > key || (q == key && v <= last)) && (q > key0 || (q == key0 && v <= last0))) ++n, m += r.weight(f);
      }
      n = block_sum(n, s_red);
      m = block_sum(m, s_red);
      return over(n, m);
    };
    uint32_t lo = 0, hi = order_key(r.mx);  // largest key in [lo, hi] whose whole prefix is over
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      if (measure(mid, V)) lo = mid;
      else hi = mid - 1;
    }
    int a = 0, b = V - 1;  // smallest id
    while (a < b) {
      const int mid = a + (b - a) / 2;
      if (measure(lo, mid)) b = mid;
      else a = mid + 1;
    }
    r.key = lo, r.last = a;
  };
  if (k < V) shortest([&](u64 n, u64) { return n >= (u64)k; });
  auto mass_of = [&]() {
    u64 m = 0;
    for (int v = tid; v < V; v += kThreads) {
      const float f = r.value(v);
      const uint32_t q = order_key(f);
      if (q > r.key || (q == r.key && v <= r.last)) m += r.weight(f);
    }
    return block_sum(m, s_red);
  };
  if (tp < 1.f) {
    const double need = fmax((double)tp, 0.0) * (double)mass_of();
    shortest([&](u64 n, u64 m) { return n > 0 && (double)m >= need; });
  }
  u64 total = 0;
  for (int v = tid; v < V; v += kThreads) {
    const float f = r.value(v);
    if (r.kept(f, v)) total += r.weight(f);
  }
  total = block_sum(total, s_red);
  float u = p.u[row];
  if (!(u > 0.f)) u = 0.f;
  u64 target = (u64)((double)u * (double)total);  // below `total`
  if (target >= total) target = total - 1;
  int a = 0, b = V - 1;
  while (a < b) {
    const int mid = a + (b - a) / 2;
    u64 m = 0;
    for (int v = tid; v <= mid; v += kThreads) {
      const float f = r.value(v);
      if (r.kept(f, v)) m += r.weight(f);
    }
    if (block_sum(m, s_red) > target) b = mid;
    else a = mid + 1;
  }
  if (tid == 0) {
    p.tokens[row] = a;
    const float x = r.value(a), d = x == r.mx ? 0.f : r.mx - x;
    if (p.logprob) p.logprob[row] = (float)(-(double)d / fmax((double)t, 1e-30) - log((double)total * 0x1p-40));
  }
}

}  // namespace

cudaError_t launch_sample(const SampleParams &p, bool f32, cudaStream_t st) {
  if (f32) k_sample<true><<<p.rows, kThreads, 0, st>>>(p);
  else k_sample<false><<<p.rows, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dc
