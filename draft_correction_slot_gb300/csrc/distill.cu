// distill.cu -- distillation loss of the drafter against the target's top
// logits, and its gradient.
//
// With z = x / T, q = softmax(z), p the teacher's shares of its K tokens,
// P = sum p:
//   loss = T^2 sum_k p_k (log p_k - z_{id_k} + lse(z))
//   d loss / d x_v = T (P q_v - sum_{k: id_k = v} p_k).
//
// Bound by the bytes of the rows: the loss reads each logit once, the gradient
// reads and writes once, and the two in one step (k_step) still read once: a
// cluster of blocks holds a whole row in registers between the sum and the
// gradient.  The log-sum-exp is a running (maximum, sum) a thread, in a fixed
// order of threads, warps and blocks, so that a row's result depends on
// nothing but the row.
//
// A row's slices are the blocks': a block of k_step (the loss alone is k_step
// without its gradient) takes up to HOLD 16-byte vectors a thread; the cluster's
// size follows from the row's bytes alone.  The teacher's tokens belong to the
// slice they lie in: each block sums its tokens' terms and writes their gradient
// after its slice's, from the logit as it was read, so that the gradient may
// overwrite the logits.
//
// 480 rows of 151936 bf16 logits: loss 43 us (146 MB, floor 22), gradient 58 us
// (292 MB, 43), both in one step 89 us (43); 2000 rows of 32001 fp32: step 128 us
// (512 MB, 76).  Longer rows keep fewer blocks an SM: 480 rows of 200008 take a
// step 142 us (57), of 262144 156 us (74).  A block's loads, barriers and stores follow one another, and
// the registers that hold the row allow four blocks an SM to fill the gaps.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace dc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxK = 1024;
constexpr int kMostBlocks = 8;
constexpr float kLog2e = 1.44269504088896340736f;

template <bool F32>
struct Row;
template <>
struct Row<false> {
  static constexpr int kVec = 8;
  using T = uint16_t;
  __device__ static float get(const T *x, int v) { return bf16_bits_to_float(x[v]); }
  __device__ static void put(T *x, int v, float f) { x[v] = (uint16_t)bf16_rn_bits(f); }
  __device__ static void unpack(const uint4 &w, float (&f)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(x[i] << 16), f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    return make_uint4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Row<true> {
  static constexpr int kVec = 4;
  using T = float;
  __device__ static float get(const T *x, int v) { return x[v]; }
  __device__ static void put(T *x, int v, float f) { x[v] = f; }
  __device__ static void unpack(const uint4 &w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (relaxed: there is nothing to publish; a release at entry cost a step of 2000 rows of 32001 fp32 logits 7 us of 129)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Puts v at `p` in block `rank` of the cluster.
__device__ __forceinline__ void put_peer(const float *p, int rank, float v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// s: kWarps entries; every thread gets the same value, warps in order.
__device__ __forceinline__ float block_reduce(float v, float *s, bool maximum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = maximum ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if (lane == 0) s[warp] = v;
  __syncthreads();
  float r = s[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) r = maximum ? fmaxf(r, s[w]) : r + s[w];
  return r;
}

struct Teacher {
  float red[kWarps];
  float logp[kMaxK];  // log p_k
  float x[kMaxK];     // the logit of a token in this block's slice; then its gradient
  int4 id4[kMaxK / 4];  // tokens, -1: left out
  __device__ int &id(int k) { return reinterpret_cast<int *>(id4)[k]; }
  // sum of p_j over the k's with this token
  __device__ float share(int token, int K) const {
    float sum = 0.f;
    for (int j = 0; j < (K + 3) / 4; ++j) {
      const int4 t = id4[j];
      if (t.x == token || t.y == token || t.z == token || t.w == token) {
        const int ts[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (ts[q] == token && logp[4 * j + q] != -INFINITY) sum += expf(logp[4 * j + q]);
      }
    }
    return sum;
  }
};

// The row's teacher into shared memory, and the logits of its tokens in [v0,
// v1); returns P.
template <bool F32>
__device__ __forceinline__ float load_teacher(const DistillParams &p, int64_t row, float inv_t, int v0, int v1,
                                              Teacher &s) {
  const typename Row<F32>::T *x = static_cast<const typename Row<F32>::T *>(p.logits) + row * p.stride;
  const int tid = threadIdx.x;
  float m = -INFINITY;
  if (tid < 3 && p.K + tid < (p.K + 3) / 4 * 4) s.id(p.K + tid) = -1;
  for (int k = tid; k < p.K; k += kThreads) {
    const int id = p.ids[row * p.K + k];
    const bool ok = id >= 0 && id < p.V;
    const float t = ok ? p.teacher[row * p.K + k] * inv_t : -INFINITY;
    s.id(k) = ok ? id : -1;
    s.logp[k] = t;
    if (id >= v0 && id < v1) s.x[k] = Row<F32>::get(x, id);
    m = fmaxf(m, t);
  }
  float lse;
  if (p.teacher_lse) {
    lse = p.teacher_lse[row];
  } else {
    m = block_reduce(m, s.red, true);
    float sum = 0.f;
    if (m != -INFINITY)
      for (int k = tid; k < p.K; k += kThreads) sum += expf(s.logp[k] - m);
    sum = block_reduce(sum, s.red, false);
    lse = m == -INFINITY ? 0.f : m + logf(sum);
  }
  float mass = 0.f;
  for (int k = tid; k < p.K; k += kThreads) {
    if (s.logp[k] != -INFINITY) s.logp[k] -= lse;
    mass += s.logp[k] == -INFINITY ? 0.f : expf(s.logp[k]);
  }
  return block_reduce(mass, s.red, false);  // (its barriers also publish id and logp)
}

// What a block says of its slice: maximum, sum of e^{(x - max) / T}, and of
// its teacher's tokens sum p_k (log p_k - (x_k - max) / T) and sum p_k.
struct Part {
  float max, sum, loss, mass;
};

// Loss, and with GRAD the gradient in the same pass.  A cluster a row.
template <bool F32, bool GRAD, int HOLD>
__global__ void __launch_bounds__(kThreads, HOLD <= 10 ? 4 : 2)
k_step(const DistillParams p, int blocks, int slice_vecs) {
  using R = Row<F32>;
  constexpr int E = R::kVec;
  __shared__ Teacher s;
  __shared__ Part s_part[kMostBlocks];
  const int tid = threadIdx.x, rank = blockIdx.z;
  const int64_t row = blockIdx.x;
  const typename R::T *x = static_cast<const typename R::T *>(p.logits) + row * p.stride;
  const int v0 = rank * slice_vecs * E, v1 = min(p.V, v0 + slice_vecs * E);
  const int nv = max(0, v1 - v0), full = nv / E;  // whole vectors; the rest singly
  const uint4 *src = reinterpret_cast<const uint4 *>(x + v0);
  const float inv_t = 1.f / p.temperature, c = inv_t * kLog2e;
  cluster_arrive_relaxed();  // this block is there

  // the slice: HOLD vectors a thread in flight and kept, what is beyond them read again
  uint4 held[HOLD];
#pragma unroll
  for (int q = 0; q < HOLD; ++q)
    if (tid + q * kThreads < full) held[q] = __ldcs(src + tid + q * kThreads);
  const float mass = load_teacher<F32>(p, row, inv_t, v0, v1, s);  // (under the loads)

  float m = -INFINITY, sum = 0.f;  // of 2^{c x}, relative to 2^{c m}
  auto add = [&](const uint4 &w) {
    float f[E];
    R::unpack(w, f);
    float top = f[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, f[e]);
    if (top > m) sum *= ex2((m - top) * c), m = top;
    const float b = m == -INFINITY ? 0.f : m;
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) part += ex2((f[e] - b) * c);  // (the difference first: large z keep their accuracy)
    sum += part;
  };
#pragma unroll
  for (int q = 0; q < HOLD; ++q)
    if (tid + q * kThreads < full) add(held[q]);
#pragma unroll 4
  for (int i = tid + HOLD * kThreads; i < full; i += kThreads) add(__ldcs(src + i));
  if (tid < nv - full * E) {
    const float f = R::get(x, v0 + full * E + tid);
    if (f > m) sum *= ex2((m - f) * c), m = f;
    if (f > -INFINITY) sum += ex2((f - m) * c);
  }
  const float bm = block_reduce(m, s.red, true);
  const float bs = block_reduce(m == -INFINITY ? 0.f : sum * ex2((m - bm) * c), s.red, false);
  const float ref = bm == -INFINITY ? 0.f : bm;
  float loss = 0.f, here = 0.f;
  for (int k = tid; k < p.K; k += kThreads) {
    const int id = s.id(k);
    if (id < v0 || id >= v1) continue;
    const float lp = s.logp[k], pk = lp == -INFINITY ? 0.f : expf(lp);
    here += pk;
    if (pk > 0.f) loss += pk * (lp - (s.x[k] - ref) * inv_t);
  }
  loss = block_reduce(loss, s.red, false);
  here = block_reduce(here, s.red, false);
  cluster_wait();  // every block of the cluster is there: its shared memory may be written
  if (tid == 0) {
    for (int b = GRAD ? 0 : blocks - 1; b < blocks; ++b) {
      const int to = GRAD ? b : 0;  // the loss alone: the first block only
      put_peer(&s_part[rank].max, to, bm);
      put_peer(&s_part[rank].sum, to, bs);
      put_peer(&s_part[rank].loss, to, loss);
      put_peer(&s_part[rank].mass, to, here);
    }
  }
  cluster_arrive();
  cluster_wait();
  if (!GRAD && rank != 0) return;
  float M = s_part[0].max, S = 0.f;
  for (int b = 1; b < blocks; ++b) M = fmaxf(M, s_part[b].max);
  for (int b = 0; b < blocks; ++b) S += s_part[b].max == -INFINITY ? 0.f : s_part[b].sum * ex2((s_part[b].max - M) * c);
  const float lse = M * inv_t + logf(S);
  if (rank == 0 && tid == 0) {
    float l = 0.f;
    for (int b = 0; b < blocks; ++b) {
      const Part q = s_part[b];
      // (log S on its own: the maxima's difference is exact where M / T + log S is rounded)
      if (q.mass > 0.f) l += q.loss + q.mass * ((M - (q.max == -INFINITY ? 0.f : q.max)) * inv_t + logf(S));
    }
    p.loss[row] = p.temperature * p.temperature * l;
    p.lse[row] = lse;
  }

  if constexpr (GRAD) {
    typename R::T *out = static_cast<typename R::T *>(p.grad) + row * p.grad_stride;
    uint4 *dst = reinterpret_cast<uint4 *>(out + v0);
    const float g = p.grad_loss[row] * p.temperature, gm = g * mass;
    for (int k = tid; k < p.K; k += kThreads) {
      const int id = s.id(k);
      if (id >= v0 && id < v1) s.x[k] = g == 0.f ? 0.f : g * (mass * expf(s.x[k] * inv_t - lse) - s.share(id, p.K));
    }
    auto gradient = [&](const uint4 &w) {
      float f[E];
      R::unpack(w, f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = gm == 0.f ? 0.f : gm * ex2(fmaf(f[e], inv_t, -lse) * kLog2e);
      return R::pack(f);
    };
    // (what a block reads again it read itself before, and nobody else writes it)
#pragma unroll
    for (int q = 0; q < HOLD; ++q)
      if (tid + q * kThreads < full) __stcs(dst + tid + q * kThreads, gradient(held[q]));
#pragma unroll 4
    for (int i = tid + HOLD * kThreads; i < full; i += kThreads) __stcs(dst + i, gradient(__ldcg(src + i)));
    if (tid < nv - full * E) {
      const int v = v0 + full * E + tid;
      R::put(out, v, gm == 0.f ? 0.f : gm * ex2(fmaf(R::get(x, v), inv_t, -lse) * kLog2e));
    }
    __syncthreads();
    for (int k = tid; k < p.K; k += kThreads)
      if (s.id(k) >= v0 && s.id(k) < v1) R::put(out, s.id(k), s.x[k]);
  }
}
// The gradient alone, from the loss call's lse: blocks of a row need nothing
// of each other.
template <bool F32>
__global__ void __launch_bounds__(kThreads) k_grad(const DistillParams p, int slice_vecs) {
  using R = Row<F32>;
  constexpr int E = R::kVec, kAtOnce = 8;
  __shared__ Teacher s;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const typename R::T *x = static_cast<const typename R::T *>(p.logits) + row * p.stride;
  typename R::T *out = static_cast<typename R::T *>(p.grad) + row * p.grad_stride;
  const int v0 = blockIdx.z * slice_vecs * E, v1 = min(p.V, v0 + slice_vecs * E);
  const int nv = max(0, v1 - v0), full = nv / E;
  const uint4 *src = reinterpret_cast<const uint4 *>(x + v0);
  uint4 *dst = reinterpret_cast<uint4 *>(out + v0);
  const float inv_t = 1.f / p.temperature;
  uint4 w[kAtOnce];
#pragma unroll
  for (int q = 0; q < kAtOnce; ++q)
    if (tid + q * kThreads < full) w[q] = __ldcs(src + tid + q * kThreads);
  const float lse = p.lse[row], g = p.grad_loss[row] * p.temperature;
  const float mass = load_teacher<F32>(p, row, inv_t, v0, v1, s);  // (under the loads)
  for (int k = tid; k < p.K; k += kThreads) {
    const int id = s.id(k);
    if (id >= v0 && id < v1) s.x[k] = g == 0.f ? 0.f : g * (mass * expf(s.x[k] * inv_t - lse) - s.share(id, p.K));
  }
  const float gm = g * mass;
  const float last = tid < nv - full * E ? R::get(x, v0 + full * E + tid) : 0.f;
  __syncthreads();  // every logit that is read singly has been read
  for (int i0 = tid; i0 < full; i0 += kAtOnce * kThreads) {
    if (i0 != tid) {
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (i0 + q * kThreads < full) w[q] = __ldcs(src + i0 + q * kThreads);
    }
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      if (i0 + q * kThreads >= full) continue;
      float f[E];
      R::unpack(w[q], f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = gm == 0.f ? 0.f : gm * ex2(fmaf(f[e], inv_t, -lse) * kLog2e);
      __stcs(dst + i0 + q * kThreads, R::pack(f));
    }
  }
  if (tid < nv - full * E) R::put(out, v0 + full * E + tid, gm == 0.f ? 0.f : gm * ex2(fmaf(last, inv_t, -lse) * kLog2e));
  __syncthreads();
  for (int k = tid; k < p.K; k += kThreads)
    if (s.id(k) >= v0 && s.id(k) < v1) R::put(out, s.id(k), s.x[k]);
}

template <bool F32>
cudaError_t launch(const DistillParams &p, cudaStream_t st) {
  constexpr int E = Row<F32>::kVec;
  const int vecs = (p.V + E - 1) / E;
  // Blocks a row, by its length alone: slices of at most 8 vectors a thread
  // (32 KB), up to eight of them.  A longer slice of the step takes up to 20
  // vectors a thread (fewer blocks an SM), what is beyond them is read twice.
  int blocks = 1;
  while (blocks < kMostBlocks && vecs > blocks * 8 * kThreads) blocks *= 2;
  const int slice = (vecs + blocks - 1) / blocks;
  const dim3 grid((unsigned)p.rows, 1, (unsigned)blocks), block(kThreads);
  if (!p.loss) return launch_ex(k_grad<F32>, grid, block, 0, st, false, 0, p, slice);
  const int hold = (slice + kThreads - 1) / kThreads;
  const auto kernel = !p.grad      ? k_step<F32, false, 10>
                      : hold <= 8  ? k_step<F32, true, 8>
                      : hold <= 10 ? k_step<F32, true, 10>
                                   : k_step<F32, true, 20>;
  return launch_ex(kernel, grid, block, 0, st, false, (unsigned)blocks, p, blocks, slice);
}

}  // namespace

cudaError_t launch_distill(const DistillParams &p, bool f32, cudaStream_t st) {
  return f32 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace dc
