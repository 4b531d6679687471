// distill.cu -- distillation loss of the drafter against the target's top
// logits, and its gradient.
//
// With z = x / T, q = softmax(z), p the teacher's shares of its K tokens,
// P = sum p:
//   loss = T^2 sum_k p_k (log p_k - z_{id_k} + lse(z))
//   d loss / d x_v = T (P q_v - sum_{k: id_k = v} p_k).
// One block a row; the row is read once for the log-sum-exp (a running
// maximum and sum a thread, joined at the end) and once for the gradient.
#include "common.cuh"
#include "kernels.h"

namespace dc {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxK = 1024;
constexpr float kLog2e = 1.44269504088896340736f;

template <bool F32>
struct Row;
template <>
struct Row<false> {
  using T = uint16_t;
  __device__ static float get(const T *x, int v) { return bf16_bits_to_float(x[v]); }
  __device__ static void put(T *x, int v, float f) { x[v] = (uint16_t)bf16_rn_bits(f); }
};
template <>
struct Row<true> {
  using T = float;
  __device__ static float get(const T *x, int v) { return x[v]; }
  __device__ static void put(T *x, int v, float f) { x[v] = f; }
};

__device__ __forceinline__ float block_reduce(float v, float *s, bool maximum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = maximum ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if (lane == 0) s[warp] = v;
  __syncthreads();
  float r = s[0];
  for (int w = 1; w < kWarps; ++w) r = maximum ? fmaxf(r, s[w]) : r + s[w];
  return r;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_distill(const DistillParams p) {
  using R = Row<F32>;
  __shared__ float s_red[kWarps], s_p[kMaxK], s_fix[kMaxK];
  __shared__ int s_id[kMaxK];
  const int row = blockIdx.x, tid = threadIdx.x;
  const typename R::T *x = static_cast<const typename R::T *>(p.logits) + row * p.stride;
  const float inv_t = 1.f / p.temperature;

  // the teacher's shares
  float tm = -INFINITY;
  for (int k = tid; k < p.K; k += kThreads) {
    const int id = p.ids[(int64_t)row * p.K + k];
    const bool ok = id >= 0 && id < p.V;
    s_id[k] = ok ? id : -1;
    s_p[k] = ok ? p.teacher[(int64_t)row * p.K + k] * inv_t : -INFINITY;  // log p_k, not yet normalised
    tm = fmaxf(tm, s_p[k]);
  }
  float t_lse;
  if (p.teacher_lse) {
    t_lse = p.teacher_lse[row];
  } else {
    tm = block_reduce(tm, s_red, true);
    float s = 0.f;
    if (tm != -INFINITY)
      for (int k = tid; k < p.K; k += kThreads) s += expf(s_p[k] - tm);
    s = block_reduce(s, s_red, false);
    t_lse = tm == -INFINITY ? 0.f : tm + logf(s);
  }
  float lse;
  if (p.loss) {
    float m = -INFINITY;
    for (int v = tid; v < p.V; v += kThreads) m = fmaxf(m, R::get(x, v));
    m = block_reduce(m, s_red, true);
    float s = 0.f;
    for (int v = tid; v < p.V; v += kThreads) s += exp2f((R::get(x, v) - m) * inv_t * kLog2e);
    s = block_reduce(s, s_red, false);
    lse = m * inv_t + logf(s);
  } else {
    lse = p.lse[row];
  }
  // loss and the corrections at the teacher's tokens
  const float g = p.grad ? p.grad_loss[row] * p.temperature : 0.f;
  float mass = 0.f, loss = 0.f;
  for (int k = tid; k < p.K; k += kThreads) {
    const float logp = s_p[k] - t_lse;
    const float pk = s_p[k] == -INFINITY ? 0.f : expf(logp);
    mass += pk;
    if (pk > 0.f) loss += pk * (logp - R::get(x, s_id[k]) * inv_t + lse);
    s_p[k] = pk;
  }
  mass = block_reduce(mass, s_red, false);
  if (p.loss) {
    loss = block_reduce(loss, s_red, false);
    if (tid == 0) {
      p.loss[row] = p.temperature * p.temperature * loss;
      p.lse[row] = lse;
    }
  }
  if (!p.grad) return;
  for (int k = tid; k < p.K; k += kThreads) {
    const int id = s_id[k];
    if (id < 0) continue;
    float sum = 0.f;
    for (int j = 0; j < p.K; ++j)
      if (s_id[j] == id) sum += s_p[j];
    s_fix[k] = g == 0.f ? 0.f : g * (mass * expf(R::get(x, id) * inv_t - lse) - sum);
  }
  __syncthreads();
  typename R::T *grad = static_cast<typename R::T *>(p.grad) + row * p.grad_stride;
  for (int v = tid; v < p.V; v += kThreads)
    R::put(grad, v, g == 0.f ? 0.f : g * mass * expf(R::get(x, v) * inv_t - lse));
  __syncthreads();
  for (int k = tid; k < p.K; k += kThreads)
    if (s_id[k] >= 0) R::put(grad, s_id[k], s_fix[k]);
}

}  // namespace

cudaError_t launch_distill(const DistillParams &p, bool f32, cudaStream_t st) {
  if (f32) k_distill<true><<<p.rows, kThreads, 0, st>>>(p);
  else k_distill<false><<<p.rows, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace dc
