// Distillation from the teacher's top K logits, restricted to the teacher's own tokens ("MCoreQAD
// Backend": top-k distillation computes the divergence only on the teacher's top-k tokens, so
// [tokens, vocab] is never materialised; types kl, rkl and a mix of both).
//
// Row i, slot k with token v = idx[i, k], beta = 1 / temperature:
//   z_k = <h_i, w_v>                      the student's logit, from its hidden state and the head row
//   p = softmax_k(beta t_k), q = softmax_k(beta z_k)   over the row's kept slots
//   x_k = log q_k - log p_k
//   KL = sum p (log p - log q) = sum p f(x),  RKL = sum q (log q - log p) = sum q f(-x),
//        f(x) = e^x - 1 - x >= 0, so that near-equal distributions do not cancel
//   loss = (1 - m) KL + m RKL
//   dz_k = beta ((1 - m) (q - p) + m q (x - RKL)),  dh_i = g_i sum_k dz_k w_v
// Slots with idx < 0 or t = -inf do not count; a row that keeps no slot has loss 0 and no gradient.
#include "common.cuh"
#include "internal.h"

namespace qad {
namespace {

constexpr int kThreadsD = 256;

struct Distill {
  const __nv_bfloat16 *h, *w;
  const int32_t* idx;
  const float *t, *mix, *g;
  float* loss;
  __nv_bfloat16* dh;
  int32_t* err;
  int64_t ldh, ldw, V;
  float beta;
  int K, d, accumulate;
};

// p f(x), with q = p e^x: a Taylor sum where e^x - 1 - x would cancel (|x| < 1/2: the first
// omitted term is below 2^-29 of the sum), the difference of the two probabilities elsewhere.
__device__ __forceinline__ float div_term(float p, float q, float x) {
  if (fabsf(x) < 0.5f) {
    float s = 1.0f / 362880.0f;
    s = fmaf(s, x, 1.0f / 40320.0f);
    s = fmaf(s, x, 1.0f / 5040.0f);
    s = fmaf(s, x, 1.0f / 720.0f);
    s = fmaf(s, x, 1.0f / 120.0f);
    s = fmaf(s, x, 1.0f / 24.0f);
    s = fmaf(s, x, 1.0f / 6.0f);
    s = fmaf(s, x, 0.5f);
    return p * x * x * s;
  }
  return q - p - p * x;
}

// The divergence of one row from its student logits z[K] in shared memory (one warp); leaves
// g * dz in z when grad, and returns the loss to every lane.
__device__ __forceinline__ float row_divergence(const Distill& p, int64_t row, float* z, const float* ts, int lane,
                                                bool grad) {
  // ts[k] = beta * teacher logit, or -inf for a slot that does not count
  float mz = -INFINITY, mt = -INFINITY;
  for (int k = lane; k < p.K; k += 32) {
    mt = fmaxf(mt, ts[k]);
    if (ts[k] != -INFINITY) mz = fmaxf(mz, z[k]);
  }
  mz = warp_max(mz);
  mt = warp_max(mt);
  float sz = 0.0f, st = 0.0f;
  for (int k = lane; k < p.K; k += 32)
    if (ts[k] != -INFINITY) {
      sz += expf(z[k] - mz);
      st += expf(ts[k] - mt);
    }
  sz = warp_sum(sz);
  st = warp_sum(st);
  const float lz = logf(sz), lt = logf(st), rz = 1.0f / sz, rt = 1.0f / st;
  float kl = 0.0f, rkl = 0.0f;
  for (int k = lane; k < p.K; k += 32)
    if (ts[k] != -INFINITY) {
      const float x = ((z[k] - mz) - lz) - ((ts[k] - mt) - lt);
      const float pk = expf(ts[k] - mt) * rt, qk = expf(z[k] - mz) * rz;
      kl += div_term(pk, qk, x);
      rkl += div_term(qk, pk, -x);
    }
  kl = warp_sum(kl);
  rkl = warp_sum(rkl);
  const float m = p.mix ? p.mix[row] : 0.0f;
  if (grad) {
    const float scale = p.beta * (p.g ? p.g[row] : 1.0f);
    for (int k = lane; k < p.K; k += 32) {
      float dz = 0.0f;
      if (ts[k] != -INFINITY) {
        const float x = ((z[k] - mz) - lz) - ((ts[k] - mt) - lt);
        const float pk = expf(ts[k] - mt) * rt, qk = expf(z[k] - mz) * rz;
        dz = (1.0f - m) * (qk - pk) + m * qk * (x - rkl);
      }
      z[k] = dz * scale;
    }
  }
  return (1.0f - m) * kl + m * rkl;
}

// One block per row: the hidden state in shared memory, one warp per head row for the logits, one
// thread per 8 columns for the gradient.
template <bool GRAD>
__global__ void __launch_bounds__(kThreadsD) distill_row_kernel(const Distill p) {
  extern __shared__ __align__(16) uint8_t sm[];
  uint4* hs = reinterpret_cast<uint4*>(sm);
  const int nv = p.d / 8;
  float* z = reinterpret_cast<float*>(hs + nv);
  float* ts = z + p.K;
  int32_t* tok = reinterpret_cast<int32_t*>(ts + p.K);
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int any;
  if (threadIdx.x == 0) any = 0;
  const uint4* hr = reinterpret_cast<const uint4*>(p.h + row * p.ldh);
  for (int c = threadIdx.x; c < nv; c += kThreadsD) hs[c] = __ldg(hr + c);
  __syncthreads();
  for (int k = threadIdx.x; k < p.K; k += kThreadsD) {
    int32_t v = p.idx[row * p.K + k];
    float t = p.t[row * p.K + k] * p.beta;
    if (v >= p.V) {
      if (p.err) atomicOr(p.err, QAD_DEV_BAD_INDEX);
      v = -1;
    }
    if (t == -INFINITY) v = -1;
    if (v < 0) t = -INFINITY;
    tok[k] = v;
    ts[k] = t;
    z[k] = 0.0f;
    if (v >= 0) any = 1;
  }
  __syncthreads();
  if (any)
    for (int k = warp; k < p.K; k += kThreadsD / 32) {
      const int32_t v = tok[k];
      if (v < 0) continue;
      const uint4* wr = reinterpret_cast<const uint4*>(p.w + (int64_t)v * p.ldw);
      float acc = 0.0f;
      for (int c = lane; c < nv; c += 32) {
        float a[8], b[8];
        unpack8(hs[c], a);
        unpack8(__ldg(wr + c), b);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc = fmaf(a[j], b[j], acc);
      }
      acc = warp_sum(acc);
      if (lane == 0) z[k] = acc * p.beta;
    }
  __syncthreads();
  if (warp == 0) {
    const float l = any ? row_divergence(p, row, z, ts, lane, GRAD) : 0.0f;
    if (lane == 0) p.loss[row] = l;
  }
  if constexpr (GRAD) {
    __syncthreads();
    for (int c = threadIdx.x; c < nv; c += kThreadsD) {
      float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      uint4* out = reinterpret_cast<uint4*>(p.dh + row * p.d) + c;
      for (int k = 0; k < p.K; ++k) {
        const int32_t v = tok[k];
        if (v < 0) continue;
        float b[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(p.w + (int64_t)v * p.ldw) + c), b);
        const float dz = z[k];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(dz, b[j], acc[j]);
      }
      if (p.accumulate) {
        float b[8];
        unpack8(*out, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += b[j];
      }
      *out = pack8(acc);
    }
  }
}

}  // namespace

cudaError_t launch_distill_topk(const void* h, int64_t ldh, const void* w, int64_t ldw, const int32_t* idx,
                                const float* t, const float* mix, float inv_temp, const float* g, float* loss, void* dh,
                                int accumulate, int64_t N, int64_t d, int64_t V, int64_t K, int32_t* err,
                                cudaStream_t st) {
  Distill p = {};
  p.h = static_cast<const __nv_bfloat16*>(h);
  p.w = static_cast<const __nv_bfloat16*>(w);
  p.idx = idx;
  p.t = t;
  p.mix = mix;
  p.g = g;
  p.loss = loss;
  p.dh = static_cast<__nv_bfloat16*>(dh);
  p.err = err;
  p.ldh = ldh;
  p.ldw = ldw;
  p.V = V;
  p.beta = inv_temp;
  p.K = (int)K;
  p.d = (int)d;
  p.accumulate = accumulate;
  const size_t smem = (size_t)d * 2 + (size_t)K * 12;
  prof_begin(QAD_K_DISTILL, st);
  if (dh) distill_row_kernel<true><<<(unsigned)N, kThreadsD, smem, st>>>(p);
  else distill_row_kernel<false><<<(unsigned)N, kThreadsD, smem, st>>>(p);
  prof_end(QAD_K_DISTILL, st);
  return cudaGetLastError();
}

}  // namespace qad
