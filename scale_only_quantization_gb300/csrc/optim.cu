// The optimizer's side of a step over lists of tensors: the global gradient norm, clipping, and AdamW.
//
//   norm = sqrt(sum g^2),   c = min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) c g,   v = b2 v + (1 - b2) (c g)^2
//   p = max(floor, p - lr decay p - lr m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps))
//
// All of it is bound by memory: 4 bytes an element for the norm, 8 more to clip, 28 for AdamW.  A list travels as a
// kernel parameter (up to 23 KB), so that nothing is copied to the device and a captured step holds its own list; the
// tensors are cut into chunks, and the blocks take chunks in turn.  The passes that follow the norm go through the
// chunks backwards: what the norm read last is still in L2.
//
// Norm and clipping of 302 M gradients 556 to 562 us (6.4 to 6.5 TB/s, both readings counted); norm and AdamW of 151 M scales 757 to
// 773 us (6.2 to 6.4 TB/s).  Of 50 thousand elements 12.3 and 16.4 us, bound by the launches.
#include "common.cuh"
#include "internal.h"

namespace qad {
namespace {

constexpr int kThreads = 256, kBlocksPerSm = 4;
constexpr int kMaxBlocks = 1024;           // partial sums in the workspace
constexpr size_t kCoef = 256;              // the coefficients of a step, behind the header
constexpr size_t kPartials = 512;

// One launch's tensors: P pointers each.
template <int P, int CAP>
struct Table {
  void* ptr[P][CAP];
  int64_t numel[CAP];
  int32_t first[CAP + 1];  // the tensor's first chunk
  uint8_t bf16[CAP];       // type of the gradients
  int n, index0;           // tensors here, and those of earlier launches
  int log_chunk;
};
constexpr int kSmall = 32, kLarge = 480;
// The norm of up to 64 chunks of 1024 elements in 32 tensors by one block: a small model's step waits for launches.  (A
// cluster of 8 blocks took 6.4 us for 50 thousand gradients, its launch and two barriers nearly all of it.)
constexpr int kFewThreads = 1024, kFewChunks = 64, kLogFew = 10;

struct Chunk {
  int tensor;
  int64_t at;
  int len;
};

template <class T>
__device__ __forceinline__ Chunk chunk_of(const T& t, int c) {
  int lo = 0, hi = t.n;  // the last tensor whose first chunk is not behind c (tensors without elements have none)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  Chunk k;
  k.tensor = lo;
  k.at = (int64_t)(c - t.first[lo]) << t.log_chunk;
  const int64_t left = t.numel[lo] - k.at;
  k.len = left < (int64_t(1) << t.log_chunk) ? (int)left : 1 << t.log_chunk;
  return k;
}

// The squares of N <= 16 values: in fp32 where none of them leaves its range (the largest in [2^-50, 2^50]), else in 64
// bits.
template <int N>
__device__ __forceinline__ double squares(const float* f) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  if (top == 0) return 0.0;
  if (top - 0x26800000u <= 0x58800000u - 0x26800000u) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(f[i], f[i], s);
    return (double)s;
  }
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) s += (double)f[i] * (double)f[i];
  return s;
}

// The block's sum, in its first thread.
template <int THREADS = kThreads>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[THREADS / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x / 32] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < THREADS / 32 ? s[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = THREADS / 64; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// fp32(sqrt(v)), in fp32 where v is in its range (64-bit square roots are slow here): off by one rounding more
__device__ __forceinline__ float root(double v) {
  return v > 1e-30 && v < 1e30 ? sqrtf((float)v) : (float)sqrt(v);
}

// A thread's part of a chunk's sum of squares: `lane` of `width` threads that share it, N values on
// their way at once.
template <int N, class T>
__device__ __forceinline__ double chunk_squares(const T& t, const Chunk& k, int lane, int width) {
  double sum = 0.0;
  float f[N];
  if (t.bf16[k.tensor]) {
    const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(t.ptr[0][k.tensor]) + k.at;
    const int whole = k.len / 8;
    for (int i = lane; i < whole; i += N / 8 * width) {
      uint4 v[N / 8];
#pragma unroll
      for (int j = 0; j < N / 8; ++j)
        v[j] = i + j * width < whole ? __ldg(reinterpret_cast<const uint4*>(g) + i + j * width) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < N / 8; ++j) unpack8(v[j], f + 8 * j);
#pragma unroll
      for (int j = 0; j < N; j += 16) sum += squares<16>(f + j);
    }
    for (int i = whole * 8 + lane; i < k.len; i += width) {
      const float one = __bfloat162float(g[i]);
      sum += squares<1>(&one);
    }
  } else {
    const float* g = static_cast<const float*>(t.ptr[0][k.tensor]) + k.at;
    const int whole = k.len / 4;
    for (int i = lane; i < whole; i += N / 4 * width) {
      float4 v[N / 4];
#pragma unroll
      for (int j = 0; j < N / 4; ++j)
        v[j] = i + j * width < whole ? __ldg(reinterpret_cast<const float4*>(g) + i + j * width)
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        f[4 * j] = v[j].x;
        f[4 * j + 1] = v[j].y;
        f[4 * j + 2] = v[j].z;
        f[4 * j + 3] = v[j].w;
      }
#pragma unroll
      for (int j = 0; j < N; j += 16) sum += squares<16>(f + j);
    }
    for (int i = whole * 4 + lane; i < k.len; i += width) sum += squares<1>(g + i);
  }
  return sum;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Table<1, CAP> t, double* part,
                                                             bool add) {
  double sum = 0.0;
  for (int c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) sum += chunk_squares<16>(t, chunk_of(t, c), threadIdx.x, kThreads);
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + sum : sum;
}

// One block, a chunk to a warp.
__global__ void __launch_bounds__(kFewThreads) grad_norm_few_kernel(const __grid_constant__ Table<1, kSmall> t,
                                                                    float* norm) {
  double sum = 0.0;
  for (int c = threadIdx.x / 32; c < t.first[t.n]; c += kFewThreads / 32)
    sum += chunk_squares<32>(t, chunk_of(t, c), threadIdx.x & 31, 32);
  sum = block_sum<kFewThreads>(sum);
  if (threadIdx.x == 0) norm[0] = root(sum);
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(const double* part, int n, float* norm) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v += part[i];
  v = block_sum(v);
  if (threadIdx.x == 0) norm[0] = root(v);
}

// min(1, max_norm / (norm + 1e-6)), and a NaN's NaN; 0 for an infinite norm, whatever max_norm
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  const float f = norm == INFINITY ? 0.0f : max_norm / (norm + 1e-6f);
  return f >= 1.0f ? 1.0f : f;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_clip_kernel(const __grid_constant__ Table<2, CAP> t, const float* norm,
                                                             float max_norm) {
  const float f = clip_factor(norm[0], max_norm);
  const int chunks = t.first[t.n];
  for (int b = blockIdx.x; b < chunks; b += gridDim.x) {
    const Chunk k = chunk_of(t, chunks - 1 - b);
    const void *in = t.ptr[0][k.tensor];
    void* out = t.ptr[1][k.tensor];
    if (f == 1.0f && in == out) continue;
    if (t.bf16[k.tensor]) {
      const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(in) + k.at;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + k.at;
      const int whole = k.len / 8;
      for (int i = threadIdx.x; i < whole; i += kThreads) {
        float v[8];
        unpack8(reinterpret_cast<const uint4*>(g)[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f;
        reinterpret_cast<uint4*>(o)[i] = pack8(v);
      }
      for (int i = whole * 8 + threadIdx.x; i < k.len; i += kThreads)
        o[i] = __float2bfloat16_rn(__bfloat162float(g[i]) * f);
    } else {
      const float* g = static_cast<const float*>(in) + k.at;
      float* o = static_cast<float*>(out) + k.at;
      const int whole = k.len / 4;
      for (int i = threadIdx.x; i < whole; i += 4 * kThreads) {
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j * kThreads < whole) v[j] = reinterpret_cast<const float4*>(g)[i + j * kThreads];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j * kThreads < whole)
            reinterpret_cast<float4*>(o)[i + j * kThreads] = make_float4(v[j].x * f, v[j].y * f, v[j].z * f, v[j].w * f);
      }
      for (int i = whole * 4 + threadIdx.x; i < k.len; i += kThreads) o[i] = g[i] * f;
    }
  }
}

struct Coef {
  float clip, inv_c1, inv_c2;  // the clip factor, 1 / (1 - b1^t), 1 / (1 - b2^t)
  int skip;                    // the norm is not finite, or the step count below 0 or at its end
};

// b^n by squaring (n <= 0: 1)
__device__ __forceinline__ double power(double b, int64_t n) {
  double v = 1.0;
  for (; n > 0; n >>= 1, b *= b)
    if (n & 1) v *= b;
  return v;
}

// One warp: lane 1 takes beta2's power beside lane 0's.
__global__ void adamw_coef_kernel(const float* norm, float max_norm, double beta1, double beta2, int64_t* steps,
                                  Coef* coef) {
  Coef c = {1.0f, 1.0f, 1.0f, 0};
  const int64_t t = (int64_t)((uint64_t)steps[0] + 1);
  c.skip = t < 1;
  if (norm) {
    c.skip |= !isfinite(norm[0]);
    c.clip = clip_factor(norm[0], max_norm);
  }
  const float inv = 1.0f / (float)(1.0 - power(threadIdx.x == 1 ? beta2 : beta1, t));
  c.inv_c1 = __shfl_sync(0xffffffffu, inv, 0);
  c.inv_c2 = __shfl_sync(0xffffffffu, inv, 1);
  if (threadIdx.x) return;
  if (!c.skip) steps[0] = t;
  *coef = c;
}

struct AdamwArgs {
  const float* lr;
  const Coef* coef;
  float beta1, rest1, beta2, rest2, eps, decay, floor;  // rest: 1 - beta, from 64 bits
};

struct Update {
  float clip, step, shrink, inv_c2;  // step = lr / (1 - b1^t), shrink = lr * decay
  __device__ __forceinline__ void operator()(const AdamwArgs& a, float& p, float g, float& m, float& v) const {
    g *= clip;
    m = fmaf(a.beta1, m, a.rest1 * g);
    v = fmaf(a.beta2, v, a.rest2 * g * g);
    const float x = p - shrink * p - step * m / (sqrtf(v * inv_c2) + a.eps);
    p = x < a.floor ? a.floor : x;  // a NaN stays
  }
};

template <int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<4, CAP> t, AdamwArgs a) {
  const Coef c = *a.coef;
  if (c.skip) return;
  const int chunks = t.first[t.n];
  for (int b = blockIdx.x; b < chunks; b += gridDim.x) {
    const Chunk k = chunk_of(t, chunks - 1 - b);
    float* p = static_cast<float*>(t.ptr[0][k.tensor]) + k.at;
    float* m = static_cast<float*>(t.ptr[2][k.tensor]) + k.at;
    float* v = static_cast<float*>(t.ptr[3][k.tensor]) + k.at;
    const float lr = a.lr[t.index0 + k.tensor];
    const Update up = {c.clip, lr * c.inv_c1, lr * a.decay, c.inv_c2};
    const bool bf16 = t.bf16[k.tensor];
    const float* g32 = static_cast<const float*>(t.ptr[1][k.tensor]) + (bf16 ? 0 : k.at);
    const __nv_bfloat16* g16 = static_cast<const __nv_bfloat16*>(t.ptr[1][k.tensor]) + (bf16 ? k.at : 0);
    const int whole = k.len / 4;
    for (int i = threadIdx.x; i < whole; i += 2 * kThreads) {
      float4 pv[2], gv[2], mv[2], vv[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = i + j * kThreads;
        if (at >= whole) break;
        pv[j] = reinterpret_cast<const float4*>(p)[at];
        mv[j] = reinterpret_cast<const float4*>(m)[at];
        vv[j] = reinterpret_cast<const float4*>(v)[at];
        if (bf16) {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(g16) + at);
          gv[j] = make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
        } else {
          gv[j] = __ldg(reinterpret_cast<const float4*>(g32) + at);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = i + j * kThreads;
        if (at >= whole) break;
        up(a, pv[j].x, gv[j].x, mv[j].x, vv[j].x);
        up(a, pv[j].y, gv[j].y, mv[j].y, vv[j].y);
        up(a, pv[j].z, gv[j].z, mv[j].z, vv[j].z);
        up(a, pv[j].w, gv[j].w, mv[j].w, vv[j].w);
        reinterpret_cast<float4*>(p)[at] = pv[j];
        reinterpret_cast<float4*>(m)[at] = mv[j];
        reinterpret_cast<float4*>(v)[at] = vv[j];
      }
    }
    for (int i = whole * 4 + threadIdx.x; i < k.len; i += kThreads)
      up(a, p[i], bf16 ? __bfloat162float(g16[i]) : g32[i], m[i], v[i]);
  }
}

int max_blocks() {
  const int n = num_sms() * kBlocksPerSm;
  return n < kMaxBlocks ? n : kMaxBlocks;
}

// Chunks of 2^10 to 2^14 elements: the largest that still give every block one.
int log_chunk_of(const qad_tensor* list, int64_t n, int blocks) {
  for (int lc = 14; lc > 10; --lc) {
    int64_t chunks = 0;
    for (int64_t i = 0; i < n && chunks < blocks; ++i) chunks += list[i].numel >> lc;
    if (chunks >= blocks) return lc;
  }
  return 10;
}

// Tables of up to CAP tensors, one after another (from `at`): fills `t` and returns the next tensor.
template <int P, int CAP>
int64_t fill(Table<P, CAP>* t, const qad_tensor* const* lists, int bf16_of, int64_t at, int64_t n, int log_chunk) {
  t->n = 0;
  t->index0 = (int)at;
  t->log_chunk = log_chunk;
  t->first[0] = 0;
  for (; at < n && t->n < CAP; ++at) {
    const int64_t numel = lists[0][at].numel;
    const int64_t end = t->first[t->n] + ((numel + (int64_t(1) << log_chunk) - 1) >> log_chunk);
    if (end > 0x7fffffff) break;
    for (int i = 0; i < P; ++i) t->ptr[i][t->n] = lists[i][at].data;
    t->numel[t->n] = numel;
    t->bf16[t->n] = lists[bf16_of][at].dtype == QAD_BF16;
    t->first[++t->n] = (int32_t)end;
  }
  return at;
}

// Calls f(table, blocks, first) for the tables of a list; f launches and returns the error.
template <int P, class F>
cudaError_t for_tables(const qad_tensor* const* lists, int bf16_of, int64_t n, F&& f) {
  const int blocks = max_blocks(), lc = log_chunk_of(lists[0], n, blocks);
  bool first = true;
  for (int64_t at = 0; at < n || first;) {
    cudaError_t e;
    if (n <= kSmall) {
      Table<P, kSmall> t;
      at = fill(&t, lists, bf16_of, at, n, lc);
      e = f(t, blocks < t.first[t.n] ? blocks : t.first[t.n], first);
    } else {
      Table<P, kLarge> t;
      at = fill(&t, lists, bf16_of, at, n, lc);
      e = f(t, blocks < t.first[t.n] ? blocks : t.first[t.n], first);
    }
    if (e != cudaSuccess) return e;
    first = false;
  }
  return cudaSuccess;
}

}  // namespace

size_t optim_workspace() { return kPartials + sizeof(double) * kMaxBlocks; }

cudaError_t launch_grad_norm(const qad_tensor* grads, int64_t n, float* norm, uint8_t* ws, cudaStream_t st) {
  double* part = reinterpret_cast<double*>(ws + kPartials);
  const qad_tensor* lists[1] = {grads};
  int parts = 0;
  prof_begin(QAD_K_GRAD_NORM, st);
  int64_t chunks = 0;
  for (int64_t i = 0; i < n && n <= kSmall; ++i) chunks += (grads[i].numel + (1 << kLogFew) - 1) >> kLogFew;
  if (n <= kSmall && chunks <= kFewChunks) {
    Table<1, kSmall> t;
    fill(&t, lists, 0, 0, n, kLogFew);
    grad_norm_few_kernel<<<1, kFewThreads, 0, st>>>(t, norm);
    prof_end(QAD_K_GRAD_NORM, st);
    return cudaGetLastError();
  }
  // every launch but the first adds to the partial sums of the first one's blocks: where others follow it has as many as
  // any of them may want (those without a chunk write a 0)
  cudaError_t e = for_tables<1>(lists, 0, n, [&](const auto& t, int blocks, bool) {
    if (blocks == 0) return cudaSuccess;
    constexpr int CAP = sizeof(t.bf16);
    if (!parts && n > CAP) blocks = max_blocks();
    grad_norm_kernel<CAP><<<blocks, kThreads, 0, st>>>(t, part, parts > 0);
    if (parts) note_launches(1);
    else parts = blocks;
    return cudaGetLastError();
  });
  if (e == cudaSuccess) {
    note_launches(1);
    grad_norm_join_kernel<<<1, kThreads, 0, st>>>(part, parts, norm);
    e = cudaGetLastError();
  }
  prof_end(QAD_K_GRAD_NORM, st);
  return e;
}

cudaError_t launch_grad_clip(const qad_tensor* grads, const qad_tensor* out, int64_t n, const float* norm,
                             float max_norm, cudaStream_t st) {
  const qad_tensor* lists[2] = {grads, out};
  prof_begin(QAD_K_GRAD_CLIP, st);
  const cudaError_t e = for_tables<2>(lists, 0, n, [&](const auto& t, int blocks, bool first) {
    if (blocks == 0) return cudaSuccess;
    constexpr int CAP = sizeof(t.bf16);
    grad_clip_kernel<CAP><<<blocks, kThreads, 0, st>>>(t, norm, max_norm);
    if (!first) note_launches(1);
    return cudaGetLastError();
  });
  prof_end(QAD_K_GRAD_CLIP, st);
  return e;
}

cudaError_t launch_adamw(const qad_tensor* params, const qad_tensor* grads, const qad_tensor* m, const qad_tensor* v,
                         int64_t n, const float* lr, double beta1, double beta2, float eps, float decay, float floor,
                         const float* norm, float max_norm, int64_t* steps, uint8_t* ws, cudaStream_t st) {
  const qad_tensor* lists[4] = {params, grads, m, v};
  AdamwArgs a;
  a.lr = lr;
  a.coef = reinterpret_cast<const Coef*>(ws + kCoef);
  a.beta1 = (float)beta1;
  a.rest1 = (float)(1.0 - beta1);
  a.beta2 = (float)beta2;
  a.rest2 = (float)(1.0 - beta2);
  a.eps = eps;
  a.decay = decay;
  a.floor = floor;
  prof_begin(QAD_K_ADAMW, st);
  adamw_coef_kernel<<<1, 32, 0, st>>>(norm, max_norm, beta1, beta2, steps, reinterpret_cast<Coef*>(ws + kCoef));
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = for_tables<4>(lists, 1, n, [&](const auto& t, int blocks, bool) {
      if (blocks == 0) return cudaSuccess;
      constexpr int CAP = sizeof(t.bf16);
      adamw_kernel<CAP><<<blocks, kThreads, 0, st>>>(t, a);
      note_launches(1);
      return cudaGetLastError();
    });
  prof_end(QAD_K_ADAMW, st);
  return e;
}

}  // namespace qad
