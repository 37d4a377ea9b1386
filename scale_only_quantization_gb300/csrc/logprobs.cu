// Log probabilities of given tokens, entropy and top alternatives of logits in one reading of them, and the gradient
// with respect to the logits.
//
//   y_v = (z_v - m) b log2(e),  S = sum 2^y,  U = sum 2^y y      m: the running maximum, per thread
//   lse = b m + ln S,   H = ln S - ln2 U / S,   logp = b (z_t - m) - ln S
//   dz = b (g (1[v = t] - p) - h p (log p + H)),   p = exp(b z - lse)
//
// Each thread keeps m, S and U of the logits it has seen (a new maximum rescales S and U); the block joins them at the
// end.  The alternatives: a logit enters the block's candidates when it is above a threshold that at least K logits
// reach.  The threshold is the K-th largest of the threads' maxima, found by bisection on the bits with block-wide
// counts; with K well below the number of threads few more than K logits reach it, so that a row of 151936 leaves some
// hundred candidates, which are sorted once.  Candidates are ordered by (value, index) as one 64-bit key: equal logits
// stand by rising index.  Rows are split over the blocks of a cluster when there are too few to fill the GPU; the
// cluster's first block joins the others' sums and candidates out of their shared memory.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace qad {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kPer = 16;                  // logits of a thread per step
constexpr int kStep = kThreads * kPer;    // of a block
constexpr int kCap = 2048;                // candidates of a block
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// max(v, lo) that keeps a NaN
__device__ __forceinline__ float floor_nan(float v, float lo) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(lo));
  return r;
}

// A number whose order as an unsigned integer is the float's order (-0 as +0); 0 for a NaN, which is below -inf's.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v != v ? 0u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

struct Logprobs {
  const void* z;
  const int32_t* token;
  float *logp, *lse, *entropy, *top_logit;
  int32_t *top_idx, *err;
  int64_t ldz;
  int V, K;
  float b;
};

// The 16 logits of a thread in one step: vectors of 16 bytes, kThreads apart.  `at` counts elements from the 16-byte
// boundary at or before the range; what lies outside [from, to) counts as -inf and is not read past `to`.
template <typename ZT>
struct Step {
  static constexpr int kVec = 16 / sizeof(ZT), kVecs = kPer / kVec;
  uint4 raw[kVecs];

  __device__ __forceinline__ static int place(int step, int i) { return (step * kVecs * kThreads + i * kThreads + (int)threadIdx.x) * kVec; }

  __device__ __forceinline__ void load(const ZT* base, int step, int to) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = place(step, i);
      if (at + kVec <= to) {
        raw[i] = __ldg(reinterpret_cast<const uint4*>(base + at));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(ZT) == 4) {
            w[j] = at + j < to ? __float_as_uint(__ldg(reinterpret_cast<const float*>(base) + at + j)) : 0xff800000u;
          } else {
            const unsigned short* h = reinterpret_cast<const unsigned short*>(base) + at + 2 * j;
            const uint32_t a = at + 2 * j < to ? __ldg(h) : 0xff80u, b = at + 2 * j + 1 < to ? __ldg(h + 1) : 0xff80u;
            w[j] = a | (b << 16);
          }
        }
        raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  __device__ __forceinline__ void unpack(float* f, int step, int from) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if constexpr (sizeof(ZT) == 4) {
        f[4 * i] = __uint_as_float(raw[i].x);
        f[4 * i + 1] = __uint_as_float(raw[i].y);
        f[4 * i + 2] = __uint_as_float(raw[i].z);
        f[4 * i + 3] = __uint_as_float(raw[i].w);
      } else {
        unpack8(raw[i], f + 8 * i);
      }
      if (step == 0 && i == 0 && threadIdx.x == 0) {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (j < from) f[j] = -INFINITY;
      }
    }
  }
  // the element's place of f[j]
  __device__ __forceinline__ static int at_of(int step, int j) { return place(step, j / kVec) + j % kVec; }
};

// Sorts s_key[0, n2) in falling order, n2 a power of two.
__device__ __forceinline__ void sort_keys(uint64_t* s_key, int n2) {
  for (int size = 2; size <= n2; size *= 2) {
    for (int half = size / 2; half; half /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < n2 / 2; i += kThreads) {
        const int a = 2 * half * (i / half) + i % half, b = a + half;
        const uint64_t x = s_key[a], y = s_key[b];
        if ((x < y) == ((a & size) == 0)) {
          s_key[a] = y;
          s_key[b] = x;
        }
      }
    }
  }
  __syncthreads();
}

// Orders the candidates and keeps the K best; returns how many are left.
__device__ __forceinline__ int keep_best(uint64_t* s_key, int n, int K) {
  int n2 = 32;
  while (n2 < n) n2 *= 2;
  __syncthreads();
  for (int i = n + threadIdx.x; i < n2; i += kThreads) s_key[i] = 0;
  sort_keys(s_key, n2);
  return min(n, K);
}

// The largest t (in its upper bits) that at least K of the block's values reach.
__device__ __forceinline__ uint32_t reached_by(uint32_t mine, int K, int bits) {
  uint32_t t = 0;
  for (int b = 31; b >= 32 - bits; --b) {
    const uint32_t trial = t | (1u << b);
    if (__syncthreads_count(mine >= trial) >= K) t = trial;
  }
  return t;
}

template <typename ZT, bool TOP, bool ENT>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(Logprobs q, int parts) {
  using St = Step<ZT>;
  __shared__ uint64_t s_key[TOP ? kCap : 1];
  __shared__ int s_n;
  __shared__ float s_m[kWarps], s_s[kWarps], s_u[kWarps];
  __shared__ float s_sum[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int64_t row = blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  const ZT* zrow = static_cast<const ZT*>(q.z) + row * q.ldz;
  const int share = ((q.V + parts - 1) / parts + 63) / 64 * 64;
  const int lo = min(q.V, part * share), len = min(q.V - lo, share);
  const int from = (int)((reinterpret_cast<uintptr_t>(zrow + lo) & 15u) / sizeof(ZT));
  const ZT* base = zrow + lo - from;
  const int to = from + len;
  const int steps = (to + kStep - 1) / kStep;
  const float b2 = q.b * kLog2e;
  float m = -INFINITY, S = 0.0f, U = 0.0f;
  uint64_t above = 0;  // a candidate's key is larger
  if (TOP && tid == 0) s_n = 0;

  St now, next;
  if (steps > 0) now.load(base, 0, to);
  for (int step = 0; step < steps; ++step) {
    if (step + 1 < steps) next.load(base, step + 1, to);
    float f[kPer];
    now.unpack(f, step, from);
    float top = f[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) top = fmaxf(top, f[i]);
    if (top > m) {
      if (m > -INFINITY) {
        const float d = (m - top) * b2, c = ex2(d);
        if constexpr (ENT) U = c == 0.0f ? 0.0f : c * fmaf(S, d, U);
        S *= c;
      }
      m = top;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    const uint64_t nref = f2pack(-ref, -ref), bb = f2pack(b2, b2);
    uint64_t s2 = f2pack(0.0f, 0.0f), u2 = s2;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const float2 y = f2unpack(f2mul(f2add(f2pack(f[i], f[i + 1]), nref), bb));
      const float y0 = floor_nan(y.x, -200.0f), y1 = floor_nan(y.y, -200.0f);  // 2^-200 is 0 in fp32
      const uint64_t e2 = f2pack(ex2(y0), ex2(y1));
      s2 = f2add(s2, e2);
      if constexpr (ENT) u2 = f2fma(e2, f2pack(y0, y1), u2);
    }
    S += f2unpack(s2).x + f2unpack(s2).y;
    if constexpr (ENT) U += f2unpack(u2).x + f2unpack(u2).y;

    if constexpr (TOP) {
      const uint32_t mine = order_of(top);
      int passing = __syncthreads_count(mine >= (uint32_t)(above >> 32));
      if (passing) {
        // a higher threshold from the maxima so far: at the first steps, and when the candidates would not fit
        if (q.K <= kThreads && ((step & (step + 1)) == 0 || passing * kPer + s_n > kCap)) {
          const uint32_t t = reached_by(order_of(m), q.K, sizeof(ZT) == 2 ? 16 : 22);
          const uint64_t up = t ? ((uint64_t)t << 32) - 1 : 0;
          if (up > above) {
            above = up;
            passing = __syncthreads_count(mine >= (uint32_t)(above >> 32));
          }
        }
        const bool fits = passing * kPer + s_n <= kCap;
        __syncthreads();  // everybody has read s_n
        if (fits) {
          if (mine >= (uint32_t)(above >> 32)) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              const int at = St::at_of(step, j);
              const uint64_t key = ((uint64_t)order_of(f[j]) << 32) | (0xffffffffu - (uint32_t)(lo + at - from));
              if (key > above && f[j] == f[j] && at >= from && at < to) s_key[atomicAdd(&s_n, 1)] = key;
            }
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < kPer; ++j) {
            const int held = s_n;
            __syncthreads();  // read by everybody before anybody adds
            if (held > kCap - kThreads) {
              const int n = keep_best(s_key, held, q.K);
              if (n == q.K && s_key[n - 1] > above) above = s_key[n - 1];
              __syncthreads();
              if (tid == 0) s_n = n;
              __syncthreads();
            }
            float v = f[0];
#pragma unroll
            for (int i = 1; i < kPer; ++i) v = i == j ? f[i] : v;
            const int at = St::at_of(step, j);
            const uint64_t key = ((uint64_t)order_of(v) << 32) | (0xffffffffu - (uint32_t)(lo + at - from));
            if (key > above && v == v && at >= from && at < to) s_key[atomicAdd(&s_n, 1)] = key;
            __syncthreads();
          }
        }
      }
    }
    now = next;
  }

  // the block's sums
  {
    const float wm = warp_max(m);
    const float c = m == -INFINITY ? 0.0f : ex2((m - wm) * b2);
    if constexpr (ENT) U = c == 0.0f ? 0.0f : c * fmaf(S, (m - wm) * b2, U);
    // a NaN stays one: where nothing but NaN and -inf was seen m is -inf, and S says which
    S = m == -INFINITY ? S : S * c;
    S = warp_sum(S);
    if constexpr (ENT) U = warp_sum(U);
    if (lane == 0) {
      s_m[warp] = wm;
      s_s[warp] = S;
      s_u[warp] = U;
    }
  }
  int n = 0;
  if constexpr (TOP) {
    __syncthreads();
    n = keep_best(s_key, s_n, q.K);
  } else {
    __syncthreads();
  }
  if (tid == 0) {
    float M = s_m[0];
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    float s = 0.0f, u = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      const float d = s_m[w] == -INFINITY ? 0.0f : (s_m[w] - M) * b2, c = ex2(d);
      s = fmaf(s_s[w], c, s);
      if (ENT && c > 0.0f) u = fmaf(c, fmaf(s_s[w], d, s_u[w]), u);
    }
    s_sum[0] = M;
    s_sum[1] = s;
    s_sum[2] = u;
    s_n = n;
  }
  if (parts > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (part == 0) {
      if (tid == 0) {
        float M = s_sum[0];
        for (int r = 1; r < parts; ++r) M = fmaxf(M, cluster.map_shared_rank(s_sum, r)[0]);
        float s = 0.0f, u = 0.0f;
        for (int r = 0; r < parts; ++r) {
          const float* o = cluster.map_shared_rank(s_sum, r);
          const float d = o[0] == -INFINITY ? 0.0f : (o[0] - M) * b2, c = ex2(d);
          s = fmaf(o[1], c, s);
          if (ENT && c > 0.0f) u = fmaf(c, fmaf(o[1], d, o[2]), u);
        }
        s_m[0] = M;
        s_s[0] = s;
        s_u[0] = u;
      }
      if constexpr (TOP) {
        for (int r = 1; r < parts; ++r) {
          const int more = *cluster.map_shared_rank(&s_n, r);
          const uint64_t* keys = cluster.map_shared_rank(s_key, r);
          for (int i = tid; i < more; i += kThreads) s_key[n + i] = keys[i];
          n += more;
        }
        n = keep_best(s_key, n, q.K);
      }
    }
    cluster.sync();  // the others' shared memory has been read
    if (part) return;
    __syncthreads();
    if (tid == 0) {
      s_sum[0] = s_m[0];
      s_sum[1] = s_s[0];
      s_sum[2] = s_u[0];
    }
  }
  if (tid == 0) {
    const float M = s_sum[0], s = s_sum[1];
    const bool empty = M == -INFINITY && s == 0.0f;
    const float ls = logf(s);
    if (q.lse) q.lse[row] = empty ? -INFINITY : M == -INFINITY ? s + NAN : fmaf(M, q.b, ls);
    if (ENT) q.entropy[row] = empty ? 0.0f : M == -INFINITY ? NAN : fmaxf(ls - kLn2 * s_sum[2] / s, 0.0f) + 0.0f * s;
    if (q.logp) {
      const int t = q.token[row];
      float lp = 0.0f;
      if (t >= q.V) {
        if (q.err) atomicOr(q.err, QAD_DEV_BAD_INDEX);
      } else if (t >= 0) {
        const ZT* at = zrow + t;
        float zt;
        if constexpr (sizeof(ZT) == 4) zt = *reinterpret_cast<const float*>(at);
        else zt = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at));
        lp = empty ? -INFINITY : M == -INFINITY ? NAN : (zt - M) * q.b - ls;
      }
      q.logp[row] = lp;
    } else if (q.token && q.err && q.token[row] >= q.V) {
      atomicOr(q.err, QAD_DEV_BAD_INDEX);
    }
  }
  if constexpr (TOP) {
    for (int i = tid; i < q.K; i += kThreads) {
      const uint64_t key = i < n ? s_key[i] : 0;
      if (q.top_idx) q.top_idx[row * q.K + i] = i < n ? (int32_t)(0xffffffffu - (uint32_t)key) : -1;
      if (q.top_logit) q.top_logit[row * q.K + i] = i < n ? value_of((uint32_t)(key >> 32)) : -INFINITY;
    }
  }
}

template <typename ZT, bool TOP, bool ENT>
cudaError_t launch(const Logprobs& q, int64_t N, cudaStream_t st) {
  // as many blocks for a row as fill the GPU twice, while each has a whole step and their candidates fit one block's list
  int parts = 1;
  while (parts < 8 && 2 * parts * N <= 2 * (int64_t)num_sms() && q.V / (2 * parts) >= kStep / 4 &&
         (!TOP || 2 * parts * q.K <= kCap))
    parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(N * parts), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = (unsigned)parts;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<ZT, TOP, ENT>, q, parts);
}

template <typename ZT>
cudaError_t launch_type(const Logprobs& q, int64_t N, cudaStream_t st) {
  if (q.K) return q.entropy ? launch<ZT, true, true>(q, N, st) : launch<ZT, true, false>(q, N, st);
  return q.entropy ? launch<ZT, false, true>(q, N, st) : launch<ZT, false, false>(q, N, st);
}

// ------------------------------------------------------------------------------------------------ gradient

constexpr int kBwdThreads = 256, kBwdVecs = 4;  // 16-byte vectors of a thread

struct LogprobsBwd {
  const void* z;
  void* dz;
  const int32_t* token;
  const float *lse, *entropy, *g_logp, *g_entropy;
  int64_t ldz, lddz, segments;  // segments of a row
  int V;
  float b;
};

template <typename ZT>
__device__ __forceinline__ float read_one(const ZT* p) {
  if constexpr (sizeof(ZT) == 4) return *reinterpret_cast<const float*>(p);
  else return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}
template <typename ZT>
__device__ __forceinline__ void write_one(ZT* p, float v) {
  if constexpr (sizeof(ZT) == 4) *reinterpret_cast<float*>(p) = v;
  else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v);
}

// A block takes a segment of one row.  ALIKE: the rows of z and dz lie alike relative to 16 bytes, so whole vectors of
// both; the row's first and last vector, and all of them otherwise, go element by element on z's side.
template <typename ZT, bool ALIKE>
__global__ void __launch_bounds__(kBwdThreads) logprobs_bwd_kernel(LogprobsBwd q) {
  constexpr int kVec = 16 / sizeof(ZT);
  const int64_t row = blockIdx.x / q.segments, seg = blockIdx.x % q.segments;
  const ZT* z = static_cast<const ZT*>(q.z) + row * q.ldz;
  ZT* dz = static_cast<ZT*>(q.dz) + row * q.lddz;
  const float lse = q.lse[row];
  const int token = q.token ? q.token[row] : -1;
  const bool live = token >= 0 && token < q.V;
  const float g = q.g_logp && live ? q.g_logp[row] : 0.0f;
  const float h = q.g_entropy ? q.g_entropy[row] : 0.0f, H = q.g_entropy ? q.entropy[row] : 0.0f;
  const bool empty = lse == -INFINITY;
  const float nlse = -lse, scale = -q.b;
  const int from = (int)((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(ZT));
  auto grad = [&](float zv, int v) {
    const float lp = floor_nan(fmaf(zv, q.b, nlse), -1e4f);
    const float p = ex2(lp * kLog2e);
    float d = scale * p * fmaf(h, lp + H, g);
    if (v == token) d += q.b * g;
    return empty ? 0.0f : d;
  };
#pragma unroll
  for (int i = 0; i < kBwdVecs; ++i) {
    const int v0 = (int)((seg * kBwdVecs + i) * kBwdThreads + threadIdx.x) * kVec - from;
    if (v0 >= q.V) break;
    if (v0 >= 0 && v0 + kVec <= q.V) {
      float f[kVec];
      if constexpr (ALIKE) {
        const uint4 u = *reinterpret_cast<const uint4*>(z + v0);
        if constexpr (sizeof(ZT) == 4) {
          f[0] = __uint_as_float(u.x);
          f[1] = __uint_as_float(u.y);
          f[2] = __uint_as_float(u.z);
          f[3] = __uint_as_float(u.w);
        } else {
          unpack8(u, f);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] = read_one(z + v0 + j);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) f[j] = grad(f[j], v0 + j);
      uint4 o;
      if constexpr (sizeof(ZT) == 4)
        o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      else
        o = pack8(f);
      *reinterpret_cast<uint4*>(dz + v0) = o;
    } else {
      for (int j = 0; j < kVec; ++j)
        if (v0 + j >= 0 && v0 + j < q.V) write_one(dz + v0 + j, grad(read_one(z + v0 + j), v0 + j));
    }
  }
}

template <typename ZT>
cudaError_t launch_bwd(LogprobsBwd q, int64_t N, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(ZT), kSegment = kBwdThreads * kBwdVecs * kVec;
  q.segments = (q.V + kVec - 1 + kSegment - 1) / kSegment;
  const int64_t blocks = N * q.segments;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const bool alike = ((reinterpret_cast<uintptr_t>(q.z) ^ reinterpret_cast<uintptr_t>(q.dz)) & 15u) == 0 &&
                     (N == 1 || (q.ldz - q.lddz) % kVec == 0);
  if (alike) logprobs_bwd_kernel<ZT, true><<<(unsigned)blocks, kBwdThreads, 0, st>>>(q);
  else logprobs_bwd_kernel<ZT, false><<<(unsigned)blocks, kBwdThreads, 0, st>>>(q);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs(const void* z, int dtype, int64_t ldz, const int32_t* token, float inv_temp, float* logp,
                            float* lse, float* entropy, int32_t* top_idx, float* top_logit, int64_t N, int64_t V,
                            int64_t K, int32_t* err, cudaStream_t st) {
  Logprobs q = {};
  q.z = z;
  q.token = token;
  q.logp = logp;
  q.lse = lse;
  q.entropy = entropy;
  q.top_idx = top_idx;
  q.top_logit = top_logit;
  q.err = err;
  q.ldz = ldz;
  q.V = (int)V;
  q.K = (int)K;
  q.b = inv_temp;
  prof_begin(QAD_K_LOGPROBS, st);
  const cudaError_t e =
      dtype == QAD_F32 ? launch_type<float>(q, N, st) : launch_type<__nv_bfloat16>(q, N, st);
  prof_end(QAD_K_LOGPROBS, st);
  return e;
}

cudaError_t launch_logprobs_bwd(const void* z, int dtype, int64_t ldz, const int32_t* token, float inv_temp,
                                const float* lse, const float* entropy, const float* g_logp, const float* g_entropy,
                                void* dz, int64_t lddz, int64_t N, int64_t V, cudaStream_t st) {
  LogprobsBwd q = {};
  q.z = z;
  q.dz = dz;
  q.token = token;
  q.lse = lse;
  q.entropy = entropy;
  q.g_logp = g_logp;
  q.g_entropy = g_entropy;
  q.ldz = ldz;
  q.lddz = lddz;
  q.V = (int)V;
  q.b = inv_temp;
  prof_begin(QAD_K_LOGPROBS_BWD, st);
  const cudaError_t e = dtype == QAD_F32 ? launch_bwd<float>(q, N, st) : launch_bwd<__nv_bfloat16>(q, N, st);
  prof_end(QAD_K_LOGPROBS_BWD, st);
  return e;
}

}  // namespace qad
