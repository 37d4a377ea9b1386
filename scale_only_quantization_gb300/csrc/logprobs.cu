// Log probabilities of given tokens, entropy and top alternatives of logits in one reading of them, and the gradient
// with respect to the logits.
//
//   y_v = (z_v - m) b log2(e),  S = sum 2^y,  U = sum 2^y y      m: the running maximum, per thread
//   lse = b m + ln S,   H = ln S - ln2 U / S,   logp = b (z_t - m) - ln S
//   dz = b (g (1[v = t] - p) - h p (log p + H)),   p = exp(b z - lse)
//
// Each thread keeps m, S and U of the logits it has seen (a new maximum rescales S and U); the block joins them at the
// end.  The alternatives: while it streams, a thread only notes the largest of each 16 logits (16 bits of its order, in
// shared memory).  At the row's end each warp takes its q-th largest lane, a lane counting by its r-th largest note, with
// 16 q r >= K: at least K logits reach the least of the 16 warps' values, and not many more than that do, so that few of
// the groups have to be read again (they are still in L2).  Their logits that reach the bound are the candidates, ordered
// by (value, index) as one 64-bit key: equal logits stand by rising index.  Taking candidates while streaming, under a
// bound renewed at steps 0, 1, 2, 4, ..., cost more than the whole softmax (500 against 230 us for 4096 x 151936).
// Rows are split over the blocks of a cluster when there are too few to fill the GPU; the cluster's first block joins
// the others' sums and candidates out of their shared memory.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace qad {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kPer = 16;                  // logits of a thread per step
constexpr int kStep = kThreads * kPer;    // of a block
constexpr int kCap = 4096;                // candidates of a block
constexpr int kNotes = 32;                // steps whose largest logits are noted before candidates are taken
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

  __device__ __forceinline__ static int place(int step, int i, int thread) {
    return (step * kVecs * kThreads + i * kThreads + thread) * kVec;
  }

  __device__ __forceinline__ void load(const ZT* base, int step, int to) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = place(step, i, threadIdx.x);
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
  // the place of a thread's f[j]
  __device__ __forceinline__ static int at_of(int step, int j, int thread) {
    return place(step, j / kVec, thread) + j % kVec;
  }
  // the logit at a place, read again
  __device__ __forceinline__ static float one(const ZT* base, int at) {
    if constexpr (sizeof(ZT) == 4) return __ldg(reinterpret_cast<const float*>(base) + at);
    else return bf16lo(__ldg(reinterpret_cast<const unsigned short*>(base) + at));
  }
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

// Orders the n candidates and keeps the K best; returns how many are left.  Up to kThreads of them each thread counts the
// keys above its own (all differ); more are sorted.
__device__ __forceinline__ int keep_best(uint64_t* s_key, int n, int K) {
  __syncthreads();
  if (n <= kThreads) {
    const int i = threadIdx.x;
    const uint64_t mine = i < n ? s_key[i] : 0;
    int rank = 0;
    if ((i & ~31) < n) {
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += s_key[j] > mine;
    }
    __syncthreads();
    if (i < n) s_key[rank] = mine;
    __syncthreads();
  } else {
    int n2 = 2 * kThreads;
    while (n2 < n) n2 *= 2;
    for (int i = n + threadIdx.x; i < n2; i += kThreads) s_key[i] = 0;
    sort_keys(s_key, n2);
  }
  return min(n, K);
}

// The q-th largest (q = 1 .. 32) of a warp's values: a bitonic sort of the lanes, falling.
__device__ __forceinline__ uint32_t warp_qth(uint32_t v, int q, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
    for (int half = size / 2; half; half /= 2) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, half);
      v = ((lane & half) == 0) == ((lane & size) == 0) ? max(v, o) : min(v, o);
    }
  }
  return __shfl_sync(0xffffffffu, v, q - 1);
}

// The r-th largest of a thread's n notes (0 if there are fewer).
template <int R>
__device__ __forceinline__ uint32_t rth_note(const uint16_t* notes, int n, int r) {
  uint32_t best[R];
#pragma unroll
  for (int i = 0; i < R; ++i) best[i] = 0;
  for (int s = 0; s < n; ++s) {
    uint32_t v = notes[s * kThreads];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint32_t hi = max(best[i], v);
      v = min(best[i], v);
      best[i] = hi;
    }
  }
  uint32_t v = best[0];
#pragma unroll
  for (int i = 1; i < R; ++i) v = i == r - 1 ? best[i] : v;
  return v;
}

struct TopSmem {  // dynamic shared memory
  uint64_t key[kCap];
  uint16_t note[kNotes][kThreads];
  uint16_t group[kCap];  // groups to read again: step * kThreads + thread
  uint32_t bound[kWarps];
  int n, groups;
};

// What a block knows of its part of a row, and the candidates it takes from it.
template <typename ZT>
struct Top {
  using St = Step<ZT>;
  TopSmem& s;
  const ZT* base;
  int lo, from, to, K;
  uint64_t above;  // a candidate's key is larger: K better ones are listed

  __device__ __forceinline__ uint64_t key_at(int at) const {
    const float v = St::one(base, at);
    return v == v ? ((uint64_t)order_of(v) << 32) | (0xffffffffu - (uint32_t)(lo + at - from)) : 0;
  }
  // cuts the list to the K best; the caller has passed a barrier since the last candidate
  __device__ __forceinline__ void cut(int n) {
    n = keep_best(s.key, n, K);
    if (n == K && s.key[n - 1] > above) above = s.key[n - 1];
    __syncthreads();
    if (threadIdx.x == 0) s.n = n;
    __syncthreads();
  }
  // the candidates of the steps [first, first + steps) behind the `held` listed ones
  __device__ __forceinline__ void take(int first, int steps, int held) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    // warps all of whose lanes have logits; q lanes of each of them, r notes of a lane
    const int full = min(kWarps, max(1, to / (32 * St::kVec)));
    const int quota = (K + full - 1) / full, r = (quota + 7) / 8, q = (quota + r - 1) / r;
    const uint16_t* mine = &s.note[0][tid];
    uint32_t w = 0;
    if (r <= 8) w = warp_qth(r == 1 ? rth_note<1>(mine, steps, 1) : rth_note<8>(mine, steps, r), q, lane);
    if (lane == 0) s.bound[warp] = w;
    if (tid == 0) s.groups = 0;
    __syncthreads();
    w = __reduce_min_sync(0xffffffffu, s.bound[min(lane, full - 1)]);
    const uint32_t bound = max(w << 16, (uint32_t)(above >> 32));
    for (int i = 0; i < steps; ++i) {
      if (mine[i * kThreads] >= bound >> 16) {
        const int slot = atomicAdd(&s.groups, 1);
        if (slot < kCap) s.group[slot] = (uint16_t)(i * kThreads + tid);
      }
    }
    __syncthreads();
    const int groups = s.groups;
    if (groups <= kCap) {
      for (int i = tid; i < groups * kPer; i += kThreads) {
        const int g = s.group[i / kPer];
        const int at = St::at_of(first + g / kThreads, i % kPer, g % kThreads);
        if (at < from || at >= to) continue;
        const uint64_t key = key_at(at);
        if (key > above && (uint32_t)(key >> 32) >= bound) {
          const int slot = atomicAdd(&s.n, 1);
          if (slot < kCap) s.key[slot] = key;
        }
      }
      __syncthreads();
      if (s.n <= kCap) return;
    }
    // very many reach the bound (equal logits, or fewer groups than K): all logits of these steps, kThreads at a time,
    // and the list is cut whenever the next ones might not fit
    __syncthreads();
    if (tid == 0) s.n = held;
    __syncthreads();
    for (int i = 0; i < steps * kPer; ++i) {
      const int n = s.n;
      __syncthreads();  // read by everybody before anybody adds
      if (n > kCap - kThreads) cut(n);
      const int at = St::at_of(first + i / kPer, i % kPer, tid);
      if (at >= from && at < to) {
        const uint64_t key = key_at(at);
        if (key > above && (uint32_t)(key >> 32) >= bound) s.key[atomicAdd(&s.n, 1)] = key;
      }
      __syncthreads();
    }
  }
};

template <typename ZT, bool TOP, bool ENT>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(Logprobs q, int parts) {
  using St = Step<ZT>;
  extern __shared__ __align__(16) uint8_t smem[];
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
  TopSmem& ts = *reinterpret_cast<TopSmem*>(smem);
  Top<ZT> alt = {ts, base, lo, from, to, q.K, 0};
  if (TOP && tid == 0) ts.n = 0;

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
      ts.note[step % kNotes][tid] = (uint16_t)(order_of(top) >> 16);
      if (step % kNotes == kNotes - 1 && step + 1 < steps) {
        __syncthreads();
        if (step >= kNotes) alt.cut(ts.n);
        alt.take(step - (kNotes - 1), kNotes, ts.n);
      }
    }
    now = next;
  }
  int n = 0;
  if constexpr (TOP) {
    __syncthreads();
    if (steps > kNotes) alt.cut(ts.n);
    if (steps > 0) alt.take((steps - 1) / kNotes * kNotes, (steps - 1) % kNotes + 1, ts.n);
    n = keep_best(ts.key, ts.n, q.K);
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
  __syncthreads();
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
    if constexpr (TOP) ts.n = n;
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
          const int more = *cluster.map_shared_rank(&ts.n, r);
          const uint64_t* keys = cluster.map_shared_rank(ts.key, r);
          for (int i = tid; i < more; i += kThreads) ts.key[n + i] = keys[i];
          n += more;
        }
        n = keep_best(ts.key, n, q.K);
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
      const uint64_t key = i < n ? ts.key[i] : 0;
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
  if (TOP) {
    cfg.dynamicSmemBytes = sizeof(TopSmem);
    if (cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<ZT, TOP, ENT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sizeof(TopSmem)))
      return e;
  }
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
