// Log probabilities of given tokens, entropy and top alternatives of logits in one reading of them, and the gradient
// with respect to the logits.
//
//   y_v = b log2(e) (z_v - m),  S = sum 2^y,  U = sum 2^y y      m: the running maximum, per thread
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;                  // 16-byte vectors of a thread per step
constexpr int kNotes = 40;                // steps whose largest logits are noted before candidates are taken
// candidates of a block: about twice K logits reach the bound
constexpr int kCapSmall = 1024, kCapLarge = 4096, kSmallK = 256;
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

// v, rounded down to the logits' type
template <typename ZT>
__device__ __forceinline__ float floor_of(float v) {
  if constexpr (sizeof(ZT) == 4) return v;
  else return __bfloat162float(__float2bfloat16_rd(v));
}

struct Logprobs {
  const void* z;
  const int32_t* token;
  float *logp, *lse, *entropy, *top_logit;
  int32_t *top_idx, *err;
  int64_t ldz;
  int V, K, cap;
  float b;
};

// The 16 logits of a thread in one step: vectors of 16 bytes, kThreads apart.  `at` counts elements from the 16-byte
// boundary at or before the range; what lies outside [from, to) counts as -inf and is not read past `to`.
template <typename ZT>
struct Step {
  static constexpr int kVec = 16 / sizeof(ZT), kPer = kVec * kVecs, kStep = kThreads * kPer;  // of a thread and a block
  uint4 raw[kVecs];

  __device__ __forceinline__ static int place(int step, int i, int thread) {
    return (step * kVecs * kThreads + i * kThreads + thread) * kVec;
  }

  // a step all of which lies before `to`
  __device__ __forceinline__ void load(const uint4* at) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) raw[i] = __ldg(at + i * kThreads);
  }
  // the last one: what lies behind `to` is not read and counts as -inf
  __device__ __forceinline__ void load_last(const ZT* base, int step, int to) {
#pragma unroll 1
    for (int i = 0; i < kVecs; ++i) {
      const int at = place(step, i, threadIdx.x);
      uint4 v;
      if (at + kVec <= to) {
        v = __ldg(reinterpret_cast<const uint4*>(base + at));
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
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (j == i) raw[j] = v;
    }
  }
  // what lies before `from` (in the first vector of the first thread) becomes -inf
  __device__ __forceinline__ void cut_front(int from) {
    if (threadIdx.x == 0 && from > 0) {
      uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < from) {
          if constexpr (sizeof(ZT) == 4) w[j] = 0xff800000u;
          else w[j / 2] = j % 2 ? (w[j / 2] & 0xffffu) | 0xff800000u : (w[j / 2] & 0xffff0000u) | 0xff80u;
        }
      raw[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // the largest; a NaN does not count
  __device__ __forceinline__ float largest() const {
    if constexpr (sizeof(ZT) == 4) {
      float top = __uint_as_float(raw[0].x);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        top = fmaxf(top, fmaxf(__uint_as_float(raw[i].x), __uint_as_float(raw[i].y)));
        top = fmaxf(top, fmaxf(__uint_as_float(raw[i].z), __uint_as_float(raw[i].w)));
      }
      return top;
    } else {
      auto pair = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
      __nv_bfloat162 top = pair(raw[0].x);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        top = __hmax2(top, __hmax2(pair(raw[i].x), pair(raw[i].y)));
        top = __hmax2(top, __hmax2(pair(raw[i].z), pair(raw[i].w)));
      }
      return fmaxf(__low2float(top), __high2float(top));
    }
  }
  // a lower bound of the logits as raise() takes it
  __device__ __forceinline__ static uint32_t packed(float low) {
    if constexpr (sizeof(ZT) == 4) return __float_as_uint(low);
    else return pack_bf16(low, low);
  }
  // max(z, low) of all; a NaN stays
  __device__ __forceinline__ void raise(uint32_t low) {
    auto up = [&](uint32_t v) {
      if constexpr (sizeof(ZT) == 4) {
        return __float_as_uint(floor_nan(__uint_as_float(v), __uint_as_float(low)));
      } else {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(low));
        return r;
      }
    };
#pragma unroll
    for (int i = 0; i < kVecs; ++i) raw[i] = make_uint4(up(raw[i].x), up(raw[i].y), up(raw[i].z), up(raw[i].w));
  }
  // logits i and i + 1 (i even)
  __device__ __forceinline__ uint64_t pair(int i) const {
    const uint4& v = raw[i / kVec];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(ZT) == 4) return f2pack(__uint_as_float(w[i % 4]), __uint_as_float(w[i % 4 + 1]));
    else return f2pack(bf16lo(w[i % 8 / 2]), bf16hi(w[i % 8 / 2]));
  }
  // the place of a thread's f[j]
  __device__ __forceinline__ static int at_of(int step, int j, int thread) {
    return place(step, j / kVec, thread) + j % kVec;
  }
  // the logits at a place, read again: one, or a vector (what lies behind `to` is not read)
  __device__ __forceinline__ static void vector(const ZT* base, int at, int to, float* f) {
    if (at + kVec <= to) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(base + at));
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
      for (int j = 0; j < kVec; ++j) f[j] = at + j < to ? one(base, at + j) : -INFINITY;
    }
  }
  __device__ __forceinline__ static float one(const ZT* base, int at) {
    if constexpr (sizeof(ZT) == 4) return __ldg(reinterpret_cast<const float*>(base) + at);
    else return bf16lo(__ldg(reinterpret_cast<const unsigned short*>(base) + at));
  }
};

// Sorts s_key[0, n2) in falling order, n2 a power of two.  Exchanges over up to 32 keys stay within a warp's 64.
__device__ __forceinline__ void sort_keys(uint64_t* s_key, int n2) {
  bool wide = true;
  for (int size = 2; size <= n2; size *= 2) {
    for (int half = size / 2; half; half /= 2) {
      if (wide || half > 32) __syncthreads();
      else __syncwarp();
      wide = half > 32;
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
#pragma unroll 8
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

struct TopSmem {  // in front of `cap` keys (8 bytes) and groups (2 bytes) in dynamic shared memory
  uint16_t note[kNotes][kThreads];
  uint32_t bound[kWarps];
  int n, groups, pad[2];
};

// What a block knows of its part of a row, and the candidates it takes from it.
template <typename ZT>
struct Top {
  using St = Step<ZT>;
  TopSmem& s;
  uint64_t* key;    // the candidates
  uint16_t* group;  // groups of 16 to read again: step * kThreads + thread
  const ZT* base;
  int lo, from, to, K, cap;
  uint64_t above;  // a candidate's key is larger: K better ones are listed

  __device__ __forceinline__ uint64_t key_of(float v, int at) const {
    return v == v ? ((uint64_t)order_of(v) << 32) | (0xffffffffu - (uint32_t)(lo + at - from)) : 0;
  }
  // cuts the list to the K best; the caller has passed a barrier since the last candidate
  __device__ __forceinline__ void cut(int n) {
    n = keep_best(key, n, K);
    if (n == K && key[n - 1] > above) above = key[n - 1];
    __syncthreads();
    if (threadIdx.x == 0) s.n = n;
    __syncthreads();
  }
  // the candidates of the steps [first, first + steps) behind the `held` listed ones
  __device__ __forceinline__ void take(int first, int steps, int held) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    // warps all of whose lanes have logits; q lanes of each of them, r notes of a lane
    const int full = min(kWarps, max(1, to / (32 * St::kVec)));
    const int quota = (K + full - 1) / full, r = (quota + 15) / 16, q = (quota + r - 1) / r;
    const uint16_t* mine = &s.note[0][tid];
    uint32_t w = 0;
    if (r == 1) w = warp_qth(rth_note<1>(mine, steps, 1), q, lane);
    else if (r <= 8) w = warp_qth(rth_note<8>(mine, steps, r), q, lane);
    if (lane == 0) s.bound[warp] = w;
    if (tid == 0) s.groups = 0;
    __syncthreads();
    w = __reduce_min_sync(0xffffffffu, s.bound[min(lane, full - 1)]);
    const uint32_t bound = max(w << 16, (uint32_t)(above >> 32));
#pragma unroll 8
    for (int i = 0; i < steps; ++i) {
      if (mine[i * kThreads] >= bound >> 16) {
        const int slot = atomicAdd(&s.groups, 1);
        if (slot < cap) group[slot] = (uint16_t)(i * kThreads + tid);
      }
    }
    __syncthreads();
    const int groups = s.groups;
    if (groups <= cap) {
      const float bound_f = bound <= 0x007fffffu ? -INFINITY : value_of(bound);
      for (int i = tid; i < groups * kVecs; i += kThreads) {
        const int g = group[i / kVecs];
        const int at = St::place(first + g / kThreads, i % kVecs, g % kThreads);
        float f[St::kVec];
        St::vector(base, at, to, f);
#pragma unroll
        for (int j = 0; j < St::kVec; ++j) {
          if (!(f[j] >= bound_f) || at + j < from || at + j >= to) continue;
          const uint64_t k = key_of(f[j], at + j);
          if (k > above && (uint32_t)(k >> 32) >= bound) {
            const int slot = atomicAdd(&s.n, 1);
            if (slot < cap) key[slot] = k;
          }
        }
      }
      __syncthreads();
      if (s.n <= cap) return;
    }
    // very many reach the bound (equal logits, or fewer groups than K): all logits of these steps, kThreads at a time,
    // and the list is cut whenever the next ones might not fit
    __syncthreads();
    if (tid == 0) s.n = held;
    __syncthreads();
    for (int i = 0; i < steps * St::kPer; ++i) {
      const int n = s.n;
      __syncthreads();  // read by everybody before anybody adds
      if (n > cap - kThreads) cut(n);
      const int at = St::at_of(first + i / St::kPer, i % St::kPer, tid);
      if (at >= from && at < to) {
        const uint64_t k = key_of(St::one(base, at), at);
        if (k > above && (uint32_t)(k >> 32) >= bound) key[atomicAdd(&s.n, 1)] = k;
      }
      __syncthreads();
    }
  }
};

template <typename ZT, bool TOP, bool ENT>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(Logprobs q, int parts) {
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
  const int steps = (to + St::kStep - 1) / St::kStep;
  const float b2 = q.b * kLog2e;
  // S = sum of 2^y and U = sum of 2^y y with y = b2 z - R, R = fp32(b2 m): one instruction for two logits.  m follows the
  // largest logit only when that is above `enough` (2^y past 2^8): most steps rescale nothing.  R is off b2 m
  // by `off` (exact), which is taken out when sums join.  A logit below `least` (y <= -200, 2^y = 0) counts as `least`, so
  // that -inf gives 0 * y and not NaN.  `wild`: products of logits of 10^36 and more would leave fp32's range; there
  // y = b2 (z - m), clamped.
  float m = -INFINITY, enough = -INFINITY, off = 0.0f;
  const float span = 200.0f / b2;
  uint64_t s2 = f2pack(0.0f, 0.0f), u2 = s2, nr = s2;  // S and U of the even and odd logits; -R twice
  const uint64_t bb = f2pack(b2, b2);
  uint32_t least = St::packed(floor_of<ZT>(-span));
  bool wild = !(span < 3e38f);
  TopSmem& ts = *reinterpret_cast<TopSmem*>(smem);
  uint64_t* keys = reinterpret_cast<uint64_t*>(smem + sizeof(TopSmem));
  if (TOP && tid == 0) ts.n = 0;

  uint16_t* note = &ts.note[0][tid];
  auto see = [&](St& now) {
    const float top = now.largest();
    if (top > enough) {
      const float R = top * b2, low = floor_of<ZT>(__fsub_rd(top, span));
      wild = !(fabsf(fmaf(low, b2, -R)) < 3e38f);
      const float off2 = wild ? 0.0f : fmaf(top, b2, -R);
      if (m > -INFINITY) {
        const float d = (m - top) * b2 - off + off2, c = ex2(d);
        const uint64_t cc = f2pack(c, c);
        if constexpr (ENT) u2 = c == 0.0f ? 0 : f2mul(cc, f2fma(s2, f2pack(d, d), u2));
        s2 = f2mul(s2, cc);
      }
      m = top;
      enough = m + 8.0f / b2;
      off = off2;
      nr = f2pack(-R, -R);
      least = St::packed(low);
    }
    if (!wild) {
      now.raise(least);
#pragma unroll
      for (int i = 0; i < St::kPer; i += 2) {
        const uint64_t y2 = f2fma(now.pair(i), bb, nr);
        const float2 y = f2unpack(y2);
        const uint64_t e2 = f2pack(ex2(y.x), ex2(y.y));
        s2 = f2add(s2, e2);
        if constexpr (ENT) u2 = f2fma(e2, y2, u2);
      }
    } else {
      const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < St::kPer; i += 2) {
        const float2 f = f2unpack(now.pair(i));
        const float y0 = floor_nan((f.x - ref) * b2, -200.0f), y1 = floor_nan((f.y - ref) * b2, -200.0f);
        const uint64_t e2 = f2pack(ex2(y0), ex2(y1));
        s2 = f2add(s2, e2);
        if constexpr (ENT) u2 = f2fma(e2, f2pack(y0, y1), u2);
      }
    }
    if constexpr (TOP) {
      *note = (uint16_t)(order_of(top) >> 16);
      note += kThreads;
    }
  };
  // candidates are taken every kNotes steps
  const int whole = to / St::kStep;
  const uint4* ahead = reinterpret_cast<const uint4*>(base) + tid;
  auto fetch = [&](St& v, int step, int end) {
    if (step >= end) return;
    if (step < whole) v.load(ahead + (int64_t)step * (kVecs * kThreads));
    else v.load_last(base, step, to);
  };
  uint64_t above = 0;
  for (int first = 0; first < steps; first += kNotes) {
    const int end = min(steps, first + kNotes);
    St even, odd;
    fetch(even, first, end);
    fetch(odd, first + 1, end);
    if (first == 0) even.cut_front(from);
    note = &ts.note[0][tid];
    for (int step = first; step < end; step += 2) {
      see(even);
      fetch(even, step + 2, end);
      if (step + 1 < end) {
        see(odd);
        fetch(odd, step + 3, end);
      }
    }
    if constexpr (TOP) {
      Top<ZT> alt = {ts, keys, reinterpret_cast<uint16_t*>(keys + q.cap), base, lo, from, to, q.K, q.cap, above};
      __syncthreads();
      if (first > 0) alt.cut(ts.n);
      alt.take(first, end - first, ts.n);
      above = alt.above;
    }
  }
  int n = 0;
  if constexpr (TOP) {
    __syncthreads();
    n = keep_best(keys, ts.n, q.K);
  }

  // the block's sums
  {
    float S = f2unpack(s2).x + f2unpack(s2).y, U = f2unpack(u2).x + f2unpack(u2).y;
    const float wm = warp_max(m);
    const float d = m == -INFINITY ? 0.0f : (m - wm) * b2 - off, c = ex2(d);
    // a thread that saw nothing but -inf and NaN has m = -inf, and S = 0 or NaN
    if constexpr (ENT) U = c == 0.0f || m == -INFINITY ? 0.0f : c * fmaf(S, d, U);
    S = warp_sum(S * c);
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
          const uint64_t* theirs = cluster.map_shared_rank(keys, r);
          for (int i = tid; i < more; i += kThreads) keys[n + i] = theirs[i];
          n += more;
        }
        n = keep_best(keys, n, q.K);
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
    const float l2 = log2f(s), ls = kLn2 * l2;
    if (q.lse) q.lse[row] = empty ? -INFINITY : M == -INFINITY ? s + NAN : fmaf(M, q.b, ls);
    if (ENT) q.entropy[row] = empty ? 0.0f : M == -INFINITY ? NAN : fmaxf(kLn2 * (l2 - s_sum[2] / s), 0.0f) + 0.0f * s;
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
      const uint64_t key = i < n ? keys[i] : 0;
      if (q.top_idx) q.top_idx[row * q.K + i] = i < n ? (int32_t)(0xffffffffu - (uint32_t)key) : -1;
      if (q.top_logit) q.top_logit[row * q.K + i] = i < n ? value_of((uint32_t)(key >> 32)) : -INFINITY;
    }
  }
}

template <typename ZT, bool TOP, bool ENT>
cudaError_t launch(const Logprobs& q, int64_t N, cudaStream_t st) {
  // as many blocks for a row as fill the GPU twice, while each has a whole step and their candidates fit one block's list
  int parts = 1;
  while (parts < 8 && 2 * parts * N <= 2 * (int64_t)num_sms() && q.V / (2 * parts) >= Step<ZT>::kStep / 4 &&
         (!TOP || 2 * parts * q.K <= q.cap))
    parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(N * parts), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  if (TOP) {
    cfg.dynamicSmemBytes = sizeof(TopSmem) + 10 * (size_t)q.cap;
    if (cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<ZT, TOP, ENT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(sizeof(TopSmem) + 10 * kCapLarge)))
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
  q.cap = K <= kSmallK ? kCapSmall : kCapLarge;
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
