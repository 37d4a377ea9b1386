// Log probabilities of given tokens, entropy and top alternatives of logits in one reading of them, and the gradient
// with respect to the logits.
//
//   y_v = b log2(e) (z_v - m),  S = sum 2^y,  U = sum 2^y y      m: a reference near the largest logit, per thread
//   lse = b m + ln S,   H = ln S - ln2 U / S,   logp = b (z_t - m) - ln S
//   dz = b (g (1[v = t] - p) - h p (log p + H)),   p = exp(b z - lse)
//
// Each thread keeps m, S and U of the logits it has seen; the block joins them at the row's end.  The alternatives: while
// it streams, a thread only notes the largest of each half of its logits of a step (16 bits of it, in shared memory).  At the
// row's end each warp takes its q-th largest lane, a lane counting by its r-th largest note, with 8 q r >= K: at least K
// logits reach the least of the 8 warps' values, and not many more than that do (about 120 for K = 64 of 151936), so that
// few of the groups have to be read again.  Their logits that reach the bound are the candidates, ordered by (value, index)
// as one 64-bit key: equal logits stand by rising index.  Taking candidates while streaming, under a bound renewed at steps
// 0, 1, 2, 4, ..., cost more than the whole softmax (500 against 230 us for 4096 x 151936).
// Rows are split over the blocks of a cluster when there are too few to fill the GPU; the cluster's first block joins
// the others' sums and candidates out of their shared memory.
//
// 4096 x 151936 bf16 (1.24 GB): without alternatives 191 us, 6.5 TB/s, bound by memory; with the top 64 282 us, 4.4 TB/s:
// 19 of a row's 57 thousand cycles (by clocks in an earlier form) go into its alternatives, most of them latencies, and the
// blocks that stream meanwhile are bound by the loads they have in flight.  One row of 151936 fp32 logits with 20
// alternatives 12.3 us.  The gradient of 4096 x 151936 385 to 394 us, 6.3 to 6.5 TB/s.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace qad {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;                  // 16-byte vectors of a thread per step
// Steps whose largest logits are noted before candidates are taken, a capacity: 20 KB of shared memory hold the notes of
// 163840 bf16 logits (81920 fp32 ones) of a block; a longer part of a row takes candidates more than once.
constexpr int kNotes = 20;
// candidates of a block: about twice K logits reach the bound
constexpr int kCapSmall = 1024, kCapLarge = 4096, kSmallK = 256;
// sort_keys() works on powers of two from 2 * kThreads up to the capacity
static_assert((kThreads & (kThreads - 1)) == 0 && 2 * kThreads <= kCapSmall && (kCapSmall & (kCapSmall - 1)) == 0 &&
              (kCapLarge & (kCapLarge - 1)) == 0, "");
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

// b (v - ref), where v - ref may leave fp32's range: halves do not
__device__ __forceinline__ float over(float v, float ref, float b) { return fmaf(0.5f, v, -0.5f * ref) * (2.0f * b); }

// min(max(v, lo), hi) that keeps a NaN
__device__ __forceinline__ float clamp_nan(float v, float lo, float hi) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(floor_nan(v, lo)), "f"(hi));
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
  // the largest, and the upper 16 bits of the largest of each half; a NaN does not count (except among NaNs)
  __device__ __forceinline__ float largest(uint16_t* note0, uint16_t* note1) const {
    if constexpr (sizeof(ZT) == 4) {
      auto most = [](const uint4& a, const uint4& b) {
        const float x = fmaxf(fmaxf(__uint_as_float(a.x), __uint_as_float(a.y)), fmaxf(__uint_as_float(a.z), __uint_as_float(a.w)));
        const float y = fmaxf(fmaxf(__uint_as_float(b.x), __uint_as_float(b.y)), fmaxf(__uint_as_float(b.z), __uint_as_float(b.w)));
        return fmaxf(x, y);
      };
      const float t0 = most(raw[0], raw[1]), t1 = most(raw[2], raw[3]);
      *note0 = (uint16_t)(__float_as_uint(t0) >> 16);
      *note1 = (uint16_t)(__float_as_uint(t1) >> 16);
      return fmaxf(t0, t1);
    } else {
      auto most = [](const uint4& a, const uint4& b) {
        auto pair = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
        const __nv_bfloat162 x = __hmax2(__hmax2(pair(a.x), pair(a.y)), __hmax2(pair(a.z), pair(a.w)));
        const __nv_bfloat162 y = __hmax2(__hmax2(pair(b.x), pair(b.y)), __hmax2(pair(b.z), pair(b.w)));
        const __nv_bfloat162 m = __hmax2(x, y), r = __hmax2(m, __lowhigh2highlow(m));
        return *reinterpret_cast<const uint32_t*>(&r);
      };
      const uint32_t t0 = most(raw[0], raw[1]), t1 = most(raw[2], raw[3]);
      *note0 = (uint16_t)t0;
      *note1 = (uint16_t)t1;
      return fmaxf(bf16lo(t0), bf16lo(t1));
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
// keys above one (all differ), two threads a key if there are half as many; more are sorted.
__device__ __forceinline__ int keep_best(uint64_t* s_key, int n, int K) {
  __syncthreads();
  if (n <= kThreads) {
    const int share = n <= kThreads / 2 ? 2 : 1, i = threadIdx.x / share;
    const uint64_t mine = i < n ? s_key[i] : 0;
    int rank = 0;
    if ((threadIdx.x & ~31) < n * share) {
#pragma unroll 8
      for (int j = threadIdx.x % share; j < n; j += share) rank += s_key[j] > mine;
      if (share > 1) rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    }
    __syncthreads();
    if (i < n && threadIdx.x % share == 0) s_key[rank] = mine;
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

// The upper 16 bits of order_of() from those of the number, or one less for -0, which no bound of take() tells apart.
__device__ __forceinline__ uint32_t note_order(uint32_t b) {
  return (b & 0x7fffu) > 0x7f80u ? 0u : (b & 0x8000u) ? b ^ 0xffffu : b | 0x8000u;
}

// The r-th largest of a thread's n notes, by their orders (0 if there are fewer).
template <int R>
__device__ __forceinline__ uint32_t rth_note(const uint16_t* notes, int n, int r) {
  uint32_t best[R];
#pragma unroll
  for (int i = 0; i < R; ++i) best[i] = 0;
#pragma unroll 8
  for (int s = 0; s < n; ++s) {
    uint32_t v = note_order(notes[s * kThreads]);
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
  uint16_t note[2 * kNotes][kThreads];  // of each half of a thread's logits of a step: the largest, its upper 16 bits
  uint32_t bound[kWarps];
  int n, groups, pad[2];
};

// What a block knows of its part of a row, and the candidates it takes from it.
template <typename ZT>
struct Top {
  using St = Step<ZT>;
  TopSmem& s;
  uint64_t* key;    // the candidates
  uint16_t* group;  // groups (halves) to read again: number * kThreads + thread
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
  // the candidates of the steps [first, first + steps) behind the `held` listed ones; peak: this thread's largest logit
  __device__ __forceinline__ void take(int first, int steps, int held, float peak) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    // warps all of whose lanes have logits; q lanes of each of them, r notes of a lane
    const int full = min(kWarps, max(1, to / (32 * St::kVec)));
    const int quota = (K + full - 1) / full, r = (quota + 15) / 16, q = (quota + r - 1) / r;
    const uint16_t* mine = &s.note[0][tid];
    uint32_t w = 0;
    if (r == 1) w = warp_qth(order_of(peak) >> 16, q, lane);
    else if (r <= 8) w = warp_qth(rth_note<8>(mine, 2 * steps, r), q, lane);
    if (lane == 0) s.bound[warp] = w;
    if (tid == 0) s.groups = 0;
    __syncthreads();
    w = __reduce_min_sync(0xffffffffu, s.bound[min(lane, full - 1)]);
    const uint32_t bound = max(w << 16, (uint32_t)(above >> 32));
    const uint32_t least = bound >> 16 == 0x8000u ? 0x7fffu : bound >> 16;
    if (order_of(peak) >> 16 >= least) {
#pragma unroll 8
      for (int i = 0; i < 2 * steps; ++i) {
        if (note_order(mine[i * kThreads]) >= least) {
          const int slot = atomicAdd(&s.groups, 1);
          if (slot < cap) group[slot] = (uint16_t)(i * kThreads + tid);
        }
      }
    }
    __syncthreads();
    const int groups = s.groups;
    if (groups <= cap) {
      const float bound_f = bound <= 0x007fffffu ? -INFINITY : value_of(bound);
      for (int i = tid; i < 2 * groups; i += kThreads) {  // a vector to a thread, a group has two
        const int g = group[i / 2], half = g / kThreads;
        const int at = St::place(first + half / 2, half % 2 * 2 + i % 2, g % kThreads);
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

// What a thread keeps of the logits it has seen.
struct Seen {
  float m, off, peak;  // the reference; see stream(); the largest logit (TOP)
  uint64_t s2, u2;     // S and U of the even and odd logits
};

// The steps [first, end) of a block's part of a row.  Not inlined: the loop keeps its registers to itself.
//
// S = sum of 2^y and U = sum of 2^y y with y = b2 z - R, R = fp32(b2 m): one instruction for two logits.  m follows the
// largest logit only when that is above `enough` (2^y past 2^8): most steps rescale nothing.  R is off b2 m by `off`
// (exact), which is taken out when sums join.  A logit below `least` (y <= -200, 2^y = 0) counts as `least`, so that -inf
// gives 0 * y and not NaN.  `wild`: there y = b2 (z - m), clamped, without R.  It is for |R| from 2^24 on, where `off` (half
// a unit of R's last place) would pass 1 and then the exponents themselves (a thread that has seen only a mask's -1e10 would
// add up 2^off), and where 200 / b2 or products of logits of 10^36 and more would leave fp32's range.  There m follows every
// larger logit: 8 / b2 may not be a number either.
template <typename ZT, bool TOP, bool ENT>
__device__ __noinline__ Seen stream(const ZT* base, int first, int end, int from, int to, uint16_t* note, float b2,
                                    Seen seen) {
  using St = Step<ZT>;
  float m = seen.m, off = seen.off, peak = seen.peak;
  uint64_t s2 = seen.s2, u2 = seen.u2;
  const uint64_t bb = f2pack(b2, b2);
  float enough;
  uint64_t nr;
  uint32_t least;
  bool wild;
  auto refer = [&]() {  // by m: R and what goes with it; returns `off`
    const float unit = 8.0f / b2;  // taken again each time: a register less over the loop, which has none to spare
    const float ref = m == -INFINITY ? 0.0f : m, R = ref * b2, low = floor_of<ZT>(__fsub_rd(ref, 25.0f * unit));
    wild = !(fabsf(fmaf(low, b2, -R)) < 3e38f && fabsf(R) < 0x1p24f);
    enough = wild ? m : m + unit;
    nr = f2pack(-R, -R);
    least = St::packed(low);
    return wild ? 0.0f : fmaf(ref, b2, -R);
  };
  refer();
  auto see = [&](St& now) {
    uint16_t note0, note1;
    const float top = now.largest(&note0, &note1);
    if (top > enough) {
      const float old = m;
      m = top;
      const float off2 = refer();
      if (old > -INFINITY) {
        const float d = over(old, top, b2) - off + off2, c = ex2(d);
        const uint64_t cc = f2pack(c, c);
        if constexpr (ENT) u2 = c == 0.0f ? 0 : f2mul(cc, f2fma(s2, f2pack(d, d), u2));
        s2 = f2mul(s2, cc);
      }
      off = off2;
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
        const float y0 = floor_nan(over(f.x, ref, b2), -200.0f), y1 = floor_nan(over(f.y, ref, b2), -200.0f);
        const uint64_t e2 = f2pack(ex2(y0), ex2(y1));
        s2 = f2add(s2, e2);
        if constexpr (ENT) u2 = f2fma(e2, f2pack(y0, y1), u2);
      }
    }
    if constexpr (TOP) {
      peak = fmaxf(peak, top);
      note[0] = note0;
      note[kThreads] = note1;
      note += 2 * kThreads;
    }
  };
  const int whole = to / St::kStep;
  const uint4* ahead = reinterpret_cast<const uint4*>(base) + threadIdx.x;
  auto fetch = [&](St& v, int step) {
    if (step >= end) return;
    if (step < whole) v.load(ahead + (int64_t)step * (kVecs * kThreads));
    else v.load_last(base, step, to);
  };
  St even, odd;
  fetch(even, first);
  fetch(odd, first + 1);
  if (first == 0) even.cut_front(from);
  for (int step = first; step < end; step += 2) {
    see(even);
    fetch(even, step + 2);
    if (step + 1 < end) {
      see(odd);
      fetch(odd, step + 3);
    }
  }
  return {m, off, peak, s2, u2};
}

template <typename ZT, bool TOP, bool ENT>
__global__ void __launch_bounds__(kThreads, TOP ? 3 : 4) logprobs_kernel(Logprobs q, int parts) {
  using St = Step<ZT>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_m[kWarps], s_s[kWarps], s_u[kWarps];
  __shared__ float s_sum[3], s_zt;
  __shared__ int s_token;
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
  if (tid == 0 && part == 0 && q.token) {  // the row's token and its logit, read early
    s_token = __ldg(q.token + row);
    if (q.logp && s_token >= 0 && s_token < q.V) s_zt = St::one(zrow, s_token);
  }
  TopSmem& ts = *reinterpret_cast<TopSmem*>(smem);
  uint64_t* keys = reinterpret_cast<uint64_t*>(smem + sizeof(TopSmem));
  if (TOP && tid == 0) ts.n = 0;
  // candidates are taken every kNotes steps
  Seen seen = {-INFINITY, 0.0f, -INFINITY, f2pack(0.0f, 0.0f), f2pack(0.0f, 0.0f)};
  uint64_t above = 0;
  for (int first = 0; first < steps; first += kNotes) {
    const int end = min(steps, first + kNotes);
    seen = stream<ZT, TOP, ENT>(base, first, end, from, to, &ts.note[0][tid], b2, seen);
    if constexpr (TOP) {
      Top<ZT> alt = {ts, keys, reinterpret_cast<uint16_t*>(keys + q.cap), base, lo, from, to, q.K, q.cap, above};
      __syncthreads();
      if (first > 0) alt.cut(ts.n);
      alt.take(first, end - first, ts.n, seen.peak);
      above = alt.above;
    }
  }
  // the warps' sums; a thread that saw nothing but -inf and NaN has m = -inf, and S = 0 or NaN
  {
    const float m = seen.m, off = seen.off;
    float S = f2unpack(seen.s2).x + f2unpack(seen.s2).y, U = f2unpack(seen.u2).x + f2unpack(seen.u2).y;
    const float wm = warp_max(m);
    const float d = m == -INFINITY ? 0.0f : over(m, wm, b2) - off, c = ex2(d);
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
  int n = 0;
  if constexpr (TOP) n = keep_best(keys, ts.n, q.K);
  // sums of the warps or blocks, one to a lane: (M, S, U)
  auto join = [&](float M, float S, float U) {
    const float top = warp_max(M), d = M == -INFINITY ? 0.0f : over(M, top, b2), c = ex2(d);
    s_sum[1] = warp_sum(S * c);
    if constexpr (ENT) s_sum[2] = warp_sum(c > 0.0f ? c * fmaf(S, d, U) : c * 0.0f);
    s_sum[0] = top;
  };
  static_assert(kWarps <= 32, "");
  // the last warp joins the sums while the others write the alternatives
  if (warp == kWarps - 1) join(lane < kWarps ? s_m[lane] : -INFINITY, lane < kWarps ? s_s[lane] : 0.0f, lane < kWarps ? s_u[lane] : 0.0f);
  if (parts > 1) {
    if constexpr (TOP) {
      if (tid == 0) ts.n = n;
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (part == 0) {
      float v[3] = {-INFINITY, 0.0f, 0.0f};
      if (warp == kWarps - 1 && lane < parts)
        for (int i = 0; i < 3; ++i) v[i] = cluster.map_shared_rank(s_sum, lane)[i];
      if constexpr (TOP) {
        // a warp to a block's list
        static_assert(kWarps >= 7, "");
        const int r = warp + 1, listed = lane < parts ? *cluster.map_shared_rank(&ts.n, lane) : 0;
        int at = 0;
        n = 0;
        for (int i = 0; i < parts; ++i) {
          if (i == r) at = n;
          n += __shfl_sync(0xffffffffu, listed, i);
        }
        if (r < parts) {
          const uint64_t* theirs = cluster.map_shared_rank(keys, r);
          const int more = __shfl_sync(0xffffffffu, listed, r);
          for (int i = lane; i < more; i += 32) keys[at + i] = theirs[i];
        }
        n = keep_best(keys, n, q.K);
      }
      __syncwarp();
      if (warp == kWarps - 1) join(v[0], v[1], v[2]);
    }
    cluster.sync();  // the others' shared memory has been read
    if (part) return;
  }
  if (tid == kThreads - 32) {
    const float M = s_sum[0], s = s_sum[1];
    const bool empty = M == -INFINITY && s == 0.0f;
    const float l2 = log2f(s), ls = kLn2 * l2;
    if (q.lse) q.lse[row] = empty ? -INFINITY : M == -INFINITY ? s + NAN : fmaf(M, q.b, ls);
    if (ENT) q.entropy[row] = empty ? 0.0f : M == -INFINITY ? NAN : fmaxf(kLn2 * (l2 - s_sum[2] / s), 0.0f) + 0.0f * s;
    const int token = q.token ? s_token : -1;
    if (token >= q.V && q.err) atomicOr(q.err, QAD_DEV_BAD_INDEX);
    if (q.logp) {
      const bool live = token >= 0 && token < q.V;
      q.logp[row] = !live ? 0.0f : empty ? -INFINITY : M == -INFINITY ? NAN : over(s_zt, M, q.b) - ls;
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
  // blocks for a row: while all rows' blocks fit the SMs, each has a quarter of a step's logits at least, and their
  // candidates fit one block's list (one row of 151936: 8 blocks)
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
  // all but the target's own term
  auto grad = [&](float zv) {
    // of a row of 10^7 and more lse's rounding may leave a positive log p of any size: p is a probability all the same
    const float lp = clamp_nan(fmaf(zv, q.b, nlse), -1e4f, 0.0f);
    const float d = scale * ex2(lp * kLog2e) * fmaf(h, lp + H, g);
    return empty ? 0.0f : d;
  };
  // The target is written again, by the thread that has its vector, with the term of its own (asked for at every element:
  // 4096 x 151936 bf16 414 us against 388).  A masked logit is a constant, the target's too.
  const int at = token + from;
  const bool own = live && at / (kVec * kBwdThreads * kBwdVecs) == (int)seg && at / kVec % kBwdThreads == (int)threadIdx.x;
  const float zt = own ? read_one(z + token) : 0.0f;
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
      for (int j = 0; j < kVec; ++j) f[j] = grad(f[j]);
      uint4 o;
      if constexpr (sizeof(ZT) == 4)
        o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      else
        o = pack8(f);
      *reinterpret_cast<uint4*>(dz + v0) = o;
    } else {
      for (int j = 0; j < kVec; ++j)
        if (v0 + j >= 0 && v0 + j < q.V) write_one(dz + v0 + j, grad(read_one(z + v0 + j)));
    }
  }
  if (own) write_one(dz + token, zt == -INFINITY ? grad(zt) : grad(zt) + q.b * g);
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
