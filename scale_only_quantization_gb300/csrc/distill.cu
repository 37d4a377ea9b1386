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
#include "internal.h"
#include "tcgen05.cuh"

namespace qad {
namespace {

constexpr int kMaxStages = 16;  // ring of stages per team
constexpr int kSlots = 3;       // token rows a team holds: being prepared, streamed, and having its loss taken
constexpr size_t kMaxSmem = 220 * 1024;
constexpr float kMaxAbove = 40.0f;  // exp(40) squared and summed over 1024 slots stays within fp32

struct Distill {
  const __nv_bfloat16 *h, *w;
  const int32_t* idx;
  const float *t, *mix, *g;
  float* loss;
  __nv_bfloat16* dh;
  int32_t* err;
  int64_t ldh, ldw, V;
  int64_t stuck;     // a row whose copies are left out (the failure path's self-check), -1: none
  long long budget;  // clock cycles that a wait of the producers may take
  float beta;
  int K, d, accumulate;
};

// beta t of a slot: -inf says that the slot does not count, so a finite logit of the lowest values, whose product leaves
// fp32's range, stays finite (its probability is 0 all the same)
__device__ __forceinline__ float softened(float t, float beta) {
  const float b = t * beta;
  return b == -INFINITY && t != -INFINITY ? -3.402823466e38f : b;
}

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

// The divergence of one row (one warp) from beta * student logits z[K] and beta * teacher logits
// ts[K], -inf for a slot that does not count; every lane returns it.
__device__ __forceinline__ float row_divergence(const Distill& p, int64_t row, const float* z, const float* ts,
                                                int lane) {
  float mz = -INFINITY, mt = -INFINITY;
  for (int k = lane; k < p.K; k += 32) {
    mt = fmaxf(mt, ts[k]);
    if (ts[k] != -INFINITY) mz = fmaxf(mz, z[k]);
  }
  mz = warp_max(mz);
  mt = warp_max(mt);
  if (mt == -INFINITY) return 0.0f;  // no slot counts
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
  // a part without a share is left out: it may be infinite (RKL, where the teacher's logit is the lowest value)
  return (m != 1.0f ? (1.0f - m) * kl : 0.0f) + (m != 0.0f ? m * rkl : 0.0f);
}

// Sums of R values over the warp's 32 lanes (R a power of two): lane l returns the sum of value
// l >> (5 - log2 R).  Each step halves the values a lane carries, so R sums cost R - 1 + 5 - log2 R
// shuffles instead of 5 R.
template <int R>
__device__ __forceinline__ float reduce_many(float (&v)[R], int lane) {
  int off = 16;
#pragma unroll
  for (int n = R; n > 1; n /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float mine = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  float s = v[0];
#pragma unroll
  for (; off; off /= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// Teams of a block: as many warps as leave each thread the registers of its sums and of R head rows
// (168 with 12 warps or fewer).
template <int CW, int V> __host__ __device__ constexpr int teams_of() {
  return CW >= 8 ? 1 : V == 1 ? 8 : CW == 1 ? 5 : 8 / CW;
}

// Two bf16 as fp32.  The two uses of a head row unpack it by different instructions, shifts here and
// byte moves in unpack_again: with the same ones the compiler keeps the unpacked values in between,
// twice the registers, and spills.
__device__ __forceinline__ uint64_t unpack_once(uint32_t v) { return f2pack(bf16lo(v), bf16hi(v)); }
__device__ __forceinline__ uint64_t unpack_again(uint32_t v) {
  return f2pack(__uint_as_float(__byte_perm(v, 0, 0x1044)), __uint_as_float(__byte_perm(v, 0, 0x3244)));
}

// 16 bytes of read-only memory without an L1 line
__device__ __forceinline__ uint4 ld_nc(const uint4* ptr) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(ptr));
  return v;
}

// loss and dh of every step-th row from first on (one warp): a pipeline wait of their block ran out
__device__ __forceinline__ void make_nan(const Distill& p, int64_t first, int64_t step, int64_t N, int lane) {
  const uint32_t nans = 0x7fff7fffu;
  for (int64_t row = first; row < N; row += step) {
    if (lane == 0) p.loss[row] = NAN;
    for (int c = lane; c < p.d / 8; c += 32)
      reinterpret_cast<uint4*>(p.dh + row * p.d)[c] = make_uint4(nans, nans, nans, nans);
  }
}

struct DistillGrid {
  int stages, teams;  // ring depth, teams per block
};

// Every head row is read once.  The gradient
//   dh = beta g ((1 - m - m sbar) A0 / S + m A1 / S - (1 - m) B),
//   A0 = sum e_k w_k, A1 = sum e_k s_k w_k, B = sum p_k w_k, e_k = exp(beta z_k - M), S = sum e_k,
//   s_k = beta (z_k - t_k) up to a constant of the row, sbar = sum e_k s_k / S
// is accumulated in fp32 while the rows stream past (x_k - RKL = s_k - sbar).  M is the first batch's
// largest logit, replaced (and the sums scaled) only by one more than kMaxAbove nats higher: e may
// exceed 1.
//
// A team of CW consumer warps takes a token row: lane l of warp w owns V 16-byte vectors of the columns,
// 32 CW apart.  A producer warp per team runs ahead: it makes the teacher's probabilities of a row,
// brings its head rows, R at a time, into a ring of shared memory (one bulk copy per row) and, when a
// row is through, takes its loss from the logits that the consumers left.  Per stage the consumers take
// the R rows into registers and free the stage, join their dot products (one shuffle reduction for all
// R, one named barrier of the team, none for CW = 1) and add the weighted rows to their sums.  When a wait runs
// out the producers arm no stage any more, the copies under way land, and the block's producers make the losses and dh of
// all its rows NaN: the sign where the caller gave no error word.
//
// What bounds it: the gathered rows come from HBM (a head of 152k rows does not stay in L2), and a stage is
// a chain of some 2000 cycles of waits, reductions and exponentials, so that the bytes that the SM's
// registers hold at once set the rate: two teams of 4 warps with 8 rows each (64 KB) reach 6.0 TB/s of
// head rows at d = 2048, K = 64 (178 to 182 us for 4096 token rows); batches of 4 rows 206 us, 8-warp teams with
// half the columns per lane 206 us.  One team of 8 warps takes d = 4096; with both divergences its third
// sum leaves it at 4.4 TB/s (967 to 976 us for 16384 token rows, K = 32; 746 us without it).  Two teams on an SM
// there, with batches of 4 rows or 2 that are read a second time from shared memory instead of held in registers,
// spill and hold each stage for its whole chain: 1670 to 2400 us.  Reading the rows a second time from L2
// for the gradient instead took 305 and 1240 us; matrix instructions (mma.sync, 8 rows a fragment) for both
// products 234 and 1358 us, their rate on this chip being a few times the FMA units' only.  Wider rows take one team of
// 16 warps with batches of 2 head rows, or of 1: 4096 token rows of d = 8192, K = 32 515 us (4.2 TB/s), mixed 880;
// 2048 of d = 16384 1455 us (1.5 TB/s), mixed 3020, where the sums spill (0.5 and 1.6 KB).
template <int CW, int V, int R, bool MIX>
__global__ void __launch_bounds__(32 * (teams_of<CW, V>() * (CW + 1)), 1)
    distill_kernel(const Distill p, const DistillGrid q, const int64_t N) {
  constexpr int TEAMS = teams_of<CW, V>();
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(8) uint64_t bars[TEAMS][2 * kMaxStages + 2 * kSlots];
  __shared__ float part[TEAMS][2][CW][R];
  __shared__ int abort_flag, late;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool producer = warp >= q.teams * CW;
  const int team = producer ? warp - q.teams * CW : warp / CW, wt = warp % CW;
  const int K = p.K, KP = (K + 3) / 4 * 4, nv = p.d / 8, stages = q.stages;
  uint8_t* base = sm + (size_t)team * ((size_t)stages * R * p.d * 2 + (size_t)(3 * kSlots + 1) * KP * 4);
  const uint4* ring = reinterpret_cast<const uint4*>(base);
  float* arr = reinterpret_cast<float*>(base + (size_t)stages * R * p.d * 2);
  auto ts = [&](int s) { return arr + (3 * s) * KP; };      // beta t, -inf: does not count
  auto pk = [&](int s) { return arr + (3 * s + 1) * KP; };  // the teacher's probabilities
  auto zz = [&](int s) { return arr + (3 * s + 2) * KP; };  // beta z
  int32_t* tok = reinterpret_cast<int32_t*>(arr + 3 * kSlots * KP);
  const uint32_t bar0 = smem_u32(bars[team]);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto done = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
  auto arrive = [&](uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
  };
  if (threadIdx.x == 0) abort_flag = late = 0;
  if (producer && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), CW);
    }
    for (int s = 0; s < kSlots; ++s) mbar_init(done(s), CW);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  int32_t* err = p.err ? p.err : &late;
  const int64_t first = (int64_t)blockIdx.x * q.teams + team, step = (int64_t)gridDim.x * q.teams;
  const int groups = (K + R - 1) / R;

  if (producer) {
    int stage = 0, slot = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    constexpr int PF = 4;  // slots per lane whose token and logit are fetched a row ahead
    int32_t next_v[PF];
    float next_t[PF];
    auto fetch = [&](int64_t row) {
#pragma unroll
      for (int j = 0; j < PF; ++j) {
        const int k = lane + 32 * j;
        const bool in = k < K && row < N;
        next_v[j] = in ? __ldg(p.idx + row * K + k) : -1;
        next_t[j] = in ? __ldg(p.t + row * K + k) : 0.0f;
      }
    };
    int64_t i = 0;
    auto finish = [&](int64_t j) {  // the loss of this team's j-th row, once its consumers are through
      const int s = (int)(j % kSlots);
      const bool got = __all_sync(0xffffffffu, mbar_wait(done(s), (uint32_t)(j / kSlots) & 1u, &abort_flag, err, p.budget));
      if (got) {
        const float l = row_divergence(p, first + j * step, zz(s), ts(s), lane);
        if (lane == 0) p.loss[first + j * step] = l;
        __syncwarp();
      }
      return got;
    };
    fetch(first);
    for (int64_t row = first; ok && row < N; row += step, ++i) {
      if (i >= kSlots) ok = finish(i - kSlots);
      if (!ok) break;
      float mt = -INFINITY;
      auto take = [&](int k, int32_t v, float t) {
        t = softened(t, p.beta);
        if (v >= p.V) {
          if (p.err) atomicOr(p.err, QAD_DEV_BAD_INDEX);
          v = -1;
        }
        if (t == -INFINITY) v = -1;
        if (v < 0) t = -INFINITY;
        mt = fmaxf(mt, t);
        tok[k] = v;
        ts(slot)[k] = t;
      };
#pragma unroll
      for (int j = 0; j < PF; ++j)
        if (lane + 32 * j < K) take(lane + 32 * j, next_v[j], next_t[j]);
      for (int k = lane + 32 * PF; k < K; k += 32) take(k, __ldg(p.idx + row * K + k), __ldg(p.t + row * K + k));
      fetch(row + step);
      mt = warp_max(mt);
      float st = 0.0f;
      for (int k = lane; k < K; k += 32) {
        const float t = ts(slot)[k];
        const float e = t == -INFINITY ? 0.0f : expf(t - mt);
        pk(slot)[k] = e;
        st += e;
      }
      st = warp_sum(st);
      const float rt = st == 0.0f ? 0.0f : 1.0f / st;  // a row that keeps no slot
      for (int k = lane; k < K; k += 32) pk(slot)[k] *= rt;
      __syncwarp();
      for (int b = 0; b < groups; ++b) {
        // a consumer whose wait ran out has raised the flag before it freed the stage: no stage is armed after that
        ok = __all_sync(0xffffffffu, mbar_wait(empty(stage), phase ^ 1u, &abort_flag, err, p.budget) &&
                                         !*static_cast<volatile int*>(&abort_flag));
        if (!ok) break;
        const int k = b * R + lane;
        const int32_t v = lane < R && k < K ? tok[k] : -1;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, v >= 0)), bytes = (uint32_t)nv * 16u;
        const bool stuck = row == p.stuck;
        if (lane == 0 && !stuck) mbar_expect_tx(full(stage), n * bytes);
        __syncwarp();
        if (v >= 0 && !stuck)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  smem_u32(ring + (size_t)(stage * R + lane) * nv)),
              "l"(reinterpret_cast<uint64_t>(p.w + (int64_t)v * p.ldw)), "r"(bytes), "r"(full(stage))
              : "memory");
        if (!stuck) armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (++slot == kSlots) slot = 0;
    }
    for (int64_t j = i > kSlots ? i - kSlots : 0; ok && j < i; ++j) ok = finish(j);
    if (*static_cast<volatile int*>(&abort_flag)) {
      volatile int none = 0;  // copies may be under way: they land (bounded wait) before shared memory is given back
      for (int s = 0; s < stages; ++s)
        if (armed & (1u << s)) mbar_wait(full(s), (armed_parity >> s) & 1u, &none, &late);
    }
    __syncthreads();  // the consumers' stores are over
    if (abort_flag) make_nan(p, first, step, N, lane);
    return;
  }

  int stage = 0, flip = 0, slot = 0;
  uint32_t phase = 0;
  for (int64_t row = first; row < N; row += step) {
    uint4 hv[V];
    uint64_t a0[V][4], a1[MIX ? V : 1][4], bb[V][4];
    const uint4* hr = reinterpret_cast<const uint4*>(p.h + row * p.ldh);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = wt * 32 + lane + j * 32 * CW;
      hv[j] = c < nv ? __ldg(hr + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a0[j][i] = bb[j][i] = f2pack(0.0f, 0.0f);
        if constexpr (MIX) a1[j][i] = f2pack(0.0f, 0.0f);
      }
    }
    float M = 0.0f, S = 0.0f, S1 = 0.0f, soff = 0.0f;
    bool some = false;
    for (int b = 0; b < groups; ++b) {
      // a wait that ran out leaves the error bit and wrong values, replaced below; the team's barriers stay in step
      mbar_wait(full(stage), phase, &abort_flag, err);
      __syncwarp();
      const int k = b * R + (lane & (R - 1));  // this lane's head row of the stage
      const float t = k < K ? ts(slot)[k] : -INFINITY;
      const bool live = t != -INFINITY;
      const uint32_t valid = __ballot_sync(0xffffffffu, live) & ((1u << R) - 1u);
      const uint4* w0 = ring + (size_t)stage * R * nv + wt * 32 + lane;
      uint4 w[R][V];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < V; ++j)  // a row that does not count is not read: its memory may hold anything
          w[r][j] = wt * 32 + lane + j * 32 * CW < nv && (valid >> r & 1u) ? w0[r * nv + j * 32 * CW]
                                                                           : make_uint4(0, 0, 0, 0);
      uint64_t d2[R];
#pragma unroll
      for (int r = 0; r < R; ++r) d2[r] = f2pack(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t y[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w};
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t x[4] = {w[r][j].x, w[r][j].y, w[r][j].z, w[r][j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d2[r] = f2fma(unpack_once(x[i]), unpack_once(y[i]), d2[r]);
        }
      }
      __syncwarp();
      if (lane == 0) arrive(empty(stage));
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
      float dot[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 d = f2unpack(d2[r]);
        dot[r] = d.x + d.y;
      }
      const float mine = reduce_many<R>(dot, lane);
      constexpr int PER = 32 / R;  // lanes that hold the same sum
      float z;
      if constexpr (CW > 1) {
        if (lane % PER == 0) part[team][flip][wt][lane / PER] = mine;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * CW) : "memory");
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < CW; ++i) z += part[team][flip][i][lane & (R - 1)];
        flip ^= 1;  // the next stage's partial sums go elsewhere: a slower warp may still read these
      } else {
        z = __shfl_sync(0xffffffffu, mine, (lane & (R - 1)) * PER);
      }
      z *= p.beta;
      if (wt == 0 && lane < R && k < K) zz(slot)[k] = z;
      if (valid) {  // alike in the whole team
        const bool jump = live && z > M + kMaxAbove;
        if (!some || __any_sync(0xffffffffu, jump)) {
          float top = live ? z : -INFINITY;
#pragma unroll
          for (int o = R / 2; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (some) {
            const float f = __expf(M - top);
            const uint64_t f2 = f2pack(f, f);
            S *= f;
            S1 *= f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a0[j][i] = f2mul(a0[j][i], f2);
                if constexpr (MIX) a1[j][i] = f2mul(a1[j][i], f2);
              }
          } else if constexpr (MIX) {
            soff = __shfl_sync(0xffffffffu, z - t, __ffs(valid) - 1);
          }
          M = top;
          some = true;
        }
        const float e = live ? __expf(z - M) : 0.0f, pr = live ? pk(slot)[k] : 0.0f;
        const float es = MIX && live ? e * (z - t - soff) : 0.0f;
        S += e;  // of this lane's head rows: joined when the token row is through
        S1 += es;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float er = __shfl_sync(0xffffffffu, e, r), qr = __shfl_sync(0xffffffffu, pr, r);
          const float sr = MIX ? __shfl_sync(0xffffffffu, es, r) : 0.0f;
          const uint64_t e2 = f2pack(er, er), p2 = f2pack(qr, qr), es2 = f2pack(sr, sr);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const uint32_t x[4] = {w[r][j].x, w[r][j].y, w[r][j].z, w[r][j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t w2 = unpack_again(x[i]);
              a0[j][i] = f2fma(e2, w2, a0[j][i]);
              bb[j][i] = f2fma(p2, w2, bb[j][i]);
              if constexpr (MIX) a1[j][i] = f2fma(es2, w2, a1[j][i]);
            }
          }
        }
      }
    }
    __syncwarp();  // the whole warp's reads and writes of the slot are over
    if (lane == 0) arrive(done(slot));
    if (++slot == kSlots) slot = 0;
#pragma unroll
    for (int o = R / 2; o; o /= 2) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      if constexpr (MIX) S1 += __shfl_xor_sync(0xffffffffu, S1, o);
    }
    const float scale = p.beta * (p.g ? __ldg(p.g + row) : 1.0f);
    const float m = MIX ? __ldg(p.mix + row) : 0.0f;
    const float rs = some ? scale / S : 0.0f;
    const bool reverse = MIX && some && m != 0.0f;  // else its sums are left out: they may be infinite
    const float ka = ((1.0f - m) - (reverse ? m * (S1 / S) : 0.0f)) * rs, k1 = m * rs, kb = -(1.0f - m) * scale;
    uint4* out = reinterpret_cast<uint4*>(p.dh + row * p.d);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = wt * 32 + lane + j * 32 * CW;
      if (c >= nv) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = f2unpack(a0[j][i]), y = f2unpack(bb[j][i]);
        v[2 * i] = ka * x.x + kb * y.x;
        v[2 * i + 1] = ka * x.y + kb * y.y;
        if constexpr (MIX) {
          const float2 u = f2unpack(a1[j][i]);
          if (reverse) {
            v[2 * i] += k1 * u.x;
            v[2 * i + 1] += k1 * u.y;
          }
        }
      }
      if (p.accumulate) {
        float o[8];
        unpack8(out[c], o);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += o[i];
      }
      out[c] = pack8(v);
    }
  }
  __syncthreads();  // with the producers
}

// As many teams as a block holds, with the deepest ring; fewer teams where the rows' arrays (many kept
// logits) leave each less than three stages.
template <int CW, int V, int R, bool MIX>
cudaError_t launch_one(const Distill& p, int64_t N, cudaStream_t st) {
  auto kern = distill_kernel<CW, V, R, MIX>;
  static bool ready[64] = {false};  // per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!ready[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  auto bytes = [&](int stages) {
    return (size_t)stages * R * p.d * 2 + (size_t)(3 * kSlots + 1) * ((p.K + 3) / 4 * 4) * 4;
  };
  DistillGrid q;
  q.teams = teams_of<CW, V>();
  while (q.teams > 1 && q.teams * bytes(3) > kMaxSmem) --q.teams;
  q.stages = kMaxStages;
  while (q.stages > 2 && q.teams * bytes(q.stages) > kMaxSmem) --q.stages;
  const size_t smem = q.teams * bytes(q.stages);
  if (smem > kMaxSmem) return cudaErrorInvalidValue;
  const int64_t fill = num_sms(), need = (N + q.teams - 1) / q.teams;
  kern<<<(unsigned)(need < fill ? need : fill), 32 * (CW + 1) * q.teams, smem, st>>>(p, q, N);
  return cudaGetLastError();
}

// The loss alone: one block per row, one warp per head row, 8 vectors of it in flight per lane; no stage,
// no barrier until the logits are there.  The partial sums are those of the teams above, in their order,
// so that the loss has the same bits: warp i's vectors are i * 32 + lane + 32 CW j.
template <int CW, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) distill_fwd_kernel(const Distill p) {
  extern __shared__ __align__(128) uint8_t sm[];
  const int nv = p.d / 8, K = p.K;
  uint4* hs = reinterpret_cast<uint4*>(sm);
  float* z = reinterpret_cast<float*>(hs + nv);
  float* ts = z + K;
  int32_t* tok = reinterpret_cast<int32_t*>(ts + K);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const uint4* hr = reinterpret_cast<const uint4*>(p.h + row * p.ldh);
  for (int c = tid; c < nv; c += THREADS) hs[c] = __ldg(hr + c);
  for (int k = tid; k < K; k += THREADS) {
    int32_t v = __ldg(p.idx + row * K + k);
    float t = softened(__ldg(p.t + row * K + k), p.beta);
    if (v >= p.V) {
      if (p.err) atomicOr(p.err, QAD_DEV_BAD_INDEX);
      v = -1;
    }
    if (t == -INFINITY) v = -1;
    if (v < 0) t = -INFINITY;
    tok[k] = v;
    ts[k] = t;
  }
  __syncthreads();
  for (int k = warp; k < K; k += THREADS / 32) {
    const int32_t v = tok[k];
    if (v < 0) continue;
    const uint4* wr = reinterpret_cast<const uint4*>(p.w + (int64_t)v * p.ldw);
    float dot[CW];
    constexpr int STEP = CW * V <= 8 ? CW : 8 / V;  // team warps whose vectors are loaded together
#pragma unroll
    for (int i0 = 0; i0 < CW; i0 += STEP) {
      uint4 u[STEP][V];
#pragma unroll
      for (int i = 0; i < STEP; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (i0 + i) * 32 + lane + 32 * CW * j;
          u[i][j] = c < nv ? ld_nc(wr + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int i = 0; i < STEP; ++i) {
        uint64_t d2 = f2pack(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (i0 + i) * 32 + lane + 32 * CW * j;
          const uint4 hv = c < nv ? hs[c] : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {u[i][j].x, u[i][j].y, u[i][j].z, u[i][j].w}, y[4] = {hv.x, hv.y, hv.z, hv.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) d2 = f2fma(unpack_once(x[q]), unpack_once(y[q]), d2);
        }
        const float2 d = f2unpack(d2);
        dot[i0 + i] = d.x + d.y;
      }
    }
    const float mine = reduce_many<CW>(dot, lane);
    float s = CW > 1 ? 0.0f : mine;
    if constexpr (CW > 1)
#pragma unroll
      for (int i = 0; i < CW; ++i) s += __shfl_sync(0xffffffffu, mine, i * (32 / CW));
    if (lane == 0) z[k] = s * p.beta;
  }
  __syncthreads();
  if (warp == 0) {
    const float l = row_divergence(p, row, z, ts, lane);
    if (lane == 0) p.loss[row] = l;
  }
}

template <int CW, int V, int R>
cudaError_t launch_team(const Distill& p, int64_t N, cudaStream_t st) {
  if (p.dh) return p.mix ? launch_one<CW, V, R, true>(p, N, st) : launch_one<CW, V, R, false>(p, N, st);
  const size_t smem = (size_t)p.d * 2 + (size_t)p.K * 12;
  // rows that do not fill the SMs: 32 warps share a row's head rows instead of 4 (64 rows of K = 64, d = 2048: 10 us;
  // one of K = 128, d = 4096: 19 us, with 4 warps 39); with more rows small blocks cover each other's ends better
  // (1000 rows of K = 100, d = 2880: 87 us with 4 warps, 96 with 16)
  if (N <= num_sms() && p.K > 4) distill_fwd_kernel<CW, V, 1024><<<(unsigned)N, 1024, smem, st>>>(p);
  else distill_fwd_kernel<CW, V, 128><<<(unsigned)N, 128, smem, st>>>(p);
  return cudaGetLastError();
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
  const StuckCopy stuck = stuck_copy();
  p.stuck = stuck.row;
  p.budget = stuck.row < 0 ? kWaitCycles : stuck.budget;
  // a team as wide as the row needs, each lane with 16 of its columns and their three sums
  prof_begin(QAD_K_DISTILL, st);
  cudaError_t e;
  if (d <= 256) e = launch_team<1, 1, 8>(p, N, st);
  else if (d <= 512) e = launch_team<1, 2, 8>(p, N, st);
  else if (d <= 1024) e = launch_team<2, 2, 8>(p, N, st);
  else if (d <= 2048) e = launch_team<4, 2, 8>(p, N, st);
  else if (d <= 4096) e = launch_team<8, 2, 8>(p, N, st);
  else if (d <= 8192) e = launch_team<16, 2, 2>(p, N, st);
  else e = launch_team<16, 4, 1>(p, N, st);
  prof_end(QAD_K_DISTILL, st);
  return e;
}

}  // namespace qad
