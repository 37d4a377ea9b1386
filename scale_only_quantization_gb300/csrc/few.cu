// The whole expert layer for a few tokens (generation), in one cooperative launch that reads the weights of the experts
// that some token names (once for each 8 tokens of an expert), fake-quantizes them on their way and multiplies them there.
//
//   fc1:  Z1 = A1 . W13_hat^T, H = bf16(silu(gate) * up)             A1 = AQ(x)
//   fc2:  Y = AQ(H) . W2_hat^T, out[t] = bf16(sum_j p[t, j] * Y_j)
//
// With so few rows the weights are all there is to move (2 bytes an element and its part of a scale), and each element
// costs about nine instructions of fake-quantization whatever the number of tokens: for many experts instructions bound
// the kernel as much as memory does, for a single token latency does.  A warp copies 64 weights of 16 rows ahead into its
// ring in shared memory; a lane quantizes 16 of a row (one quantization block) in registers in the tensor cores' fragment
// layout, and four m16n8k16 products take them as they lie.  The order of k inside a product does not matter as long as
// both operands agree, so the tokens' rows (shared memory, up to 8 columns) are read in the same order.  A warp reads only
// what it copied itself: the ring needs no block barrier.  tcgen05 would want the quantized weights in shared memory: a
// write and a read of every element for products that are idle most of the time here.  One block of 24 warps per SM: with
// 16 in two blocks the quantizers' latencies were not hidden (32 tokens 358 against 302 us).
//
// One nvfp4 token naming 8 of 128 experts of 2048 x 768 (85 MB): 39 us, 5.5 of them clearing and launch; 32 w4a16 tokens naming
// 111 of them 292 to 300 us, 3.6 TB/s; 5 fp8 tokens on 32 experts of 2880 x 2880 161 to 177 us, by how
// many experts they name.  8 nvfp4 tokens on 64 experts issue 13 instructions a weight at 2.5 a cycle.
//
// Between fc1 and fc2 the blocks wait for one another; their first weights of fc2 are on their way by then.
#include "common.cuh"
#include "internal.h"

namespace qad {
namespace {

constexpr int kThreads = 768, kWarps = kThreads / 32;
constexpr int kCols = 8;     // tokens of one expert that a pass over its weights serves, at most
constexpr int kMaxTeam = 8;  // warps that share a tile
constexpr int kChunk = 64;   // elements along K of one step: 16 for each lane of a quad
constexpr int kPitch = 2 * kChunk + 16;   // bytes between the rows of a chunk: 16-byte reads of 8 lanes meet no bank twice
constexpr int kSlot = 16 * kPitch + 256;  // bytes of a warp's chunk: 16 rows of weights, up to 4 scales a row
constexpr long long kWaitCycles = 4000000000ll;  // after which a block gives up on the others (two seconds)

struct Half {                  // fc1 or fc2
  const __nv_bfloat16* act;    // x [T, K], or H [T * k, K]
  const __nv_bfloat16* w;      // [E, rows, K], rows = 2N (fc1) or N (fc2)
  const float* s;
  __nv_bfloat16* rows;         // [T * k, N]: H, or Y
  int K, N, scales;            // scales: per weight row
  int chunks, team, per_warp;  // of a tile along K; warps that share a tile; chunks for each of them
  int tiles;                   // of an expert: fc1 8 gate rows and the 8 up rows that go with them, fc2 16 rows
  int64_t up, sup;             // from a tile's first 8 rows to the others: weights, scales
  bool ragged;                 // K ends inside a chunk
};

struct FewParams {
  Half fc1, fc2;
  const int32_t* idx;
  const float* p;
  __nv_bfloat16* out;
  int32_t* err;
  uint32_t* arrived;   // blocks that are through with fc1 (0 before)
  uint32_t* arrivals;  // [d / 16]: passes that have written a tile of Y (0 before)
  int T, k, E;
  int cols, depth;     // token rows of a pass; chunks of a warp in its ring: the one worked on and 1 or 2 on their way
};

__host__ __device__ constexpr int few_stride(int K) { return (K + kChunk - 1) / kChunk * kChunk * 2 + 16; }

// Dynamic shared memory: the warps' rings, the staged token rows, the masks and first passes of E experts.
__host__ __device__ constexpr int few_rows_at(int depth) { return kWarps * depth * kSlot; }
__host__ __device__ constexpr int few_mask_at(int K, int cols, int depth) { return few_rows_at(depth) + cols * few_stride(K); }
__host__ __device__ constexpr int few_smem(int K, int cols, int E, int depth) {
  return few_mask_at(K, cols, depth) + 8 * E + 2 * (E + 1) + 6;
}

// The pairs by expert, found by every block for itself.  A pass serves up to `cols` tokens of one expert.
// Up to 32 pairs and a pass for each expert: a pair to a lane, in every warp alike and without a barrier; the passes stand
// in the order of their experts' first pairs.  Else by masks in shared memory, the passes in the order of the experts.
struct Route {
  bool small;
  int passes;
  // small: this lane's pair
  int expert;
  uint32_t group, leaders, valid;  // the pairs of its expert; the first pair of each expert; the pairs that count
  // else
  uint64_t* mask;   // [E]: the tokens that name the expert
  uint32_t* live;   // [T]: the slots of a token that count
  uint16_t* first;  // [E + 1]: the expert's first pass
  int E, k, cols;

  __device__ __forceinline__ uint32_t below() const { return (1u << (threadIdx.x & 31)) - 1; }
  __device__ __forceinline__ int leader_of(int pass) const {  // its lane
    const bool mine = (group & below()) == 0 && group && __popc(leaders & below()) == pass;
    return __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  }
  // all lanes of a warp together
  __device__ __forceinline__ int expert_of(int pass) const {
    if (small) return __shfl_sync(0xffffffffu, expert, leader_of(pass));
    int e = 0;  // the last expert whose first pass is not behind this one
    for (int b = 512; b; b >>= 1)
      if (e + b < E && first[e + b] <= pass) e += b;
    return e;
  }
  // the pair (t * k + j) of lane's column of the pass, or -1: all lanes of a warp together
  __device__ __forceinline__ int pair_of(int pass, int e, const int32_t* idx) const {
    const int lane = threadIdx.x & 31;
    if (small) {
      uint32_t m = __shfl_sync(0xffffffffu, group, leader_of(pass));
      for (int i = lane; i > 0 && m; --i) m &= m - 1;
      return m ? __ffs(m) - 1 : -1;
    }
    uint64_t m = mask[e];
    for (int i = (pass - first[e]) * cols + lane; i > 0 && m; --i) m &= m - 1;
    int pair = -1;
    if (m && lane < cols) {
      const int t = __ffsll((long long)m) - 1;
      for (int j = 0; j < k; ++j)
        if ((live[t] >> j & 1) && __ldg(idx + t * k + j) == e) pair = t * k + j;
    }
    return pair;
  }
  __device__ __forceinline__ uint32_t slots_of(int t) const {
    return small ? valid >> (t * k) & (k == 32 ? 0xffffffffu : (1u << k) - 1) : live[t];
  }
};

__device__ __forceinline__ Route route(const FewParams& q, uint64_t* mask, uint16_t* first, uint32_t* live, int* err) {
  const int tid = threadIdx.x, lane = tid & 31, pairs = q.T * q.k;
  Route r;
  r.mask = mask;
  r.live = live;
  r.first = first;
  r.E = q.E;
  r.k = q.k;
  r.cols = q.cols;
  r.small = pairs <= 32 && q.T <= q.cols;
  if (r.small) {
    const int e = lane < pairs ? __ldg(q.idx + lane) : -1;
    const bool in = e >= 0 && e < q.E;
    const uint32_t same = __match_any_sync(0xffffffffu, in ? e : -1 - lane);
    const uint32_t earlier = r.below() & ~((1u << (lane < pairs ? lane / q.k * q.k : 0)) - 1);  // slots of this token
    const bool again = in && (same & earlier);
    r.valid = __ballot_sync(0xffffffffu, in && !again);
    r.expert = e;
    r.group = in && !again ? same & r.valid : 0;
    r.leaders = __ballot_sync(0xffffffffu, r.group && !(r.group & r.below()));
    r.passes = __popc(r.leaders);
    *err = (__any_sync(0xffffffffu, lane < pairs && !in) ? QAD_DEV_BAD_INDEX : 0) |
           (__any_sync(0xffffffffu, again) ? QAD_DEV_DUP_INDEX : 0);
    return r;
  }
  for (int e = tid; e < q.E; e += kThreads) mask[e] = 0;
  for (int t = tid; t < q.T; t += kThreads) live[t] = 0;
  __syncthreads();
  int bad = 0;
  for (int i = tid; i < pairs; i += kThreads) {
    const int t = i / q.k, j = i % q.k, e = __ldg(q.idx + i);
    if (e < 0 || e >= q.E) {
      bad |= QAD_DEV_BAD_INDEX;
      continue;
    }
    bool again = false;
    for (int jj = 0; jj < j; ++jj) again |= __ldg(q.idx + t * q.k + jj) == e;
    if (again) {
      bad |= QAD_DEV_DUP_INDEX;
      continue;
    }
    atomicOr(reinterpret_cast<unsigned long long*>(mask + e), 1ull << t);
    atomicOr(live + t, 1u << j);
  }
  *err = (__syncthreads_or(bad & QAD_DEV_BAD_INDEX) ? QAD_DEV_BAD_INDEX : 0) |
         (__syncthreads_or(bad & QAD_DEV_DUP_INDEX) ? QAD_DEV_DUP_INDEX : 0);
  if (tid < 32) {
    const int per = (q.E + 31) / 32, lo = min(q.E, tid * per), hi = min(q.E, lo + per);
    int n = 0;
    for (int e = lo; e < hi; ++e) n += (__popcll(mask[e]) + q.cols - 1) / q.cols;
    int at = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (tid >= o) at += v;
    }
    at -= n;
    for (int e = lo; e < hi; ++e) {
      first[e] = (uint16_t)at;
      at += (__popcll(mask[e]) + q.cols - 1) / q.cols;
    }
    if (tid == 31) first[q.E] = (uint16_t)at;
  }
  __syncthreads();
  r.passes = first[q.E];
  return r;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

struct Block16 {
  uint32_t v[8];
};
__device__ __forceinline__ Block16 read16(const uint32_t* place) {
  const uint4 lo = reinterpret_cast<const uint4*>(place)[0], hi = reinterpret_cast<const uint4*>(place)[1];
  return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}

// W_hat of 16 weights that share scale s, the bits of fakequant16_packed (see there for the quotient).  What follows the
// quotient x = fp32(w / s) takes fewer instructions here:
//  - E2M1: bf16(fp32(q s)) takes eight magnitudes, which the 3-bit codes of four weights look up by two byte permutations.
//    Four of them are halves or doubles of bf16(s) and bf16(1.5 s), that is their bits with the exponent moved;
//  - INT4, INT8: bf16(fp32(q s)) does not fall as q rises, so that clamping q is clamping it, two at a time.
// `odd` stays 0 while the scale is in [2^-60, 2^16) and no quotient is inf or NaN; else quantize_pairs has to do it.
template <int WK>
__device__ __forceinline__ Block16 quantize16(const Block16& w, float s, uint32_t* odd) {
  if constexpr (WK == kQNone) {
    return w;
  } else {
    Block16 out;
    const float r = __frcp_rn(s);
    const uint64_t r2 = f2pack(r, r), ns2 = f2pack(-s, -s), zero2 = f2pack(0.0f, 0.0f);
    uint64_t probe = zero2;
    auto quotient2 = [&](uint32_t v) {
      const uint64_t w2 = f2pack(bf16lo(v), bf16hi(v));
      const uint64_t q2 = f2mul(w2, r2), x2 = f2fma(f2fma(q2, ns2, w2), r2, q2);
      probe = f2fma(x2, zero2, probe);  // stays 0 unless a quotient is inf or NaN
      return x2;
    };
    if constexpr (WK == kQE2M1) {
      const uint32_t m23 = pack_bf16(s, __fmul_rn(1.5f, s));
      const uint32_t m01 = (m23 << 16) - 0x00800000u, m45 = m23 + 0x00800080u, m67 = m23 + 0x01000100u;
      const uint32_t lo03 = __byte_perm(m01, m23, 0x6420), lo47 = __byte_perm(m45, m67, 0x6420);
      const uint32_t hi03 = __byte_perm(m01, m23, 0x7531), hi47 = __byte_perm(m45, m67, 0x7531);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float2 a = f2unpack(quotient2(w.v[i])), b = f2unpack(quotient2(w.v[i + 1]));
        const float2 c = f2unpack(quotient2(w.v[i + 2])), d = f2unpack(quotient2(w.v[i + 3]));
        uint32_t codes;
        asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
            "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
            : "=r"(codes)
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
        codes &= 0x77777777u;
        const uint32_t up = codes >> 16;
        const uint32_t l0 = __byte_perm(lo03, lo47, codes), h0 = __byte_perm(hi03, hi47, codes);
        const uint32_t l1 = __byte_perm(lo03, lo47, up), h1 = __byte_perm(hi03, hi47, up);
        out.v[i] = __byte_perm(l0, h0, 0x5140) | (w.v[i] & 0x80008000u);
        out.v[i + 1] = __byte_perm(l0, h0, 0x7362) | (w.v[i + 1] & 0x80008000u);
        out.v[i + 2] = __byte_perm(l1, h1, 0x5140) | (w.v[i + 2] & 0x80008000u);
        out.v[i + 3] = __byte_perm(l1, h1, 0x7362) | (w.v[i + 3] & 0x80008000u);
      }
    } else if constexpr (WK == kQE4M3) {
      const float sc = s * 0x1p112f;
      const uint64_t sc2 = f2pack(sc, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = f2unpack(quotient2(w.v[i]));
        uint16_t c;
        uint32_t h2;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(x.x), "f"(x.y));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
        const uint32_t la = (h2 << 13) & 0x0FFFE000u, lb = (h2 >> 3) & 0x0FFFE000u;
        const float2 m = f2unpack(f2mul(f2pack(__uint_as_float(la), __uint_as_float(lb)), sc2));
        out.v[i] = pack_bf16(m.x, m.y) | (w.v[i] & 0x80008000u);
      }
    } else {
      const uint64_t big2 = f2pack(12582912.0f, 12582912.0f), s2 = f2pack(s, s);  // 1.5 * 2^23
      const float lo = __fmul_rn(Clip<WK>::lo, s), hi = __fmul_rn(Clip<WK>::hi, s);
      const uint32_t lo2 = pack_bf16(lo, lo), hi2 = pack_bf16(hi, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 m = f2unpack(f2mul(f2sub(f2add(quotient2(w.v[i]), big2), big2), s2));
        uint32_t v = pack_bf16(m.x, m.y);
        asm("max.bf16x2 %0, %0, %1;\n\tmin.bf16x2 %0, %0, %2;" : "+r"(v) : "r"(lo2), "r"(hi2));
        out.v[i] = v | (w.v[i] & 0x80008000u);
      }
    }
    const float2 p = f2unpack(probe);
    *odd |= (__float_as_uint(p.x + p.y) << 1) | (__float_as_uint(s) - 0x21800000u >= 0x47800000u - 0x21800000u);
    return out;
  }
}

// The same for any scale and weight, pair by pair in the block's place in shared memory.
template <int WK>
__device__ __forceinline__ Block16 quantize_pairs(uint32_t* place, float s) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const float2 c = q_pair<WK>(quotient(bf16lo(place[i]), s), quotient(bf16hi(place[i]), s));
    place[i] = pack_bf16(__fmul_rn(c.x, s), __fmul_rn(c.y, s));
  }
  return read16(place);
}

// Token rows through their quantizer into shared memory, zeros behind K; `share` warps work on a row.  The scale of a
// whole row needs a barrier in between (top: zeros before).  Read from L2: other blocks have written the rows of fc2.
template <int AK>
__device__ __forceinline__ void stage_rows(const __nv_bfloat16* act, const int* src, uint32_t* top, uint8_t* rows, int K,
                                           int share) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, col = min(warp / share, kCols);  // the last warps may have none
  const int first = warp % share * 32 + lane, step = share * 32;
  const int nblk = K / 16, padded = (K + kChunk - 1) / kChunk * (kChunk / 16);
  const bool has = col < kCols && src[col] >= 0;
  const uint4* in = reinterpret_cast<const uint4*>(act + (int64_t)(has ? src[col] : 0) * K);
  uint4* out = reinterpret_cast<uint4*>(rows + col * few_stride(K));
  float s_row = 0.0f;
  if constexpr (act_needs_row(AK)) {
    float amax = 0.0f;
    if (has)
      for (int b = first; b < nblk; b += step) {
        float f[16];
        unpack8(__ldcg(in + 2 * b), f);
        unpack8(__ldcg(in + 2 * b + 1), f + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
      }
    amax = warp_max(amax);
    if (has && lane == 0) atomicMax(top + col, __float_as_uint(amax));
    __syncthreads();
    amax = has ? __uint_as_float(top[col]) : 0.0f;
    s_row = AK == kQE4M3   ? __fdiv_rn(amax, 448.0f)
            : AK == kQInt8 ? __fdiv_rn(amax, 127.0f)
                           : deploy_tensor_scale(__fdiv_rn(amax, 6.0f));
  }
  if (!has) return;
#pragma unroll 1
  for (int b = first; b < padded; b += step) {
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (b < nblk) {
      u0 = __ldcg(in + 2 * b);
      u1 = __ldcg(in + 2 * b + 1);
      if constexpr (AK != kQNone) {
        float f[16];
        unpack8(u0, f);
        unpack8(u1, f + 8);
        if constexpr (row_scaled(AK)) {
          fakequant_act_inplace<AK, 16>(f, s_row);
        } else {
          float amax = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
          float sc = __fdiv_rn(amax, 6.0f);
          if constexpr (AK == kQE2M1G) sc = deployed_scale(sc, s_row);
          fakequant_act_inplace<kQE2M1, 16>(f, sc);
        }
        u0 = pack8(f);
        u1 = pack8(f + 8);
      }
    }
    out[2 * b] = u0;
    out[2 * b + 1] = u1;
  }
}

// A block takes a consecutive share [lo, hi) of all (pass, tile) pairs, passes outermost, so that it stages few passes'
// tokens; its teams of warps take the tiles of a pass in turn, and the warps of a team the chunks of a tile along K.
struct Share {
  int lo, hi;
  __device__ __forceinline__ Share(int passes, int tiles) {
    const int64_t total = (int64_t)passes * tiles;
    lo = (int)(total * blockIdx.x / gridDim.x);
    hi = (int)(total * (blockIdx.x + 1) / gridDim.x);
  }
};

// The chunks of this warp's tiles, in order, on their way into its ring.
template <int WK, bool FC1>
struct Loader {
  const Half& h;
  const Route& r;
  const int hi, depth, my_team, in_team, teams;
  const uint32_t ring;
  int tile = 0, last = 0, next, chunk = 0, slot = 0;  // next: where the next pass's tiles begin
  const __nv_bfloat16 *we = nullptr, *pw = nullptr;
  const float *se = nullptr, *ps = nullptr;

  __device__ __forceinline__ Loader(const Half& h, const Route& r, Share s, int depth, uint8_t* smem)
      : h(h), r(r), hi(s.hi), depth(depth), my_team((int)threadIdx.x / 32 / h.team), in_team((int)threadIdx.x / 32 % h.team),
        teams(kWarps / h.team), ring((uint32_t)__cvta_generic_to_shared(smem + threadIdx.x / 32 * depth * kSlot)),
        next(s.lo) {
    open_tile();
    load();
    if (depth > 2) load();
  }
  __device__ __forceinline__ void open_tile() {
    const int lane = threadIdx.x & 31;
    while (tile >= last && next < hi) {
      const int pass = next / h.tiles, tile0 = next - pass * h.tiles, e = r.expert_of(pass);
      last = min(h.tiles, tile0 + hi - next);
      next += last - tile0;
      tile = tile0 + my_team;
      we = h.w + (int64_t)e * (FC1 ? 2 * h.N : h.N) * h.K;
      se = h.s + (int64_t)e * (FC1 ? 2 * h.N : h.N) * h.scales;
    }
    const int row = tile * (FC1 ? 8 : 16);
    // a copy of the warp takes 4 rows of 128 bytes: lane / 8 the row, lane % 8 its 16 bytes
    pw = we + (int64_t)(row + lane / 8) * h.K;
    // E2M1: lane / 4 the row, lane % 4 its block of the chunk; else lane the row (16 of them)
    ps = se + (int64_t)(row + (WK == kQE2M1 ? lane / 4 : lane & 7)) * h.scales;
    if (WK != kQE2M1 && (lane & 8)) ps += h.sup;
    chunk = in_team;
  }
  __device__ __forceinline__ void load() {
    const int lane = threadIdx.x & 31, piece = lane & 7;
    if (tile < last) {
      if (chunk < h.chunks) {
        const int k0 = chunk * kChunk, bytes = k0 + 8 * piece < h.K ? 16 : 0;  // zeros behind K
        const __nv_bfloat16* from = pw + (bytes ? k0 + 8 * piece : 0);
        const uint32_t at = ring + slot * kSlot, to = at + lane / 8 * kPitch + piece * 16;
        copy16(to, from, bytes);
        copy16(to + 4 * kPitch, from + 4 * (int64_t)h.K, bytes);
        copy16(to + 8 * kPitch, from + h.up, bytes);
        copy16(to + 12 * kPitch, from + h.up + 4 * (int64_t)h.K, bytes);
        if constexpr (WK == kQE2M1) {
          const int b = k0 / 16 + (lane & 3), in = b < h.scales ? b : 0;
          copy4(at + 16 * kPitch + lane * 4, ps + in);
          copy4(at + 16 * kPitch + 128 + lane * 4, ps + in + h.sup);
        } else if constexpr (WK != kQNone) {
          if (lane < 16) copy4(at + 16 * kPitch + lane * 4, ps + (WK == kQInt4 ? k0 / 128 : 0));
        }
      }
      chunk += h.team;
      if (chunk >= h.per_warp * h.team) {
        tile += teams;
        open_tile();
      }
    }
    slot = slot + 1 == depth ? 0 : slot + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

struct FewSmem {
  float part[2][kWarps][16][kCols];
  uint32_t live[64], top[kCols];
  int row[kCols], src[kCols];
};

template <int WK, int AK, bool FC1>
__device__ __forceinline__ void run_half(const FewParams& q, const Half& h, const Route& r, Share share,
                                         Loader<WK, FC1>& loader, uint8_t* smem, FewSmem& s) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane / 4, t4 = lane & 3;
  const int team = h.team, my_team = loader.my_team, in_team = loader.in_team, teams = loader.teams;
  const int stride = few_stride(h.K), depth = q.depth;
  uint8_t* rows = smem + few_rows_at(depth);
  const int col = min(g, q.cols - 1);  // columns that are not staged give results that nobody reads
  int slot = 0, parity = 0;
  for (int u = share.lo; u < share.hi;) {
    const int pass = u / h.tiles, tile0 = u % h.tiles, ntiles = min(share.hi - u, h.tiles - tile0), e = r.expert_of(pass);
    u += ntiles;
    __syncthreads();  // the tokens of the pass before are no longer read
    if (warp == 0) {
      const int pair = r.pair_of(pass, e, q.idx);
      if (lane < kCols) {
        s.row[lane] = pair;
        s.src[lane] = FC1 && pair >= 0 ? pair / q.k : pair;
        s.top[lane] = 0;
      }
    }
    __syncthreads();
    int staged = 0;
#pragma unroll
    for (int i = 0; i < kCols; ++i) staged += s.row[i] >= 0;
    stage_rows<AK>(h.act, s.src, s.top, rows, h.K, kWarps / staged);
    __syncthreads();

    for (int tile = tile0 + my_team; tile < tile0 + ntiles; tile += teams) {
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int c = 0; c < h.per_warp; ++c) {
        if (depth > 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();  // the other lanes' copies too, and nobody reads the slot that the next load fills
        loader.load();
        const int chunk = c * team + in_team;
        if (chunk < h.chunks) {
          uint8_t* mine = smem + (warp * depth + slot) * kSlot;
          const float* sv = reinterpret_cast<const float*>(mine + 16 * kPitch) + (WK == kQE2M1 ? lane : g);
          uint32_t* wv = reinterpret_cast<uint32_t*>(mine + g * kPitch + t4 * 32);
          float sa = sv[0], sb = sv[WK == kQE2M1 ? 32 : 8];
          if (h.ragged && chunk * kChunk + 16 * t4 >= h.K) sa = sb = 1.0f;
          uint32_t odd = 0;
          Block16 a = quantize16<WK>(read16(wv), sa, &odd), b = quantize16<WK>(read16(wv + 8 * kPitch / 4), sb, &odd);
          if constexpr (WK != kQNone) {
            if (__builtin_expect(odd != 0, 0)) {
              a = quantize_pairs<WK>(wv, sa);
              b = quantize_pairs<WK>(wv + 8 * kPitch / 4, sb);
            }
          }
          const uint4* xs = reinterpret_cast<const uint4*>(rows + col * stride) + chunk * (kChunk / 8) + 2 * t4;
          const uint4 x0 = xs[0], x1 = xs[1];
          mma_bf16(acc, a.v[0], b.v[0], a.v[1], b.v[1], x0.x, x0.y);
          mma_bf16(acc, a.v[2], b.v[2], a.v[3], b.v[3], x0.z, x0.w);
          mma_bf16(acc, a.v[4], b.v[4], a.v[5], b.v[5], x1.x, x1.y);
          mma_bf16(acc, a.v[6], b.v[6], a.v[7], b.v[7], x1.z, x1.w);
        }
        slot = slot + 1 == depth ? 0 : slot + 1;
      }
      // the team's partial sums are joined in warp order
      float(*part)[kCols] = s.part[parity][warp];
      part[g][2 * t4] = acc[0];
      part[g][2 * t4 + 1] = acc[1];
      part[g + 8][2 * t4] = acc[2];
      part[g + 8][2 * t4 + 1] = acc[3];
      if (team > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + my_team), "r"(32 * team) : "memory");
      else __syncwarp();
      const float(*sum)[16][kCols] = &s.part[parity][my_team * team];
      for (int i = in_team * 32 + lane; i < (FC1 ? 64 : 128); i += 32 * team) {
        const int cc = FC1 ? i / 8 : i / 16, n = FC1 ? i % 8 : i % 16;
        if (s.row[cc] < 0) continue;
        if constexpr (FC1) {
          float zg = 0.0f, zu = 0.0f;
          for (int w = 0; w < team; ++w) {
            zg += sum[w][n][cc];
            zu += sum[w][n + 8][cc];
          }
          h.rows[(int64_t)s.row[cc] * h.N + tile * 8 + n] =
              __float2bfloat16_rn(__fmul_rn(silu_f(round_bf16(zg)), round_bf16(zu)));
        } else {
          float y = 0.0f;
          for (int w = 0; w < team; ++w) y += sum[w][n][cc];
          h.rows[(int64_t)s.row[cc] * h.N + tile * 16 + n] = __float2bfloat16_rn(y);
        }
      }
      parity ^= 1;
    }
    if constexpr (!FC1) {
      // the pass that completes a tile of Y combines it, in slot order whoever comes last
      __threadfence();
      __syncthreads();
      for (int i = warp; i < ntiles; i += kWarps) {
        const int n0 = (tile0 + i) * 16;
        uint32_t seen = 0;
        if (lane == 0) seen = atomicAdd(q.arrivals + tile0 + i, 1u);
        seen = __shfl_sync(0xffffffffu, seen, 0);
        if (seen + 1 != (uint32_t)r.passes) continue;
        __threadfence();
        for (int o = lane; o < q.T * 8; o += 32) {
          const int t = o / 8, n = n0 + 2 * (o % 8);
          const uint32_t live = r.slots_of(t);
          float v0 = 0.0f, v1 = 0.0f;
#pragma unroll 8
          for (int j = 0; j < q.k; ++j) {
            if (!(live >> j & 1)) continue;
            const uint32_t y = __ldcg(reinterpret_cast<const uint32_t*>(h.rows + (int64_t)(t * q.k + j) * h.N + n));
            const float pj = __ldg(q.p + t * q.k + j);
            v0 = fmaf(pj, bf16lo(y), v0);
            v1 = fmaf(pj, bf16hi(y), v1);
          }
          *reinterpret_cast<uint32_t*>(q.out + (int64_t)t * h.N + n) = pack_bf16(v0, v1);
        }
      }
    }
  }
}

// Every block is through with fc1 (they are all resident: a cooperative launch).  False: some did not come.
__device__ __forceinline__ bool all_arrived(uint32_t* arrived) {
  __threadfence();
  __syncthreads();
  bool there = true;
  if (threadIdx.x == 0) {
    atomicAdd(arrived, 1u);
    const long long t0 = clock64();
    uint32_t seen;
    do {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(arrived) : "memory");
      there = seen >= gridDim.x;
    } while (!there && clock64() - t0 < kWaitCycles);
  }
  return __syncthreads_and(there);
}

template <int WK, int AK>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewParams q) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FewSmem s;
  uint64_t* mask = reinterpret_cast<uint64_t*>(smem + few_mask_at(max(q.fc1.K, q.fc2.K), q.cols, q.depth));
  int err;
  const Route r = route(q, mask, reinterpret_cast<uint16_t*>(mask + q.E), s.live, &err);
  if (blockIdx.x == 0 && threadIdx.x == 0 && err) atomicOr(q.err, err);
  if (r.passes == 0) {  // every pair was dropped
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < q.T * q.fc2.N / 8; i += gridDim.x * kThreads)
      reinterpret_cast<uint4*>(q.out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  {
    const Share share(r.passes, q.fc1.tiles);
    Loader<WK, true> loader(q.fc1, r, share, q.depth, smem);
    run_half<WK, AK, true>(q, q.fc1, r, share, loader, smem, s);
  }
  const Share share(r.passes, q.fc2.tiles);
  Loader<WK, false> loader(q.fc2, r, share, q.depth, smem);
  if (!all_arrived(q.arrived) && threadIdx.x == 0) atomicOr(q.err, QAD_DEV_TIMEOUT);
  run_half<WK, AK, false>(q, q.fc2, r, share, loader, smem, s);
}

// Warps that share a tile along K: as many as leave less than an eighth of them idle at the last chunk.
int team_of(int chunks) {
  for (int w = kMaxTeam; w > 1; w /= 2)
    if ((chunks + w - 1) / w * w * 8 <= chunks * 9) return w;
  return 1;
}

void shape_half(Half* h, int64_t K, int64_t N, int block, bool fc1) {
  h->K = (int)K;
  h->N = (int)N;
  h->scales = block ? h->K / block : 1;
  h->chunks = (h->K + kChunk - 1) / kChunk;
  h->team = team_of(h->chunks);
  h->per_warp = (h->chunks + h->team - 1) / h->team;
  h->tiles = h->N / (fc1 ? 8 : 16);
  h->up = (fc1 ? N : 8) * K;
  h->sup = (fc1 ? N : 8) * h->scales;
  h->ragged = h->K % kChunk != 0;
}

template <int WK, int AK>
cudaError_t launch(FewParams q, cudaStream_t st) {
  constexpr int kMost = 227 * 1024 - (int)sizeof(FewSmem) - 1024;
  const int K = q.fc1.K > q.fc2.K ? q.fc1.K : q.fc2.K;
  q.cols = q.T < kCols ? q.T : kCols;
  while (q.cols > 1 && few_smem(K, q.cols, q.E, 2) > kMost) --q.cols;  // rows of 8192: 5, or 4 beside 1024 experts
  q.depth = few_smem(K, q.cols, q.E, 3) <= kMost ? 3 : 2;
  const int bytes = few_smem(K, q.cols, q.E, q.depth);
  const auto kernel = few_kernel<WK, AK>;
  // the same limit at every call: it belongs to the kernel, and another host thread's call may come before this launch
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)) return e;
  const int64_t units = (int64_t)q.T * q.k * (q.fc1.tiles > q.fc2.tiles ? q.fc1.tiles : q.fc2.tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units < num_sms() ? units : num_sms()), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeCooperative;
  a[0].val.cooperative = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, q);
}

cudaError_t launch_kind(int wk, int ak, const FewParams& q, cudaStream_t st) {
  if (wk == kQE2M1 && ak == kQE2M1) return launch<kQE2M1, kQE2M1>(q, st);
  if (wk == kQE2M1 && ak == kQE2M1G) return launch<kQE2M1, kQE2M1G>(q, st);
  if (wk == kQE2M1) return launch<kQE2M1, kQNone>(q, st);
  if (wk == kQInt4 && ak == kQE4M3) return launch<kQInt4, kQE4M3>(q, st);
  if (wk == kQInt4) return launch<kQInt4, kQNone>(q, st);
  if (wk == kQE4M3) return launch<kQE4M3, kQE4M3>(q, st);
  if (wk == kQInt8) return launch<kQInt8, kQInt8>(q, st);
  return launch<kQNone, kQNone>(q, st);
}

}  // namespace

int few_layout_of(const qad_moe_shape& s, FewLayout* L) {
  Layout whole;
  const int rc = layout_of(s, &whole);
  if (rc != QAD_OK) return rc;
  if (s.flags & ~QAD_FLAG_NO_QUANT) return QAD_ERR_INVALID_ARG;
  if (s.T > QAD_MOE_FEW_MAX_T || s.d > QAD_MOE_FEW_MAX_D || s.F > QAD_MOE_FEW_MAX_D) return QAD_ERR_UNSUPPORTED;
  auto up = [](int64_t v) { return (size_t)((v + 1023) / 1024 * 1024); };
  const int64_t R = s.T * s.topk;
  L->counters = 8 + 4 * (size_t)(s.d / 16);
  L->h = up(L->counters);
  L->y = L->h + up(2 * R * s.F);
  L->total = L->y + up(2 * R * s.d);
  return QAD_OK;
}

cudaError_t launch_moe_few(const qad_moe_shape& s, const FewLayout& L, const void* x, const int32_t* idx, const float* p,
                           const void* w13, const float* s13, const void* w2, const float* s2, void* out, uint8_t* ws,
                           cudaStream_t st) {
  const bool quant = !(s.flags & QAD_FLAG_NO_QUANT);
  const int wk = quant ? weight_kind(s.fmt) : kQNone, ak = quant ? act_kind(s.fmt) : kQNone;
  const int block = wk == kQE2M1 ? 16 : wk == kQInt4 ? 128 : 0;
  FewParams q = {};
  shape_half(&q.fc1, s.d, s.F, block, true);
  q.fc1.act = static_cast<const __nv_bfloat16*>(x);
  q.fc1.w = static_cast<const __nv_bfloat16*>(w13);
  q.fc1.s = s13;
  q.fc1.rows = reinterpret_cast<__nv_bfloat16*>(ws + L.h);
  shape_half(&q.fc2, s.F, s.d, block, false);
  q.fc2.act = q.fc1.rows;
  q.fc2.w = static_cast<const __nv_bfloat16*>(w2);
  q.fc2.s = s2;
  q.fc2.rows = reinterpret_cast<__nv_bfloat16*>(ws + L.y);
  q.idx = idx;
  q.p = p;
  q.out = static_cast<__nv_bfloat16*>(out);
  q.err = reinterpret_cast<int32_t*>(ws);
  q.arrived = reinterpret_cast<uint32_t*>(ws) + 1;
  q.arrivals = reinterpret_cast<uint32_t*>(ws) + 2;
  q.T = (int)s.T;
  q.k = s.topk;
  q.E = (int)s.E;
  if (cudaError_t e = cudaMemsetAsync(ws, 0, L.counters, st)) return e;
  prof_begin(QAD_K_MOE_FEW, st);
  const cudaError_t e = launch_kind(wk, ak, q, st);
  prof_end(QAD_K_MOE_FEW, st);
  return e;
}

}  // namespace qad
