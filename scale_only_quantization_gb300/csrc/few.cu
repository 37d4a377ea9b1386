// The whole expert layer for a few tokens (generation): two launches, each of which reads the weights of the experts
// that some token names once, fake-quantizes them in registers and multiplies them there.
//
//   fc1:  Z1 = A1 . W13_hat^T, H = bf16(silu(gate) * up)             A1 = AQ(x)
//   fc2:  Y = AQ(H) . W2_hat^T, out[t] = bf16(sum_j p[t, j] * Y_j)
//
// With so few rows the weights are all there is to move (2 bytes an element and its part of a scale), and each element
// costs about eight instructions of fake-quantization whatever the number of tokens.  So a warp copies 64 weights of 16
// rows ahead into its ring in shared memory; a lane quantizes 16 of a row (one quantization block) in registers in
// the tensor cores' fragment layout, and four m16n8k16 products take them as they lie.  The order of k inside a product
// does not matter as long as both operands agree, so the tokens' rows (shared memory, up to 8 columns) are read in the
// same order.  A warp reads only what it copied itself: the ring needs no block barrier.  tcgen05 would want the quantized weights
// in shared memory: a write and a read of every element for products that are idle most of the time here.
#include "common.cuh"
#include "dependents.cuh"
#include "internal.h"

namespace qad {
namespace {

constexpr int kThreads = 768, kWarps = kThreads / 32;  // one block per SM
constexpr int kCols = 8;    // tokens of one expert that a pass over its weights serves, at most
constexpr int kMaxTeam = 8; // warps that share a tile
constexpr int kChunk = 64;  // elements along K of one step: 16 for each lane of a quad
constexpr int kPitch = 2 * kChunk + 16;   // bytes between the rows of a chunk: 16-byte reads of 8 lanes meet no bank twice
constexpr int kSlot = 16 * kPitch + 256;  // bytes of a warp's chunk: 16 rows of weights, up to 4 scales a row

struct FewParams {
  const __nv_bfloat16* act;  // fc1: x [T, K]; fc2: H [T * k, K]
  const __nv_bfloat16* w;    // [E, rows, K], rows = 2N (fc1) or N (fc2)
  const float* s;
  const int32_t* idx;
  const float* p;
  __nv_bfloat16* rows;  // fc1: H [T * k, N]; fc2: Y [T * k, N]
  __nv_bfloat16* out;   // fc2: [T, N]
  int32_t* err;
  uint32_t* arrivals;  // [d / 16]: experts' passes that have written a tile of Y
  int T, k, E, K, N, scales;  // scales: per row
  int team, cols, d_tiles;    // team: warps that share a tile; cols: token rows staged at once
  int depth;                  // chunks of a warp in its ring: the one that is worked on and 1 or 2 on their way
};

__host__ __device__ constexpr int few_stride(int K) { return (K + kChunk - 1) / kChunk * kChunk * 2 + 16; }

struct Route {
  uint64_t* mask;    // [E]: the tokens that name the expert
  uint32_t* live;    // [T]: the slots of a token that count
  uint16_t* first;   // [E + 1]: the expert's first pass (`cols` tokens each)
};

// Dynamic shared memory: the warps' rings, the staged token rows, the masks and first passes of E experts.
__host__ __device__ constexpr int few_rows_at(int depth) { return kWarps * depth * kSlot; }
__host__ __device__ constexpr int few_mask_at(int K, int cols, int depth) { return few_rows_at(depth) + cols * few_stride(K); }
__host__ __device__ constexpr int few_smem(int K, int cols, int E, int depth) {
  return few_mask_at(K, cols, depth) + 8 * E + 2 * (E + 1) + 6;
}

// The pairs by expert, in every block for itself: at most 2048 of them.  Returns the passes in all.
__device__ __forceinline__ int route(const FewParams& q, const Route& r, int* err) {
  const int tid = threadIdx.x;
  for (int e = tid; e < q.E; e += kThreads) r.mask[e] = 0;
  for (int t = tid; t < q.T; t += kThreads) r.live[t] = 0;
  __syncthreads();
  int bad = 0;
  for (int i = tid; i < q.T * q.k; i += kThreads) {
    const int t = i / q.k, j = i % q.k;
    const int e = __ldg(q.idx + i);
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
    atomicOr(reinterpret_cast<unsigned long long*>(r.mask + e), 1ull << t);
    atomicOr(r.live + t, 1u << j);
  }
  *err = (__syncthreads_or(bad & QAD_DEV_BAD_INDEX) ? QAD_DEV_BAD_INDEX : 0) |
         (__syncthreads_or(bad & QAD_DEV_DUP_INDEX) ? QAD_DEV_DUP_INDEX : 0);
  if (tid < 32) {
    const int per = (q.E + 31) / 32, lo = min(q.E, tid * per), hi = min(q.E, lo + per);
    int n = 0;
    for (int e = lo; e < hi; ++e) n += (__popcll(r.mask[e]) + q.cols - 1) / q.cols;
    int at = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (tid >= o) at += v;
    }
    at -= n;
    for (int e = lo; e < hi; ++e) {
      r.first[e] = (uint16_t)at;
      at += (__popcll(r.mask[e]) + q.cols - 1) / q.cols;
    }
    if (tid == 31) r.first[q.E] = (uint16_t)at;
  }
  __syncthreads();
  return r.first[q.E];
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

// W_hat of 16 weights that share scale s, the bits of fakequant16_packed (see there for the quotient).  What follows the
// quotient x = fp32(w / s) takes fewer instructions here:
//  - E2M1: bf16(fp32(q s)) takes eight magnitudes, which the 3-bit codes of four weights look up by two byte permutations.
//    Four of them are halves or doubles of bf16(s) and bf16(1.5 s), that is their bits with the exponent moved;
//  - INT4, INT8: bf16(fp32(q s)) does not fall as q rises, so that clamping q is clamping it, two at a time.
// Scales and quotients out of range: pair by pair, in the weights' place in shared memory (16-byte aligned).
template <int WK>
__device__ __forceinline__ Block16 quantize16(uint32_t* place, float s) {
  auto read = [&]() {
    const uint4 lo = reinterpret_cast<const uint4*>(place)[0], hi = reinterpret_cast<const uint4*>(place)[1];
    return Block16{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
  };
  const Block16 w = read();
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
    if (__builtin_expect(!(s >= 0x1p-60f && s < 0x1p16f) || !(p.x == 0.0f && p.y == 0.0f), 0)) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const float2 c = q_pair<WK>(quotient(bf16lo(place[i]), s), quotient(bf16hi(place[i]), s));
        place[i] = pack_bf16(__fmul_rn(c.x, s), __fmul_rn(c.y, s));
      }
      return read();
    }
    return out;
  }
}

// Token rows through their quantizer into shared memory, zeros behind K; `share` warps work on a row.  The scale of a
// whole row needs a barrier in between (top: zeros before).
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
        unpack8(in[2 * b], f);
        unpack8(in[2 * b + 1], f + 8);
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
      u0 = in[2 * b];
      u1 = in[2 * b + 1];
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

// Tiles of 16 weight rows: fc1 8 gate rows and the 8 up rows that go with them, fc2 16 output rows.  A block takes a
// consecutive share of all (pass, tile) pairs, passes outermost, so that it stages few passes' tokens; its teams of warps
// take the tiles of a pass in turn, and the warps of a team the chunks of a tile along K.
template <int WK, int AK, bool FC1>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(FewParams q) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_live[64];
  __shared__ float s_part[2][kWarps][16][kCols];
  __shared__ int s_row[kCols], s_src[kCols];
  __shared__ uint32_t s_top[kCols];
  uint64_t* s_mask = reinterpret_cast<uint64_t*>(smem + few_mask_at(q.K, q.cols, q.depth));
  uint16_t* s_first = reinterpret_cast<uint16_t*>(s_mask + q.E);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane / 4, t4 = lane & 3;
  const int stride = few_stride(q.K), chunks = (q.K + kChunk - 1) / kChunk;
  const int team = q.team, my_team = warp / team, in_team = warp % team, teams = kWarps / team;
  const int tiles = FC1 ? q.N / 8 : q.N / 16;
  if (FC1) let_next_kernel_start();
  int err;
  const int passes = route(q, {s_mask, s_live, s_first}, &err);
  if (FC1 && blockIdx.x == 0) {
    if (tid == 0) *q.err = err;
    for (int i = tid; i < q.d_tiles; i += kThreads) q.arrivals[i] = 0;
  }
  if (!FC1 && passes == 0) {  // every pair was dropped
    wait_for_kernel_before();
    for (int i = blockIdx.x * kThreads + tid; i < q.T * q.N / 8; i += gridDim.x * kThreads)
      reinterpret_cast<uint4*>(q.out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t total = (int64_t)passes * tiles;
  const int lo = (int)(total * blockIdx.x / gridDim.x), hi = (int)(total * (blockIdx.x + 1) / gridDim.x);
  const int per_warp = (chunks + team - 1) / team;
  auto expert_of = [&](int pass) {  // the last expert whose first pass is not behind this one
    int e = 0;
    for (int b = 512; b; b >>= 1)
      if (e + b < q.E && s_first[e + b] <= pass) e += b;
    return e;
  };

  // the chunks of this warp's tiles, in order, on their way into its ring
  // a copy of the warp takes 4 rows of 128 bytes: lane / 8 the row, lane % 8 its 16 bytes
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem + warp * q.depth * kSlot);
  const int piece = lane & 7;
  const int64_t up = FC1 ? (int64_t)q.N * q.K : 8 * (int64_t)q.K, sup = FC1 ? (int64_t)q.N * q.scales : 8 * (int64_t)q.scales;
  int ld_tile = 0, ld_last = 0, ld_next = lo, ld_chunk = 0, ld_slot = 0;  // ld_next: where the next pass's tiles begin
  const __nv_bfloat16 *ld_w = nullptr, *pw = nullptr;
  const float *ld_s = nullptr, *ps = nullptr;
  auto open_tile = [&]() {
    while (ld_tile >= ld_last && ld_next < hi) {
      const int pass = ld_next / tiles, tile0 = ld_next - pass * tiles, e = expert_of(pass);
      ld_last = min(tiles, tile0 + hi - ld_next);
      ld_next += ld_last - tile0;
      ld_tile = tile0 + my_team;
      ld_w = q.w + (int64_t)e * (FC1 ? 2 * q.N : q.N) * q.K;
      ld_s = q.s + (int64_t)e * (FC1 ? 2 * q.N : q.N) * q.scales;
    }
    const int row = ld_tile * (FC1 ? 8 : 16);
    pw = ld_w + (int64_t)(row + lane / 8) * q.K;
    // E2M1: lane / 4 the row, lane % 4 its block of the chunk; else lane the row (16 of them)
    ps = ld_s + (int64_t)(row + (WK == kQE2M1 ? lane / 4 : lane & 7)) * q.scales;
    if (WK != kQE2M1 && (lane & 8)) ps += sup;
    ld_chunk = in_team;
  };
  open_tile();
  auto load = [&]() {
    if (ld_tile < ld_last) {
      if (ld_chunk < chunks) {
        const int k0 = ld_chunk * kChunk, bytes = k0 + 8 * piece < q.K ? 16 : 0;  // zeros behind K
        const __nv_bfloat16* from = pw + (bytes ? k0 + 8 * piece : 0);
        const uint32_t at = ring + ld_slot * kSlot, to = at + lane / 8 * kPitch + piece * 16;
        copy16(to, from, bytes);
        copy16(to + 4 * kPitch, from + 4 * (int64_t)q.K, bytes);
        copy16(to + 8 * kPitch, from + up, bytes);
        copy16(to + 12 * kPitch, from + up + 4 * (int64_t)q.K, bytes);
        if constexpr (WK == kQE2M1) {
          const int b = k0 / 16 + (lane & 3), in = b < q.scales ? b : 0;
          copy4(at + 16 * kPitch + lane * 4, ps + in);
          copy4(at + 16 * kPitch + 128 + lane * 4, ps + in + sup);
        } else if constexpr (WK != kQNone) {
          if (lane < 16) copy4(at + 16 * kPitch + lane * 4, ps + (WK == kQInt4 ? k0 / 128 : 0));
        }
      }
      ld_chunk += team;
      if (ld_chunk >= per_warp * team) {
        ld_tile += teams;
        open_tile();
      }
    }
    ld_slot = ld_slot + 1 == q.depth ? 0 : ld_slot + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  load();
  if (q.depth > 2) load();
  if (!FC1) wait_for_kernel_before();

  int slot = 0, parity = 0;
  const int col = min(g, q.cols - 1);  // columns that are not staged give results that nobody reads
  for (int u = lo; u < hi;) {
    const int pass = u / tiles, tile0 = u % tiles, ntiles = min(hi - u, tiles - tile0), e = expert_of(pass);
    u += ntiles;
    __syncthreads();  // the tokens of the pass before are no longer read
    if (tid < kCols) {
      uint64_t m = s_mask[e];
      for (int i = (pass - s_first[e]) * q.cols + tid; i > 0 && m; --i) m &= m - 1;
      int row = -1, src = -1;
      if (m && tid < q.cols) {
        const int t = __ffsll((long long)m) - 1;
        for (int j = 0; j < q.k; ++j)
          if ((s_live[t] >> j & 1) && __ldg(q.idx + t * q.k + j) == e) row = t * q.k + j;
        src = FC1 ? t : row;
      }
      s_row[tid] = row;
      s_src[tid] = src;
      s_top[tid] = 0;
    }
    __syncthreads();
    const int staged = min(q.cols, __popcll(s_mask[e]) - (pass - s_first[e]) * q.cols);
    stage_rows<AK>(q.act, s_src, s_top, smem + few_rows_at(q.depth), q.K, kWarps / staged);
    __syncthreads();

    for (int tile = tile0 + my_team; tile < tile0 + ntiles; tile += teams) {
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int c = 0; c < per_warp; ++c) {
        if (q.depth > 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();  // the other lanes' copies too, and nobody reads the slot that the next load fills
        load();
        const int chunk = c * team + in_team;
        if (chunk < chunks) {
          uint8_t* mine = smem + (warp * q.depth + slot) * kSlot;
          const float* sv = reinterpret_cast<const float*>(mine + 16 * kPitch) + (WK == kQE2M1 ? lane : g);
          uint32_t* wv = reinterpret_cast<uint32_t*>(mine + g * kPitch + t4 * 32);
          const bool in = chunk * kChunk + 16 * t4 < q.K;
          const Block16 a = quantize16<WK>(wv, in ? sv[0] : 1.0f);
          const Block16 b = quantize16<WK>(wv + 8 * kPitch / 4, in ? sv[WK == kQE2M1 ? 32 : 8] : 1.0f);
          const uint4* xs = reinterpret_cast<const uint4*>(smem + few_rows_at(q.depth) + col * stride) + chunk * (kChunk / 8) + 2 * t4;
          const uint4 x0 = xs[0], x1 = xs[1];
          mma_bf16(acc, a.v[0], b.v[0], a.v[1], b.v[1], x0.x, x0.y);
          mma_bf16(acc, a.v[2], b.v[2], a.v[3], b.v[3], x0.z, x0.w);
          mma_bf16(acc, a.v[4], b.v[4], a.v[5], b.v[5], x1.x, x1.y);
          mma_bf16(acc, a.v[6], b.v[6], a.v[7], b.v[7], x1.z, x1.w);
        }
        slot = slot + 1 == q.depth ? 0 : slot + 1;
      }
      // the team's partial sums are joined in warp order
      float(*part)[kCols] = s_part[parity][warp];
      part[g][2 * t4] = acc[0];
      part[g][2 * t4 + 1] = acc[1];
      part[g + 8][2 * t4] = acc[2];
      part[g + 8][2 * t4 + 1] = acc[3];
      if (team > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + my_team), "r"(32 * team) : "memory");
      else __syncwarp();
      const float(*sum)[16][kCols] = &s_part[parity][my_team * team];
      for (int i = in_team * 32 + lane; i < (FC1 ? 64 : 128); i += 32 * team) {
        const int cc = FC1 ? i / 8 : i / 16, n = FC1 ? i % 8 : i % 16;
        if (s_row[cc] < 0) continue;
        if constexpr (FC1) {
          float zg = 0.0f, zu = 0.0f;
          for (int w = 0; w < team; ++w) {
            zg += sum[w][n][cc];
            zu += sum[w][n + 8][cc];
          }
          q.rows[(int64_t)s_row[cc] * q.N + tile * 8 + n] =
              __float2bfloat16_rn(__fmul_rn(silu_f(round_bf16(zg)), round_bf16(zu)));
        } else {
          float y = 0.0f;
          for (int w = 0; w < team; ++w) y += sum[w][n][cc];
          q.rows[(int64_t)s_row[cc] * q.N + tile * 16 + n] = __float2bfloat16_rn(y);
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
        if (seen + 1 != (uint32_t)passes) continue;
        __threadfence();
        for (int o = lane; o < q.T * 8; o += 32) {
          const int t = o / 8, n = n0 + 2 * (o % 8);
          const uint32_t live = s_live[t];
          float v0 = 0.0f, v1 = 0.0f;
#pragma unroll 8
          for (int j = 0; j < q.k; ++j) {
            if (!(live >> j & 1)) continue;
            const uint32_t y = __ldcg(reinterpret_cast<const uint32_t*>(q.rows + (int64_t)(t * q.k + j) * q.N + n));
            const float pj = __ldg(q.p + t * q.k + j);
            v0 = fmaf(pj, bf16lo(y), v0);
            v1 = fmaf(pj, bf16hi(y), v1);
          }
          *reinterpret_cast<uint32_t*>(q.out + (int64_t)t * q.N + n) = pack_bf16(v0, v1);
        }
      }
    }
  }
}

// Warps that share a tile along K: as many as leave less than an eighth of them idle at the last chunk.
int team_of(int64_t K) {
  const int chunks = (int)((K + kChunk - 1) / kChunk);
  for (int w = kMaxTeam; w > 1; w /= 2)
    if ((chunks + w - 1) / w * w * 8 <= chunks * 9) return w;
  return 1;
}

template <int WK, int AK, bool FC1>
cudaError_t launch(FewParams q, int64_t units, cudaStream_t st) {
  constexpr int kMost = 227 * 1024 - 26 * 1024;  // less what the kernel declares itself
  q.cols = q.T < kCols ? q.T : kCols;
  while (q.cols > 1 && few_smem(q.K, q.cols, q.E, 2) > kMost) q.cols /= 2;  // 4 for rows of 8192
  q.depth = few_smem(q.K, q.cols, q.E, 3) <= kMost ? 3 : 2;
  const int bytes = few_smem(q.K, q.cols, q.E, q.depth);
  const auto kernel = few_kernel<WK, AK, FC1>;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
  const unsigned blocks = (unsigned)(units < num_sms() ? units : num_sms());
  if (!FC1) return launch_dependent(kernel, blocks, kThreads, bytes, st, q);
  kernel<<<blocks, kThreads, bytes, st>>>(q);
  return cudaGetLastError();
}

template <bool FC1>
cudaError_t launch_kind(int wk, int ak, const FewParams& q, int64_t units, cudaStream_t st) {
  if (wk == kQE2M1 && ak == kQE2M1) return launch<kQE2M1, kQE2M1, FC1>(q, units, st);
  if (wk == kQE2M1 && ak == kQE2M1G) return launch<kQE2M1, kQE2M1G, FC1>(q, units, st);
  if (wk == kQE2M1) return launch<kQE2M1, kQNone, FC1>(q, units, st);
  if (wk == kQInt4 && ak == kQE4M3) return launch<kQInt4, kQE4M3, FC1>(q, units, st);
  if (wk == kQInt4) return launch<kQInt4, kQNone, FC1>(q, units, st);
  if (wk == kQE4M3) return launch<kQE4M3, kQE4M3, FC1>(q, units, st);
  if (wk == kQInt8) return launch<kQInt8, kQInt8, FC1>(q, units, st);
  return launch<kQNone, kQNone, FC1>(q, units, st);
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
  L->arrivals = 256;
  L->h = up(256 + 4 * (s.d / 16));
  L->y = L->h + up(2 * R * s.F);
  L->total = L->y + up(2 * R * s.d);
  return QAD_OK;
}

cudaError_t launch_moe_few(const qad_moe_shape& s, const FewLayout& L, const void* x, const int32_t* idx, const float* p,
                           const void* w13, const float* s13, const void* w2, const float* s2, void* out, uint8_t* ws,
                           cudaStream_t st) {
  const bool quant = !(s.flags & QAD_FLAG_NO_QUANT);
  const int kind = quant ? weight_kind(s.fmt) : kQNone;
  const int block = kind == kQE2M1 ? 16 : kind == kQInt4 ? 128 : 0;
  FewParams q = {};
  q.idx = idx;
  q.p = p;
  q.out = static_cast<__nv_bfloat16*>(out);
  q.err = reinterpret_cast<int32_t*>(ws);
  q.arrivals = reinterpret_cast<uint32_t*>(ws + L.arrivals);
  q.T = (int)s.T;
  q.k = s.topk;
  q.E = (int)s.E;
  const int ak = quant ? act_kind(s.fmt) : kQNone;
  q.d_tiles = (int)(s.d / 16);
  const int64_t pairs = s.T * s.topk;  // no more passes than pairs

  q.act = static_cast<const __nv_bfloat16*>(x);
  q.w = static_cast<const __nv_bfloat16*>(w13);
  q.s = s13;
  q.rows = reinterpret_cast<__nv_bfloat16*>(ws + L.h);
  q.K = (int)s.d;
  q.N = (int)s.F;
  q.scales = block ? q.K / block : 1;
  q.team = team_of(q.K);
  prof_begin(QAD_K_MOE_FEW, st);
  cudaError_t e = launch_kind<true>(kind, ak, q, pairs * (q.N / 8), st);
  if (e == cudaSuccess) {
    q.act = reinterpret_cast<const __nv_bfloat16*>(ws + L.h);
    q.w = static_cast<const __nv_bfloat16*>(w2);
    q.s = s2;
    q.rows = reinterpret_cast<__nv_bfloat16*>(ws + L.y);
    q.K = (int)s.F;
    q.N = (int)s.d;
    q.scales = block ? q.K / block : 1;
    q.team = team_of(q.K);
    note_launches(1);
    e = launch_kind<false>(kind, ak, q, pairs * (q.N / 16), st);
  }
  prof_end(QAD_K_MOE_FEW, st);
  return e;
}

}  // namespace qad
