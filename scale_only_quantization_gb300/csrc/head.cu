// Softmax cross entropy of hidden states h [N, d] against an output head W [V, d] (kept in high
// precision and frozen, as the router is), in pieces of the vocabulary: the logits are never kept.
//
//   z = h W^T,  loss_i = lse_i - z_it = log(1 + sum_{v != t} exp(z_iv - z_it))
//   dh_i = g_i (sum_v q_iv w_v - w_t),  dW_v = sum_i g_i (q_iv - 1[v = t]) h_i
//
// One sweep over the vocabulary gives the loss and dh: the logits of a piece leave the tensor
// cores as e = exp(z - ref_i) with ref_i the row's own target logit, known before the sweep from one
// dot product; e (bf16, the target's column left out) is multiplied by the same piece of W at
// once and accumulated in fp32, and the row's 1 / sum e is applied at the end.  So the logits are
// computed once, not once for the normaliser and once for the gradient.  With the target as the
// reference, sum_{v != t} e is the loss's own argument (no cancellation however sure the model is)
// and (q_t - 1) w_t is added in fp32.  e may be far above 1 (bf16 has fp32's range): only the row
// tiles in which some row's largest logit is over kMaxAbove nats above its target's are swept again, that row
// with the largest as its reference (the second sweep's kernels leave at once when no row asked for it).
// dW needs the final normaliser, so its pieces are computed from the logits a second time.
//
// The products run on SM pairs (tcgen05 cta_group::2, 256 x 256 tiles) with the roles and
// barriers of the grouped GEMMs: warp 0 of each CTA loads, warp 1 of the leader issues the MMAs,
// warps 2-9 run the epilogue of one accumulator while the other is filled.
//
// What bounds it: the tensor cores from a few hundred token rows on (8192 x 2048 x 151936 with dh: 4 N V d
// flop in 6.0 to 6.3 ms as the power cap allows, 1.62 to 1.70 PFLOP/s; the logits kernel at 88% of the tensor pipe's
// cycles, its epilogue of 5500 cycles a tile under the 16400 of the tile's MMAs, the product with the head at 97%);
// below that the head's one reading per product (8 rows' loss 111 to 114 us, 5.5 TB/s; with dh the head is read twice,
// 234 us: one piece is the whole vocabulary, so the second product finds none of it in L2).  At d = 256 the
// epilogue is longer than the MMAs, and the launches of the short kernels weigh as much (512 x 256 x 32000: 51 us).
//
// Roundings to bf16: e before the product with the head (2^-8 of a term, below dh's own rounding: dh is as far from
// the 64-bit value as with fp32 probabilities, 1.7e-3), and the normalised residual g (q - 1) before the product with h,
// which raises dW's error from 1.7e-3 to 2.4e-3: the tensor cores take bf16 operands.  exp is the intrinsic (2
// ulp and 1.2 ulp per nat of its argument): the loss is off by 1.7e-7 instead of 7.5e-8.
#include <utility>

#include "internal.h"
#include "tcgen05.cuh"

namespace qad {
namespace {

constexpr int kTile = 256;            // rows and columns of a pair tile
constexpr int kThreadsH = 320;
constexpr int kEpiWarps = 8;
constexpr float kMaxAbove = 60.0f;    // exp(60) summed over 2^30 columns stays below fp32's range

// M_LOGITS: e [rows, piece];  M_U: U += e W;  M_DW: dW = e^T h.  With kFewRows token rows or fewer the
// products are taken transposed (M_*_T: the vocabulary, or the columns of U, as the 256 rows of a
// tile and the tokens as its 128 columns), so that the tensor cores do not multiply empty rows and
// the head streams at the memory's rate.
enum { M_LOGITS = 0, M_U = 1, M_DW = 2, M_LOGITS_T = 3, M_U_T = 4, M_DW_T = 5 };
constexpr int kFewRows = 128;
constexpr int kMaxPairs = 76;  // SM pairs of the grid at most: bounds the partial sums of a split contraction

struct HeadParams {
  const int32_t* gate;  // null, or a word: 0 = nothing to do, else (LISTED) the row tiles to do
  const int32_t* list;  // those row tiles
  int32_t* err;
  int mt, nt, num_kb;   // tiles along the output's rows and columns, K blocks
  int n_fast;           // tile order: columns fastest
  int split;            // slabs of K blocks that are contracted apart (U; else 1)
  int a_row0, b_row0;   // first row of the A / B tensors of this piece
  int64_t N;            // token rows
  // logits: columns c0 .. c0 + cols of the vocabulary
  int c0, cols;
  const float *ref, *mul;       // per row: reference, factor (null: 1)
  const float* tval;            // per row: what the target's column holds (null: 0)
  const int32_t* target;        // per row: the target's column
  float *psum, *pmax;           // partial sums without the target / maxima, or null
  int join;                     // add to the parts, which an earlier piece has written
  int store_p;
  __nv_bfloat16* p;             // e: [N, ldp], transposed [piece, kFewRows]
  int64_t ldp;
  float* u;  // U: partial sums [slab, N, d]
  int d, add;
};

// The kernels of a call are launched as dependents of one another: each is set up while the one before it
// ends, and touches memory only after this wait, which the whole grid before it has completed by.  What those
// before it wrote (ref, mul, tval, tcol, zt, psum, pmax, u, the header) is read by ordinary loads: the non-coherent
// path of __ldg and of const __restrict__ is for memory that nobody writes while the kernel is resident, and such a
// load could be moved above the wait.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <int MODE> struct HCfg {
  static constexpr bool A_MN = MODE == M_DW || MODE == M_U_T, B_MN = MODE != M_LOGITS && MODE != M_LOGITS_T;
  static constexpr int TN = MODE == M_LOGITS_T || MODE == M_U_T ? kFewRows : kTile;  // columns of a tile
  static constexpr int ATOMS = MODE == M_U ? 1 : 2;
  static constexpr int BKE = ATOMS * BK;
  static constexpr int A_ATOM = BM * 128, B_ATOM = TN / 2 * 128;
  static constexpr int A_BYTES = ATOMS * A_ATOM, B_BYTES = ATOMS * B_ATOM;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = (192 * 1024) / STAGE;
  static constexpr bool BOXES = MODE == M_DW || MODE == M_DW_T;  // stores through TMA
  static constexpr int STAGING = BOXES ? kEpiWarps * 4096 : MODE == M_LOGITS_T ? 4 * kFewRows * 4 : 0;
  static constexpr int SMEM = STAGES * STAGE + 512 + 1024 + STAGING;
};

struct HTile {
  int mb, nb;
};
// LISTED: of the row tiles in p.list only, mt of them
template <bool LISTED>
__device__ __forceinline__ HTile htile(const HeadParams& p, int mt, int t) {
  HTile x;
  if (p.n_fast) {
    x.mb = t / p.nt;
    x.nb = t - x.mb * p.nt;
  } else {
    x.nb = t / mt;
    x.mb = t - x.nb * mt;
  }
  if constexpr (LISTED) x.mb = p.list[x.mb];
  return x;
}

// The tiles of one pair, or, where the contraction is split, its slabs of tiles: every role of the CTA walks
// the same sequence.  Slab s covers the K blocks [s num_kb / split, (s + 1) num_kb / split); the pairs take
// all tiles of a slab before the next one's, so that those running together read the same K blocks of
// both operands from L2.
template <bool LISTED> struct Walk {
  int tile, kb0, kb1, slab;
  int at, step, mt, tiles;
  __device__ __forceinline__ Walk(const HeadParams& p, int pair, int pairs)
      : at(pair), step(pairs), mt(LISTED ? *p.gate : p.mt), tiles(mt * p.nt) {}
  __device__ __forceinline__ bool next(const HeadParams& p) {
    if (at >= tiles * p.split) return false;
    slab = at / tiles;
    tile = at - slab * tiles;
    kb0 = (int)((int64_t)slab * p.num_kb / p.split);
    kb1 = (int)((int64_t)(slab + 1) * p.num_kb / p.split);
    at += step;
    return true;
  }
};

// A 32 x 32 bf16 box of this warp through its staging memory (64-byte swizzle: 16-byte chunk c of
// row r at c ^ ((r >> 1) & 3)) and out by TMA; two boxes in turn.
__device__ __forceinline__ void store_box32(const CUtensorMap* tm, uint32_t stage_base, uint32_t& buf, int lane,
                                            const uint4 (&v)[4], int x, int y) {
  const uint32_t box = stage_base + buf * 2048u;
  if (lane == 0) bulk_wait_read<1>();
  __syncwarp();
  const uint32_t sw = ((uint32_t)lane >> 1) & 3u;
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) st_shared_v4(box + (uint32_t)lane * 64u + ((((uint32_t)ch) ^ sw) << 4), v[ch]);
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(tm, box, x, y);
    bulk_commit();
  }
  buf ^= 1u;
}

__device__ __forceinline__ void st_b32x8(uint32_t* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Row r's 128 columns of a logits tile: e = exp(z - ref) (x factor), its sum without the target,
// the largest logit, and the bf16 piece for the product that follows.
__device__ __forceinline__ void epi_logits(const HeadParams& p, const HTile& ti, int rank, uint32_t tbase, int q,
                                           int lane, int half) {
  const int64_t row = ti.mb * kTile + rank * BM + 32 * q + lane;
  const bool live = row < p.N;
  const float ref = live ? p.ref[row] : 0.0f;
  const float mul = live && p.mul ? p.mul[row] : 1.0f;
  const float tv = live && p.tval ? p.tval[row] : 0.0f;
  const int col0 = ti.nb * kTile + half * 128;  // within the piece
  const int target = live ? p.target[row] - p.c0 - col0 : -1;  // within these 128 columns
  const bool edge = col0 + 128 > p.cols;
  float sum = 0.0f, top = -INFINITY;
  uint32_t r[32], next[32];
  tmem_ld32_issue(tbase + half * 128, r);
  tmem_wait32(r);
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    if (c < 3) tmem_ld32_issue(tbase + half * 128 + 32 * (c + 1), next);
    const int tc = target - 32 * c, valid = p.cols - (col0 + 32 * c);
    // the chunks that hold no row's target, and lie inside the vocabulary, need no comparison per element
    const bool special = edge || __any_sync(0xffffffffu, (unsigned)tc < 32u);
    uint4 out[4];
    uint32_t* o = reinterpret_cast<uint32_t*>(out);
    if (special) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float e[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float z = __uint_as_float(r[i + j]);
          float x = __expf(z - ref);
          const bool out_of = edge && i + j >= valid;
          if (!out_of) top = fmaxf(top, z);
          if (out_of || i + j == tc) x = 0.0f;
          sum += x;
          x *= mul;
          if (i + j == tc) x = tv;
          e[j] = x;
        }
        o[i / 2] = pack_bf16(e[0], e[1]);
      }
    } else if (p.psum) {  // the sweep: no factor
      const uint64_t nr2 = f2pack(-ref, -ref);
      uint64_t sum2 = f2pack(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float a = __uint_as_float(r[i]), b = __uint_as_float(r[i + 1]);
        const float2 x = f2unpack(f2add(f2pack(a, b), nr2));
        const float e0 = __expf(x.x), e1 = __expf(x.y);
        top = fmaxf(top, fmaxf(a, b));
        sum2 = f2add(sum2, f2pack(e0, e1));
        o[i / 2] = pack_bf16(e0, e1);
      }
      const float2 s2 = f2unpack(sum2);
      sum += s2.x + s2.y;
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        o[i / 2] = pack_bf16(__expf(__uint_as_float(r[i]) - ref) * mul, __expf(__uint_as_float(r[i + 1]) - ref) * mul);
    }
    if (p.store_p && live) {  // two 32-byte sectors of the row
      uint32_t* to = reinterpret_cast<uint32_t*>(p.p + row * p.ldp + col0 + 32 * c);
      st_b32x8(to, out[0], out[1]);
      st_b32x8(to + 8, out[2], out[3]);
    }
    __syncwarp();  // the next tensor-memory load is the whole warp's
    if (c < 3) {
      tmem_wait32(next);
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = next[i];
    }
  }
  if (p.psum && live) {
    const int64_t at = (int64_t)(2 * ti.nb + half) * p.N + row;
    p.psum[at] = p.join ? p.psum[at] + sum : sum;
    p.pmax[at] = p.join ? fmaxf(p.pmax[at], top) : top;
  }
}

// Vocabulary row v's e for 64 of the tokens, 8 at a time; sums[i], tops[i]: token 8 i + lane / 4 of these 64,
// over all rows that this warp has seen
__device__ __forceinline__ void epi_logits_t(const HeadParams& p, const float* tok, const HTile& ti, int rank,
                                             uint32_t tbase, int q, int lane, int half, float (&sums)[8],
                                             float (&tops)[8]) {
  const int vr = ti.mb * kTile + rank * BM + 32 * q + lane;  // within the piece
  const bool live = vr < p.cols;
  const int v = p.c0 + vr;
  const float4* ref = reinterpret_cast<const float4*>(tok);
  const float4* mul = ref + kFewRows / 4;
  const float4* tv = mul + kFewRows / 4;
  const int4* tgt = reinterpret_cast<const int4*>(tv + kFewRows / 4);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (64 * half + 32 * c >= p.N && !p.store_p) continue;  // tokens that are not there; if stored, their e must be 0
    uint32_t r[32];
    tmem_ld32_issue(tbase + 64 * half + 32 * c, r);
    tmem_wait32(r);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n0 = 64 * half + 32 * c + 8 * k;
      if (n0 >= p.N && !p.store_p) continue;
      float x[8], y[8];
#pragma unroll
      for (int i4 = 0; i4 < 2; ++i4) {
        const float4 rf = ref[n0 / 4 + i4], mf = mul[n0 / 4 + i4], tf = tv[n0 / 4 + i4];
        const int4 tg = tgt[n0 / 4 + i4];
        const float rr[4] = {rf.x, rf.y, rf.z, rf.w}, mm[4] = {mf.x, mf.y, mf.z, mf.w}, tt[4] = {tf.x, tf.y, tf.z, tf.w};
        const int gg[4] = {tg.x, tg.y, tg.z, tg.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __expf(__uint_as_float(r[8 * k + 4 * i4 + i]) - rr[i]);
          const bool none = !live || n0 + 4 * i4 + i >= p.N;
          x[4 * i4 + i] = none || gg[i] == v ? 0.0f : e;
          y[4 * i4 + i] = none ? 0.0f : gg[i] == v ? tt[i] : e * mm[i];
        }
      }
      if (p.store_p) *reinterpret_cast<uint4*>(p.p + (int64_t)vr * kFewRows + n0) = pack8(y);
      if (p.psum && n0 < p.N) {
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = live ? __uint_as_float(r[8 * k + i]) : -INFINITY;
        // over the warp's 32 rows: three steps halve the tokens a lane carries, until it has one
#pragma unroll
        for (int off = 16, n = 4; n; off /= 2, n /= 2) {
          const bool up = lane & off;
#pragma unroll
          for (int i = 0; i < n; ++i) {
            x[i] = (up ? x[i + n] : x[i]) + __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + n], off);
            z[i] = fmaxf(up ? z[i + n] : z[i], __shfl_xor_sync(0xffffffffu, up ? z[i] : z[i + n], off));
          }
        }
#pragma unroll
        for (int off = 2; off; off /= 2) {
          x[0] += __shfl_xor_sync(0xffffffffu, x[0], off);
          z[0] = fmaxf(z[0], __shfl_xor_sync(0xffffffffu, z[0], off));
        }
        sums[4 * c + k] += x[0];
        tops[4 * c + k] = fmaxf(tops[4 * c + k], z[0]);
      }
    }
  }
}

// Row dd (a column of U) of 64 tokens: U^T += W^T e, this slab's partial sums, fp32
__device__ __forceinline__ void epi_u_t(const HeadParams& p, const HTile& ti, int slab, int rank, uint32_t tbase, int q,
                                        int lane, int half) {
  const int dd = ti.mb * kTile + rank * BM + 32 * q + lane;
  float* u = p.u + (int64_t)slab * p.N * p.d + dd;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int n0 = 64 * half + 32 * c;
    if (n0 >= p.N) continue;
    uint32_t r[32];
    tmem_ld32_issue(tbase + n0, r);
    tmem_wait32(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (n0 + i >= p.N || dd >= p.d) continue;
      float* at = u + (int64_t)(n0 + i) * p.d;
      *at = __uint_as_float(r[i]) + (p.add ? *at : 0.0f);
    }
    __syncwarp();  // the next tensor-memory load is the whole warp's
  }
}

__device__ __forceinline__ void ld_f32x8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p) : "memory");
}
__device__ __forceinline__ void st_f32x8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Row r's 128 columns of U += e W, this slab's partial sums, fp32 in global memory
__device__ __forceinline__ void epi_u(const HeadParams& p, const HTile& ti, int slab, int rank, uint32_t tbase, int q,
                                      int lane, int half) {
  const int64_t row = ti.mb * kTile + rank * BM + 32 * q + lane;
  const int col0 = ti.nb * kTile + half * 128;
  float* to = p.u + ((int64_t)slab * p.N + row) * p.d + col0;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld32_issue(tbase + half * 128 + 32 * c, r);
    // one 32-byte sector of the row per access: the warp's lanes are 32 rows
    float* u = to + 32 * c;
    const bool live = row < p.N;
    float before[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p.add && live && col0 + 32 * c + 8 * i < p.d) ld_f32x8(u + 8 * i, before[i]);
    tmem_wait32(r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!live || col0 + 32 * c + 8 * i >= p.d) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[8 * i + j]) + (p.add ? before[i][j] : 0.0f);
      st_f32x8(u + 8 * i, v);
    }
    __syncwarp();  // the next tensor-memory load is the whole warp's
  }
}

// Row r's 128 columns of dW, bf16
__device__ __forceinline__ void epi_dw(const HeadParams& p, const CUtensorMap* tm, const HTile& ti, int rank,
                                       uint32_t tbase, int q, int lane, int half, uint32_t stage_base, uint32_t& buf) {
  const int y = ti.mb * kTile + rank * BM + 32 * q;
  const int col0 = ti.nb * kTile + half * 128;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld32_issue(tbase + half * 128 + 32 * c, r);
    tmem_wait32(r);
    // a box that starts past the piece's rows or past d is not stored; one that straddles the
    // head's end or d is cut by the tensor map's extent
    if (col0 + 32 * c >= p.d || y >= p.cols) continue;
    uint4 out[4];
    uint32_t* o = reinterpret_cast<uint32_t*>(out);
#pragma unroll
    for (int i = 0; i < 32; i += 2) o[i / 2] = pack_bf16(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
    store_box32(tm, stage_base, buf, lane, out, col0 + 32 * c, p.c0 + y);
  }
}

template <int MODE, bool LISTED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsH, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const HeadParams p) {
  using C = HCfg<MODE>;
  constexpr int STAGES = C::STAGES, BKE = C::BKE, ATOMS = C::ATOMS, TN = C::TN;
  constexpr uint32_t IDESC = instr_desc<TN, C::A_MN, C::B_MN>();
  let_next_start();
  wait_for_previous();
  if (p.gate && *p.gate == 0) return;  // the whole grid alike
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t a_ring = smem0, b_ring = smem0 + STAGES * C::A_BYTES;
  const uint32_t stage_out = smem0 + STAGES * C::STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (smem0 - smem_u32(smem_raw)) + STAGES * C::STAGE + C::STAGING);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* late = reinterpret_cast<int32_t*>(tmem_slot + 2);  // error word of the waits that drain

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    *late = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  float* tok = reinterpret_cast<float*>(smem_raw + (stage_out - smem_u32(smem_raw)));  // M_LOGITS_T: per token values
  if constexpr (MODE == M_LOGITS_T) {
    for (int i = threadIdx.x; i < kFewRows; i += kThreadsH) {
      const bool live = i < p.N;
      tok[i] = live ? p.ref[i] : 0.0f;
      tok[kFewRows + i] = live && p.mul ? p.mul[i] : 1.0f;
      tok[2 * kFewRows + i] = live && p.tval ? p.tval[i] : 0.0f;
      reinterpret_cast<int32_t*>(tok)[3 * kFewRows + i] = live ? p.target[i] : -1;
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2u * TN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int pair = (int)cluster_id(), pairs = (int)cluster_count();
  Walk<LISTED> wk(p, pair, pairs);

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    const int half = (int)rank * BM, half_n = (int)rank * (TN / 2);
    while (ok && wk.next(p)) {
      const HTile ti = htile<LISTED>(p, LISTED ? wk.mt : p.mt, wk.tile);
      for (int kb = wk.kb0; kb < wk.kb1; ++kb) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (leader) mbar_expect_tx(full_bar(stage), 2 * C::STAGE);
        const uint32_t fb = peer_addr(full_bar(stage), 0);
        const uint32_t sa = a_ring + stage * C::A_BYTES, sb = b_ring + stage * C::B_BYTES;
        // K-major: one box {64, 128 rows} per 128-byte K atom; MN-major: one box {64, BKE K rows} per
        // 64 columns
#pragma unroll
        for (int i = 0; i < (C::A_MN ? 2 : ATOMS); ++i) {
          if constexpr (C::A_MN)
            tma_load_2d(sa + i * BKE * 128, &tmA, ti.mb * kTile + half + i * 64, p.a_row0 + kb * BKE, fb);
          else
            tma_load_2d(sa + i * C::A_ATOM, &tmA, kb * BKE + i * BK, p.a_row0 + ti.mb * kTile + half, fb);
        }
#pragma unroll
        for (int i = 0; i < (C::B_MN ? TN / 128 : ATOMS); ++i) {
          if constexpr (C::B_MN)
            tma_load_2d(sb + i * BKE * 128, &tmB, ti.nb * TN + half_n + i * 64, p.b_row0 + kb * BKE, fb);
          else
            tma_load_2d(sb + i * C::B_ATOM, &tmB, kb * BKE + i * BK, p.b_row0 + ti.nb * TN + half_n, fb);
        }
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (*abort_flag) {  // let every load land before the CTA releases its shared memory
      for (int s = 0; s < STAGES; ++s)
        if (armed & (1u << s)) {
          volatile int zero = 0;
          if (leader) mbar_wait(full_bar(s), (armed_parity >> s) & 1u, &zero, late);
        }
    }
  } else if (warp == 1 && lane == 0 && leader) {
    // ------------------------------------------------------------------ MMA issuer (leader)
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    while (ok && wk.next(p)) {
      if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(acc * TN);
      for (int kb = wk.kb0; kb < wk.kb1; ++kb) {
        if (!mbar_wait(full_bar(stage), phase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = a_ring + stage * C::A_BYTES, sb = b_ring + stage * C::B_BYTES;
#pragma unroll
        for (int k = 0; k < ATOMS * 4; ++k) {
          const uint64_t ad = C::A_MN ? smem_desc(sa + k * 2048, BKE * 128, 1024)
                                      : smem_desc(sa + (k / 4) * C::A_ATOM + (k % 4) * 32, 16, 1024);
          const uint64_t bd = C::B_MN ? smem_desc(sb + k * 2048, BKE * 128, 1024)
                                      : smem_desc(sb + (k / 4) * C::B_ATOM + (k % 4) * 32, 16, 1024);
          mma_issue<false>(d_tmem, ad, bd, IDESC, kb != wk.kb0 || k != 0 ? 1u : 0u);
        }
        mma_commit(empty_bar(stage), 3);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      mma_commit(tfull_bar(acc), 3);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    mma_commit(drain_bar, 1);
    volatile int zero = 0;
    mbar_wait(drain_bar, 0, &zero, late);
  } else if (warp >= 2) {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t my_stage = stage_out + (uint32_t)(warp - 2) * 4096u;
    int acc = 0;
    uint32_t acc_phase = 0, buf = 0;
    float sums[8], tops[8];  // M_LOGITS_T
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[i] = 0.0f;
      tops[i] = -INFINITY;
    }
    if constexpr (C::BOXES) tma_prefetch_desc(&tmC);
    while (wk.next(p)) {
      const HTile ti = htile<LISTED>(p, LISTED ? wk.mt : p.mt, wk.tile);
      const bool got = mbar_wait(tfull_bar(acc), acc_phase, abort_flag, p.err);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * TN);
      if constexpr (MODE == M_LOGITS) epi_logits(p, ti, (int)rank, tbase, q, lane, half);
      else if constexpr (MODE == M_U) epi_u(p, ti, wk.slab, (int)rank, tbase, q, lane, half);
      else if constexpr (MODE == M_LOGITS_T) epi_logits_t(p, tok, ti, (int)rank, tbase, q, lane, half, sums, tops);
      else if constexpr (MODE == M_U_T) epi_u_t(p, ti, wk.slab, (int)rank, tbase, q, lane, half);
      else epi_dw(p, &tmC, ti, (int)rank, tbase, q, lane, half, my_stage, buf);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(peer_addr(tempty_bar(acc), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if constexpr (C::BOXES) {
      if (lane == 0) bulk_wait_all();
    }
    if constexpr (MODE == M_LOGITS_T) {  // one part per CTA and lane quadrant
      if (p.psum && (lane & 3) == 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = 64 * half + 8 * i + lane / 4;
          const int64_t at = (int64_t)((pair * 2 + (int)rank) * 4 + q) * kFewRows + n;
          p.psum[at] = p.join ? p.psum[at] + sums[i] : sums[i];
          p.pmax[at] = p.join ? fmaxf(p.pmax[at], tops[i]) : tops[i];
        }
    }
  }

  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2u * TN) : "memory");
  }
}

// ref_i = <h_i, w_t>, the target's logit (of token 0 for a row without a target: any logit of the
// row serves as the reference).  One warp per row.
__global__ void __launch_bounds__(128) ce_ref_kernel(const __nv_bfloat16* __restrict__ h, int64_t ldh,
                                                     const __nv_bfloat16* __restrict__ w, int64_t ldw,
                                                     const int32_t* __restrict__ target, int64_t N, int d, int64_t V,
                                                     float* __restrict__ ref, float* __restrict__ zt,
                                                     int32_t* __restrict__ tcol, int32_t* hdr, int32_t* asked) {
  let_next_start();
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (threadIdx.x == 0 && row % kTile == 0) asked[row / kTile] = 0;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x < 64) hdr[threadIdx.x] = 0;  // nothing of this call has written it yet
  if (row >= N) return;
  const int32_t t = __ldg(target + row);
  const bool bad = t >= V;
  const int64_t v = t < 0 || bad ? 0 : t;
  const uint4* hr = reinterpret_cast<const uint4*>(h + row * ldh);
  const uint4* wr = reinterpret_cast<const uint4*>(w + v * ldw);
  float acc = 0.0f;
  for (int c = lane; c < d / 8; c += 32) {
    float a[8], b[8];
    unpack8(__ldg(hr + c), a);
    unpack8(__ldg(wr + c), b);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = fmaf(a[j], b[j], acc);
  }
  acc = warp_sum(acc);
  if (lane == 0) {
    ref[row] = zt[row] = acc;
    tcol[row] = (int32_t)v;
  }
}

// Per row, from the sweep's partial sums [parts, np]: the loss, lse and the factors of the gradients.
// A row whose largest logit lies over kMaxAbove above its reference asks for the second sweep (again =
// 0) of its tile: the first one to ask appends the tile to the list (asked: a word per tile, 0 or 1, then the list),
// whose order changes no result.  One block per 32 rows, its 32 warps taking the parts in turn.
__global__ void __launch_bounds__(1024) ce_stats_kernel(const int32_t* gate, const float* psum, const float* pmax,
                                                        int parts, int np, int64_t N,
                                                        const int32_t* __restrict__ target, int64_t V,
                                                        const float* __restrict__ g, const float* zt, float* ref,
                                                        float* mul, float* tval, float* loss, float* lse, int again,
                                                        int32_t* hdr, int32_t* asked) {
  let_next_start();
  wait_for_previous();
  if (gate && *gate == 0) return;
  __shared__ float ss[32][33], sm[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = (int64_t)blockIdx.x * 32;
  if (again && !asked[first / kTile]) return;  // its results stand
  float s = 0.0f, m = -INFINITY;
  if (first + lane < N)
#pragma unroll 4
    for (int i = warp; i < parts; i += 32) {
      s += psum[(int64_t)i * np + first + lane];
      m = fmaxf(m, pmax[(int64_t)i * np + first + lane]);
    }
  ss[warp][lane] = s;
  sm[warp][lane] = m;
  __syncthreads();
  const int64_t row = first + warp;  // from here a warp per row
  if (row >= N) return;
  s = warp_sum(ss[lane][warp]);
  m = warp_max(sm[lane][warp]);
  if (lane) return;
  const int32_t t = target[row];
  if (!again && t >= V) atomicOr(hdr, QAD_DEV_BAD_INDEX);
  const float r = ref[row], z = zt[row];
  if (!again && m - r > kMaxAbove && m < INFINITY) {  // an infinite logit gains nothing from it
    ref[row] = m;
    if (atomicExch(asked + row / kTile, 1) == 0) asked[(N + kTile - 1) / kTile + atomicAdd(hdr + 1, 1)] = (int32_t)(row / kTile);
    return;
  }
  const float et = expf(z - r);  // 1 unless the row's reference was replaced
  const float total = s + et;
  const float log_sum = r == z ? log1pf(s) : logf(total);
  const float l = (r - z) + log_sum;
  const bool live = t >= 0 && t < V;
  const float gi = live ? (g ? g[row] : 1.0f) : 0.0f;
  loss[row] = live ? l : 0.0f;
  lse[row] = r + log_sum;  // not by way of the target's logit, which may be far below
  // a row that carries no loss has a zero gradient whatever its logits are
  mul[row] = live ? gi / total : 0.0f;
  tval[row] = live ? -gi * (s / total) : 0.0f;
}

// dh_i = mul_i U_i + tval_i w_t (+ dh_i), U_i the sum over the slabs: one warp per row
__global__ void __launch_bounds__(128) ce_dh_kernel(const float* u, int slabs, const __nv_bfloat16* __restrict__ w,
                                                    int64_t ldw, const int32_t* tcol, const float* mul,
                                                    const float* tval, int64_t N, int d, int accumulate,
                                                    __nv_bfloat16* dh) {
  wait_for_previous();
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= N) return;
  const float a = mul[row], b = tval[row];
  const uint4* wr = reinterpret_cast<const uint4*>(w + (int64_t)tcol[row] * ldw);
  uint4* out = reinterpret_cast<uint4*>(dh + row * d);
  for (int c = 32 * blockIdx.y + lane; c < d / 8; c += 32 * gridDim.y) {
    const float* ur = u + row * d + 8 * c;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8];
#pragma unroll 4
    for (int s = 0; s < slabs; ++s) {
      const float4* at = reinterpret_cast<const float4*>(ur + (int64_t)s * N * d);
      const float4 u0 = at[0], u1 = at[1];
      x[0] += u0.x; x[1] += u0.y; x[2] += u0.z; x[3] += u0.w;
      x[4] += u1.x; x[5] += u1.y; x[6] += u1.z; x[7] += u1.w;
    }
    unpack8(__ldg(wr + c), v);
    // a row that carries no loss keeps its zero gradient whatever its logits were
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (a == 0.0f && b == 0.0f) ? 0.0f : a * x[j] + b * v[j];
    if (accumulate) {
      float o[8];
      unpack8(out[c], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += o[j];
    }
    out[c] = pack8(x);
  }
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// SM pairs that can run the kernel at the same time (its persistent grid)
template <int MODE, bool LISTED>
int head_pairs(cudaError_t* err) {
  auto kern = head_gemm_kernel<MODE, LISTED>;
  constexpr int SMEM = HCfg<MODE>::SMEM;
  static int max_pairs[64] = {0};  // per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!max_pairs[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) {
      *err = e;
      return 0;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2), 1, 1);
    cfg.blockDim = dim3(kThreadsH, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = num_sms() / 2;
    }
    max_pairs[dev] = n < kMaxPairs ? n : kMaxPairs;
  }
  return max_pairs[dev];
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

// *used (may be null): the pairs launched
template <int MODE, bool LISTED = false>
cudaError_t launch_head(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const HeadParams& p,
                        int kid, cudaStream_t st, int* used = nullptr) {
  cudaError_t e = cudaSuccess;
  const int most = head_pairs<MODE, LISTED>(&e);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.mt * p.nt * p.split;
  const int pairs = (int)(units < most ? units : most);
  if (used) *used = pairs;
  if (pairs < 1) return cudaSuccess;
  prof_begin(kid, st);
  e = launch_dependent(head_gemm_kernel<MODE, LISTED>, dim3((unsigned)(2 * pairs), 1, 1), kThreadsH, HCfg<MODE>::SMEM, st, ta, tb,
                       tc, p);
  prof_end(kid, st);
  return e;
}

constexpr size_t kPieceBytes = size_t(832) << 20;  // bound on the stored piece of exp(logits)
constexpr size_t kSlabBytes = size_t(192) << 20;   // and on the partial sums of U beyond the first

// Slabs that the product with the head is split into: fewer tiles than SM pairs, or a last round of tiles
// that fills few of them, leave pairs idle, which more and smaller units of work avoid; each slab is one
// more fp32 [N, d] written and read.  Costs in K blocks of one pair; a written and read tile is worth about
// kSlabCost of them.
int choose_slabs(int64_t tiles, int64_t num_kb, int64_t N, int64_t d) {
  constexpr double kSlabCost = 24.0;
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= 2 * kMaxPairs && s <= num_kb && (s == 1 || (s - 1) * 4.0 * N * d <= (double)kSlabBytes); ++s) {
    const double rounds = (double)((tiles * s + kMaxPairs - 1) / kMaxPairs);
    const double cost = rounds * ((double)num_kb / s + kSlabCost);
    if (s == 1 || cost < 0.99 * least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

size_t align_up(size_t v) { return (v + 1023) / 1024 * 1024; }

}  // namespace

int ce_layout_of(int64_t N, int64_t d, int64_t V, int grad, int dw, CeLayout* L) {
  if (N < 0 || d <= 0 || V <= 0) return QAD_ERR_INVALID_ARG;
  if (d % 16 || d > 65536 || V >= (int64_t(1) << 30) || N >= (int64_t(1) << 30)) return QAD_ERR_UNSUPPORTED;
  const bool few = N <= kFewRows;
  const int64_t width = few ? kFewRows : N;  // tokens in a row of the stored piece and of the partial sums
  // pieces of equal width (whole tiles) whose exp(logits) stay within kPieceBytes; one at least
  const int64_t vt = cdiv(V, kTile);
  int64_t most = (int64_t)(kPieceBytes / 2) / (kTile * width);
  if (most < 1) most = 1;
  L->pieces = (int)cdiv(vt, most);
  L->piece = (int)(cdiv(vt, L->pieces) * kTile);
  L->pieces = (int)cdiv(V, L->piece);
  const int64_t tiles = (few ? 1 : cdiv(N, kTile)) * cdiv(d, kTile);
  const int64_t bke = few ? HCfg<M_U_T>::BKE : HCfg<M_U>::BKE;
  L->slabs = tiles ? choose_slabs(tiles, cdiv(L->pieces > 1 ? L->piece : V, bke), N, d) : 1;
  // two parts per tile of a piece (transposed: eight per pair), which the pieces after the first add to
  L->parts = few ? kMaxPairs * 8 : 2 * (L->piece / kTile);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  L->header = take(256);
  L->asked = take(8 * (size_t)cdiv(N, kTile));
  L->ref = take(4 * (size_t)N);
  L->zt = take(4 * (size_t)N);
  L->tcol = take(4 * (size_t)N);
  L->mul = take(4 * (size_t)N);
  L->tval = take(4 * (size_t)N);
  L->psum = take(4 * (size_t)width * L->parts);
  L->pmax = take(4 * (size_t)width * L->parts);
  L->u = take(grad ? 4 * (size_t)L->slabs * (size_t)(N * d) : 0);
  L->p = take(grad || dw ? 2 * (size_t)width * L->piece : 0);
  L->total = o;
  return QAD_OK;
}

cudaError_t linear_ce(const CeLayout& L, const void* h, int64_t ldh, const void* w, int64_t ldw, const int32_t* target,
                      const float* g, float* loss, float* lse, void* dh, void* dw, int accumulate, int64_t N, int64_t d,
                      int64_t V, uint8_t* ws, cudaStream_t st) {
  int32_t* hdr = reinterpret_cast<int32_t*>(ws + L.header);
  int32_t* asked = reinterpret_cast<int32_t*>(ws + L.asked);
  float* ref = reinterpret_cast<float*>(ws + L.ref);
  float* zt = reinterpret_cast<float*>(ws + L.zt);
  int32_t* tcol = reinterpret_cast<int32_t*>(ws + L.tcol);
  float* mul = reinterpret_cast<float*>(ws + L.mul);
  float* tval = reinterpret_cast<float*>(ws + L.tval);
  float* psum = reinterpret_cast<float*>(ws + L.psum);
  float* pmax = reinterpret_cast<float*>(ws + L.pmax);
  float* u = reinterpret_cast<float*>(ws + L.u);
  void* ep = ws + L.p;
  const auto* hb = static_cast<const __nv_bfloat16*>(h);
  const auto* wb = static_cast<const __nv_bfloat16*>(w);
  const bool few = N <= kFewRows;
  const int64_t width = few ? kFewRows : N;
  cudaError_t e = cudaSuccess;
  // operands K-major for the logits; the head MN-major for U; e [token, piece] or, transposed, [piece, token]
  CUtensorMap tm_h, tm_w, tm_e, tm_wu, tm_hd, tm_ed, tm_dw;
  bool ok = make_tmap(&tm_h, h, d, N, ldh, few ? kFewRows / 2 : BM) && make_tmap(&tm_w, w, d, V, ldw, BM);
  if (ok && dh) {
    ok = make_tmap(&tm_wu, w, d, V, ldw, few ? HCfg<M_U_T>::BKE : HCfg<M_U>::BKE) &&
         (few ? make_tmap(&tm_e, ep, kFewRows, L.piece, kFewRows, HCfg<M_U_T>::BKE)
              : make_tmap(&tm_e, ep, L.piece, N, L.piece, BM));
  }
  if (ok && dw) {
    ok = make_tmap(&tm_hd, h, d, N, ldh, HCfg<M_DW>::BKE) && make_store_tmap(&tm_dw, dw, d, V, d) &&
         (few ? make_tmap(&tm_ed, ep, kFewRows, L.piece, kFewRows, BM)
              : make_tmap(&tm_ed, ep, L.piece, N, L.piece, HCfg<M_DW>::BKE));
  }
  if (!ok) return cudaErrorInvalidValue;
  note_launches(1);
  ce_ref_kernel<<<(unsigned)cdiv(N, 4), 128, 0, st>>>(hb, ldh, wb, ldw, target, N, (int)d, V, ref, zt, tcol, hdr,
                                                    asked);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  HeadParams base = {};
  base.err = hdr;
  base.N = N;
  base.d = (int)d;
  base.ref = ref;
  base.target = tcol;
  base.split = 1;
  int parts = 0;  // partial sums of the sweep
  auto logits = [&](int piece, const int32_t* gate, bool sums, bool store, bool final) -> cudaError_t {
    const int64_t c0 = (int64_t)piece * L.piece, cols = V - c0 < L.piece ? V - c0 : L.piece;
    HeadParams p = base;
    p.gate = gate;
    p.list = asked + cdiv(N, kTile);
    p.c0 = (int)c0;
    p.cols = (int)cols;
    p.num_kb = (int)cdiv(d, HCfg<M_LOGITS>::BKE);
    p.store_p = store;
    p.p = static_cast<__nv_bfloat16*>(ep);
    p.ldp = L.piece;
    if (sums) {
      p.psum = psum;
      p.pmax = pmax;
      p.join = piece > 0;
    }
    if (final) {  // normalised, with the target's column
      p.mul = mul;
      p.tval = tval;
    }
    if (few) {
      p.a_row0 = (int)c0;
      p.mt = (int)cdiv(cols, kTile);
      p.nt = 1;
      int pairs = 0;
      const cudaError_t e = launch_head<M_LOGITS_T>(tm_w, tm_h, tm_h, p, QAD_K_CE_LOGITS, st, &pairs);
      if (piece == 0) parts = pairs * 8;  // no later piece has more tiles
      return e;
    }
    p.b_row0 = (int)c0;
    p.mt = (int)cdiv(N, kTile);
    p.nt = (int)cdiv(cols, kTile);
    parts = L.parts;
    return gate ? launch_head<M_LOGITS, true>(tm_h, tm_w, tm_h, p, QAD_K_CE_LOGITS, st)
                : launch_head<M_LOGITS>(tm_h, tm_w, tm_h, p, QAD_K_CE_LOGITS, st);
  };
  auto product = [&](int piece, const int32_t* gate) -> cudaError_t {
    const int64_t c0 = (int64_t)piece * L.piece;
    // every piece is contracted over the same number of K blocks, so that its slabs are the same: the last
    // one's rows of the head past V read as zeros
    const int64_t cols = L.pieces > 1 ? L.piece : V;
    HeadParams q = base;
    q.gate = gate;
    q.list = asked + cdiv(N, kTile);
    q.nt = few ? 1 : (int)cdiv(d, kTile);
    q.mt = few ? (int)cdiv(d, kTile) : (int)cdiv(N, kTile);
    q.n_fast = 1;
    q.split = L.slabs;
    q.u = u;
    q.add = c0 > 0;
    q.num_kb = (int)cdiv(cols, few ? HCfg<M_U_T>::BKE : HCfg<M_U>::BKE);
    cudaError_t e;
    if (few) {
      q.a_row0 = (int)c0;
      e = launch_head<M_U_T>(tm_wu, tm_e, tm_e, q, QAD_K_CE_DH, st);
    } else {
      q.b_row0 = (int)c0;
      e = gate ? launch_head<M_U, true>(tm_e, tm_wu, tm_e, q, QAD_K_CE_DH, st)
               : launch_head<M_U>(tm_e, tm_wu, tm_e, q, QAD_K_CE_DH, st);
    }
    return e;
  };
  // the sweep: exp(logits) of a piece, then its product with the piece of the head
  auto sweep = [&](const int32_t* gate) -> cudaError_t {
    for (int i = 0; i < L.pieces; ++i) {
      cudaError_t e = logits(i, gate, true, dh != nullptr, false);
      if (e == cudaSuccess && dh) e = product(i, gate);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  };
  auto stats = [&](const int32_t* gate, int again) {
    note_launches(1);
    return launch_dependent(ce_stats_kernel, dim3((unsigned)cdiv(N, 32), 1, 1), 1024, 0, st, gate, psum, pmax, parts,
                            (int)width, N, target, V, g, zt, ref, mul, tval, loss, lse, again, hdr, asked);
  };
  if ((e = sweep(nullptr)) != cudaSuccess) return e;
  if ((e = stats(nullptr, 0)) != cudaSuccess) return e;
  if ((e = sweep(hdr + 1)) != cudaSuccess) return e;
  if ((e = stats(hdr + 1, 1)) != cudaSuccess) return e;
  if (dh) {
    note_launches(1);
    // few rows: a block column per 256 columns, so that their slabs are read side by side
    const dim3 grid((unsigned)cdiv(N, 4), few ? (unsigned)cdiv(d, 256) : 1u, 1);
    e = launch_dependent(ce_dh_kernel, grid, 128, 0, st, u, L.slabs, wb, ldw, tcol, mul, tval, N, (int)d, accumulate,
                         static_cast<__nv_bfloat16*>(dh));
    if (e != cudaSuccess) return e;
  }
  for (int i = 0; dw && i < L.pieces; ++i) {
    const int64_t c0 = (int64_t)i * L.piece, cols = V - c0 < L.piece ? V - c0 : L.piece;
    if ((e = logits(i, nullptr, false, true, true)) != cudaSuccess) return e;
    HeadParams q = base;
    q.c0 = (int)c0;
    q.cols = (int)cols;
    q.mt = (int)cdiv(cols, kTile);
    q.nt = (int)cdiv(d, kTile);
    q.n_fast = 1;
    q.num_kb = (int)cdiv(N, HCfg<M_DW>::BKE);
    e = few ? launch_head<M_DW_T>(tm_ed, tm_hd, tm_dw, q, QAD_K_CE_DW, st)
            : launch_head<M_DW>(tm_ed, tm_hd, tm_dw, q, QAD_K_CE_DW, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qad
