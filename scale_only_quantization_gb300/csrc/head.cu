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
// and (q_t - 1) w_t is added in fp32.  e may be far above 1 (bf16 has fp32's range): only a row
// whose largest logit is over kMaxAbove nats above its target's is swept again, with the largest
// as its reference (the second sweep's kernels leave at once when no row asked for it).
// dW needs the final normaliser, so its pieces are computed from the logits a second time.
//
// The products run on SM pairs (tcgen05 cta_group::2, 256 x 256 tiles) with the roles and
// barriers of the grouped GEMMs: warp 0 of each CTA loads, warp 1 of the leader issues the MMAs,
// warps 2-9 run the epilogue of one accumulator while the other is filled.
#include "internal.h"
#include "tcgen05.cuh"

namespace qad {
namespace {

constexpr int kTile = 256;            // rows and columns of a pair tile
constexpr int kThreadsH = 320;
constexpr int kEpiWarps = 8;
constexpr float kMaxAbove = 60.0f;    // exp(60) summed over 2^31 columns stays below fp32's range

enum { M_LOGITS = 0, M_U = 1, M_DW = 2 };

struct HeadParams {
  const int32_t* gate;  // null, or a word: 0 = nothing to do
  int32_t* err;
  int mt, nt, num_kb;   // tiles along the output's rows and columns, K blocks
  int n_fast;           // tile order: columns fastest
  int a_row0, b_row0;   // first row of the A / B tensors of this piece
  int64_t N;            // token rows
  // logits: columns c0 .. c0 + cols of the vocabulary
  int c0, cols;
  const float *ref, *mul;       // per row: reference, factor (null: 1)
  const float* tval;            // per row: what the target's column holds (null: 0)
  const int32_t* target;        // per row: the target's column
  float *psum, *pmax;           // [column halves of tiles, N] sums without the target / maxima, or null
  int store_p;
  // U
  float* u;
  int d, add;
};

template <int MODE> struct HCfg {
  static constexpr bool A_MN = MODE == M_DW, B_MN = MODE != M_LOGITS;
  static constexpr int ATOMS = MODE == M_U ? 1 : 2;
  static constexpr int BKE = ATOMS * BK;
  static constexpr int A_ATOM = BM * 128, B_ATOM = BM * 128;
  static constexpr int A_BYTES = ATOMS * A_ATOM, B_BYTES = ATOMS * B_ATOM;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = (192 * 1024) / STAGE;
  static constexpr int STAGING = MODE == M_U ? 0 : kEpiWarps * 4096;
  static constexpr int SMEM = STAGES * STAGE + 512 + 1024 + STAGING;
};

struct HTile {
  int mb, nb;
};
__device__ __forceinline__ HTile htile(const HeadParams& p, int t) {
  HTile x;
  if (p.n_fast) {
    x.mb = t / p.nt;
    x.nb = t - x.mb * p.nt;
  } else {
    x.nb = t / p.mt;
    x.mb = t - x.nb * p.mt;
  }
  return x;
}

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

// Row r's 128 columns of a logits tile: e = exp(z - ref) (x factor), its sum without the target,
// the largest logit, and the bf16 piece for the product that follows.
__device__ __forceinline__ void epi_logits(const HeadParams& p, const CUtensorMap* tm, const HTile& ti, int rank,
                                           uint32_t tbase, int q, int lane, int half, uint32_t stage_base,
                                           uint32_t& buf) {
  const int y = ti.mb * kTile + rank * BM + 32 * q;
  const int64_t row = y + lane;
  const bool live = row < p.N;
  const float ref = live ? __ldg(p.ref + row) : 0.0f;
  const float mul = live && p.mul ? __ldg(p.mul + row) : 1.0f;
  const float tv = live && p.tval ? __ldg(p.tval + row) : 0.0f;
  const int col0 = ti.nb * kTile + half * 128;  // within the piece
  const int target = live ? __ldg(p.target + row) - p.c0 - col0 : -1;  // within these 128 columns
  const bool edge = col0 + 128 > p.cols;
  float sum = 0.0f, top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld32_issue(tbase + half * 128 + 32 * c, r);
    tmem_wait32(r);
    const int tc = target - 32 * c;
    const int valid = p.cols - (col0 + 32 * c);
    uint4 out[4];
    uint32_t* o = reinterpret_cast<uint32_t*>(out);
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
    if (p.store_p && y < p.N) store_box32(tm, stage_base, buf, lane, out, col0 + 32 * c, y);
  }
  if (p.psum && live) {
    const int64_t at = (int64_t)((p.c0 / kTile + ti.nb) * 2 + half) * p.N + row;
    p.psum[at] = sum;
    p.pmax[at] = top;
  }
}

// Row r's 128 columns of U += e W, fp32 in global memory
__device__ __forceinline__ void epi_u(const HeadParams& p, const HTile& ti, int rank, uint32_t tbase, int q, int lane,
                                      int half) {
  const int64_t row = ti.mb * kTile + rank * BM + 32 * q + lane;
  const int col0 = ti.nb * kTile + half * 128;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld32_issue(tbase + half * 128 + 32 * c, r);
    tmem_wait32(r);
    float4* u = reinterpret_cast<float4*>(p.u + row * p.d + col0 + 32 * c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (row >= p.N || col0 + 32 * c + 4 * i >= p.d) continue;
      float4 v = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), __uint_as_float(r[4 * i + 2]),
                             __uint_as_float(r[4 * i + 3]));
      if (p.add) {
        const float4 w = u[i];
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      u[i] = v;
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

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsH, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const HeadParams p) {
  using C = HCfg<MODE>;
  constexpr int STAGES = C::STAGES, BKE = C::BKE, ATOMS = C::ATOMS;
  constexpr uint32_t IDESC = instr_desc<kTile, C::A_MN, C::B_MN>();
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
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2u * kTile)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = p.mt * p.nt;
  const int first = (int)cluster_id(), step = (int)cluster_count();

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    const int half = (int)rank * BM;
    for (int t = first; ok && t < total; t += step) {
      const HTile ti = htile(p, t);
      for (int kb = 0; kb < p.num_kb; ++kb) {
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
        for (int i = 0; i < (C::B_MN ? 2 : ATOMS); ++i) {
          if constexpr (C::B_MN)
            tma_load_2d(sb + i * BKE * 128, &tmB, ti.nb * kTile + half + i * 64, p.b_row0 + kb * BKE, fb);
          else
            tma_load_2d(sb + i * C::B_ATOM, &tmB, kb * BKE + i * BK, p.b_row0 + ti.nb * kTile + half, fb);
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
    for (int t = first; ok && t < total; t += step) {
      if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kTile);
      for (int kb = 0; kb < p.num_kb; ++kb) {
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
          mma_issue<false>(d_tmem, ad, bd, IDESC, (kb | k) != 0 ? 1u : 0u);
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
    if constexpr (MODE != M_U) tma_prefetch_desc(&tmC);
    for (int t = first; t < total; t += step) {
      const HTile ti = htile(p, t);
      const bool got = mbar_wait(tfull_bar(acc), acc_phase, abort_flag, p.err);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kTile);
      if constexpr (MODE == M_LOGITS) epi_logits(p, &tmC, ti, (int)rank, tbase, q, lane, half, my_stage, buf);
      else if constexpr (MODE == M_U) epi_u(p, ti, (int)rank, tbase, q, lane, half);
      else epi_dw(p, &tmC, ti, (int)rank, tbase, q, lane, half, my_stage, buf);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(peer_addr(tempty_bar(acc), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if constexpr (MODE != M_U) {
      if (lane == 0) bulk_wait_all();
    }
  }

  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2u * kTile) : "memory");
  }
}

// ref_i = <h_i, w_t>, the target's logit (of token 0 for a row without a target: any logit of the
// row serves as the reference).  One warp per row.
__global__ void __launch_bounds__(128) ce_ref_kernel(const __nv_bfloat16* __restrict__ h, int64_t ldh,
                                                     const __nv_bfloat16* __restrict__ w, int64_t ldw,
                                                     const int32_t* __restrict__ target, int64_t N, int d, int64_t V,
                                                     float* __restrict__ ref, float* __restrict__ zt,
                                                     int32_t* __restrict__ tcol, int32_t* hdr) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
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
    if (bad) atomicOr(hdr, QAD_DEV_BAD_INDEX);
  }
}

// Per row, from the sweep's partial sums: the loss, lse and the factors of the gradients.  A row
// whose largest logit lies over kMaxAbove above its reference asks for the second sweep (again = 0).
// One block per 32 rows, its 8 warps taking the parts in turn.
__global__ void __launch_bounds__(256) ce_stats_kernel(const int32_t* gate, const float* __restrict__ psum,
                                                       const float* __restrict__ pmax, int parts, int64_t N,
                                                       const int32_t* __restrict__ target, int64_t V,
                                                       const float* __restrict__ g, const float* __restrict__ zt,
                                                       float* __restrict__ ref, float* __restrict__ mul,
                                                       float* __restrict__ tval, float* __restrict__ loss,
                                                       float* __restrict__ lse, int again, int32_t* request) {
  if (gate && *gate == 0) return;
  __shared__ float ss[8][32], sm[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f, m = -INFINITY;
  if (row < N)
    for (int i = warp; i < parts; i += 8) {
      s += psum[(int64_t)i * N + row];
      m = fmaxf(m, pmax[(int64_t)i * N + row]);
    }
  ss[warp][lane] = s;
  sm[warp][lane] = m;
  __syncthreads();
  if (warp || row >= N) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    s += ss[i][lane];
    m = fmaxf(m, sm[i][lane]);
  }
  const float r = ref[row], z = zt[row];
  if (!again && m - r > kMaxAbove && m < INFINITY) {  // an infinite logit gains nothing from it
    ref[row] = m;
    atomicOr(request, 1);
    return;
  }
  const float et = expf(z - r);  // 1 unless the row's reference was replaced
  const float total = s + et;
  const float l = (r - z) + (r == z ? log1pf(s) : logf(total));
  const int32_t t = target[row];
  const bool live = t >= 0 && t < V;
  const float gi = live ? (g ? g[row] : 1.0f) : 0.0f;
  loss[row] = live ? l : 0.0f;
  lse[row] = z + l;
  // a row that carries no loss has a zero gradient whatever its logits are
  mul[row] = live ? gi / total : 0.0f;
  tval[row] = live ? -gi * (s / total) : 0.0f;
}

// dh_i = mul_i U_i + tval_i w_t (+ dh_i): one warp per row
__global__ void __launch_bounds__(128) ce_dh_kernel(const float* __restrict__ u, const __nv_bfloat16* __restrict__ w,
                                                    int64_t ldw, const int32_t* __restrict__ tcol,
                                                    const float* __restrict__ mul, const float* __restrict__ tval,
                                                    int64_t N, int d, int accumulate, __nv_bfloat16* dh) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= N) return;
  const float a = __ldg(mul + row), b = __ldg(tval + row);
  const uint4* wr = reinterpret_cast<const uint4*>(w + (int64_t)__ldg(tcol + row) * ldw);
  const float4* ur = reinterpret_cast<const float4*>(u + row * d);
  uint4* out = reinterpret_cast<uint4*>(dh + row * d);
  for (int c = lane; c < d / 8; c += 32) {
    const float4 u0 = ur[2 * c], u1 = ur[2 * c + 1];
    float v[8], x[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
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

template <int MODE>
cudaError_t launch_head(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const HeadParams& p,
                        int kid, cudaStream_t st) {
  auto kern = head_gemm_kernel<MODE>;
  constexpr int SMEM = HCfg<MODE>::SMEM;
  static int max_pairs[64] = {0};  // per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!max_pairs[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2), 1, 1);
    cfg.blockDim = dim3(kThreadsH, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = num_sms() / 2;
    }
    max_pairs[dev] = n;
  }
  const int64_t tiles = (int64_t)p.mt * p.nt;
  const int64_t pairs = tiles < max_pairs[dev] ? tiles : max_pairs[dev];
  if (pairs < 1) return cudaSuccess;
  prof_begin(kid, st);
  kern<<<(unsigned)(2 * pairs), kThreadsH, SMEM, st>>>(ta, tb, tc, p);
  prof_end(kid, st);
  return cudaGetLastError();
}

constexpr size_t kPieceBytes = size_t(1) << 30;  // bound on the stored piece of exp(logits)

size_t align_up(size_t v) { return (v + 1023) / 1024 * 1024; }

}  // namespace

int ce_layout_of(int64_t N, int64_t d, int64_t V, int grad, int dw, CeLayout* L) {
  if (N < 0 || d <= 0 || V <= 0) return QAD_ERR_INVALID_ARG;
  if (d % 16 || d > 65536 || V >= (int64_t(1) << 30) || N >= (int64_t(1) << 30)) return QAD_ERR_UNSUPPORTED;
  L->parts = (int)(2 * cdiv(V, kTile));
  // pieces of equal width (whole tiles) whose exp(logits) stay within kPieceBytes; one at least
  const int64_t vt = cdiv(V, kTile);
  int64_t most = (int64_t)(kPieceBytes / 2) / (kTile * (N > 0 ? N : 1));
  if (most < 1) most = 1;
  const int64_t pieces = cdiv(vt, most);
  L->piece = (int)(cdiv(vt, pieces) * kTile);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  L->header = take(256);
  L->ref = take(4 * (size_t)N);
  L->zt = take(4 * (size_t)N);
  L->tcol = take(4 * (size_t)N);
  L->mul = take(4 * (size_t)N);
  L->tval = take(4 * (size_t)N);
  L->psum = take(4 * (size_t)N * L->parts);
  L->pmax = take(4 * (size_t)N * L->parts);
  L->u = take(grad ? 4 * (size_t)(N * d) : 0);
  L->p = take(grad || dw ? 2 * (size_t)N * L->piece : 0);
  L->total = o;
  return QAD_OK;
}

cudaError_t linear_ce(const CeLayout& L, const void* h, int64_t ldh, const void* w, int64_t ldw, const int32_t* target,
                      const float* g, float* loss, float* lse, void* dh, void* dw, int accumulate, int64_t N, int64_t d,
                      int64_t V, uint8_t* ws, cudaStream_t st) {
  int32_t* hdr = reinterpret_cast<int32_t*>(ws + L.header);
  float* ref = reinterpret_cast<float*>(ws + L.ref);
  float* zt = reinterpret_cast<float*>(ws + L.zt);
  int32_t* tcol = reinterpret_cast<int32_t*>(ws + L.tcol);
  float* mul = reinterpret_cast<float*>(ws + L.mul);
  float* tval = reinterpret_cast<float*>(ws + L.tval);
  float* psum = reinterpret_cast<float*>(ws + L.psum);
  float* pmax = reinterpret_cast<float*>(ws + L.pmax);
  float* u = reinterpret_cast<float*>(ws + L.u);
  const auto* hb = static_cast<const __nv_bfloat16*>(h);
  const auto* wb = static_cast<const __nv_bfloat16*>(w);
  cudaError_t e = cudaMemsetAsync(hdr, 0, 256, st);
  if (e != cudaSuccess) return e;
  CUtensorMap th, tw, tps, tp, tw_mn, th_mn, tp_mn, tdw;
  if (!make_tmap(&th, h, d, N, ldh, BM) || !make_tmap(&tw, w, d, V, ldw, BM)) return cudaErrorInvalidValue;
  tps = th;
  if (dh || dw) {
    if (!make_store_tmap(&tps, ws + L.p, L.piece, N, L.piece) || !make_tmap(&tp, ws + L.p, L.piece, N, L.piece, BM) ||
        !make_tmap(&tw_mn, w, d, V, ldw, HCfg<M_U>::BKE))
      return cudaErrorInvalidValue;
  }
  if (dw) {
    if (!make_tmap(&th_mn, h, d, N, ldh, HCfg<M_DW>::BKE) ||
        !make_tmap(&tp_mn, ws + L.p, L.piece, N, L.piece, HCfg<M_DW>::BKE) || !make_store_tmap(&tdw, dw, d, V, d))
      return cudaErrorInvalidValue;
  }
  note_launches(2);
  ce_ref_kernel<<<(unsigned)cdiv(N, 4), 128, 0, st>>>(hb, ldh, wb, ldw, target, N, (int)d, V, ref, zt, tcol, hdr);

  HeadParams base = {};
  base.err = hdr;
  base.N = N;
  base.d = (int)d;
  base.ref = ref;
  base.target = tcol;
  auto logits = [&](int64_t c0, int64_t cols) {
    HeadParams p = base;
    p.c0 = p.b_row0 = (int)c0;
    p.cols = (int)cols;
    p.mt = (int)cdiv(N, kTile);
    p.nt = (int)cdiv(cols, kTile);
    p.num_kb = (int)cdiv(d, HCfg<M_LOGITS>::BKE);
    return p;
  };
  // the sweep: exp(logits) of a piece, then its product with the piece of the head
  auto sweep = [&](const int32_t* gate) -> cudaError_t {
    for (int64_t c0 = 0; c0 < V; c0 += L.piece) {
      const int64_t cols = V - c0 < L.piece ? V - c0 : L.piece;
      HeadParams p = logits(c0, cols);
      p.gate = gate;
      p.psum = psum;
      p.pmax = pmax;
      p.store_p = dh != nullptr;
      cudaError_t e = launch_head<M_LOGITS>(th, tw, tps, p, QAD_K_CE_LOGITS, st);
      if (e != cudaSuccess) return e;
      if (!dh) continue;
      HeadParams q = base;
      q.gate = gate;
      q.b_row0 = (int)c0;
      q.mt = (int)cdiv(N, kTile);
      q.nt = (int)cdiv(d, kTile);
      q.n_fast = 1;
      q.num_kb = (int)cdiv(cols, HCfg<M_U>::BKE);
      q.u = u;
      q.add = c0 > 0;
      e = launch_head<M_U>(tp, tw_mn, tp, q, QAD_K_CE_DH, st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  };
  auto stats = [&](const int32_t* gate, int again) {
    ce_stats_kernel<<<(unsigned)cdiv(N, 32), 256, 0, st>>>(gate, psum, pmax, L.parts, N, target, V, g, zt, ref, mul,
                                                            tval, loss, lse, again, hdr + 1);
    note_launches(1);
    return cudaGetLastError();
  };
  if ((e = sweep(nullptr)) != cudaSuccess) return e;
  if ((e = stats(nullptr, 0)) != cudaSuccess) return e;
  if ((e = sweep(hdr + 1)) != cudaSuccess) return e;
  if ((e = stats(hdr + 1, 1)) != cudaSuccess) return e;
  if (dh) {
    note_launches(1);
    ce_dh_kernel<<<(unsigned)cdiv(N, 4), 128, 0, st>>>(u, wb, ldw, tcol, mul, tval, N, (int)d, accumulate,
                                                        static_cast<__nv_bfloat16*>(dh));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (dw) {
    for (int64_t c0 = 0; c0 < V; c0 += L.piece) {
      const int64_t cols = V - c0 < L.piece ? V - c0 : L.piece;
      HeadParams p = logits(c0, cols);
      p.mul = mul;
      p.tval = tval;
      p.store_p = 1;
      if ((e = launch_head<M_LOGITS>(th, tw, tps, p, QAD_K_CE_LOGITS, st)) != cudaSuccess) return e;
      HeadParams q = base;
      q.c0 = (int)c0;
      q.cols = (int)cols;
      q.mt = (int)cdiv(cols, kTile);
      q.nt = (int)cdiv(d, kTile);
      q.n_fast = 1;
      q.num_kb = (int)cdiv(N, HCfg<M_DW>::BKE);
      if ((e = launch_head<M_DW>(tp_mn, th_mn, tdw, q, QAD_K_CE_DW, st)) != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace qad
