// The whole expert layer for a few tokens (generation): two launches, each of which reads the weights of the experts
// that some token names once, fake-quantizes them in registers and multiplies them there.
//
//   fc1:  Z1 = A1 . W13_hat^T, H = bf16(silu(gate) * up)             A1 = AQ(x)
//   fc2:  Y = AQ(H) . W2_hat^T, out[t] = bf16(sum_j p[t, j] * Y_j)
//
// With so few rows the weights are all there is to move (2 bytes an element and its part of a scale), and each element
// costs about seven instructions of fake-quantization whatever the number of tokens.  So the weights go straight from
// global memory to registers in the tensor cores' fragment layout: a lane loads 16 consecutive weights of a row (one
// 32-byte load, one quantization block), quantizes them, and four m16n8k16 products take them as they lie.  The order of
// k inside a product does not matter as long as both operands agree, so the tokens' rows (shared memory, up to 8
// columns) are read in the same order.  tcgen05 would want the quantized weights in shared memory first: a write and a
// read of every element for products that are idle most of the time here.
#include "common.cuh"
#include "internal.h"

namespace qad {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCols = 8;    // tokens of one expert that a pass over its weights serves
constexpr int kDepth = 4;   // chunks of a warp in flight
constexpr int kChunk = 64;  // elements along K of one step: 16 for each lane of a quad

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
  int aq, team, d_tiles;      // team: warps that share a tile
  bool wide;                  // weights on a 32-byte boundary
};

__host__ __device__ constexpr int few_stride(int K) { return (K + kChunk - 1) / kChunk * kChunk * 2 + 16; }

struct Route {
  uint64_t* mask;    // [E]: the tokens that name the expert
  uint32_t* live;    // [T]: the slots of a token that count
  uint16_t* first;   // [E + 1]: the expert's first pass (8 tokens each)
};

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
    for (int e = lo; e < hi; ++e) n += (__popcll(r.mask[e]) + kCols - 1) / kCols;
    int at = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (tid >= o) at += v;
    }
    at -= n;
    for (int e = lo; e < hi; ++e) {
      r.first[e] = (uint16_t)at;
      at += (__popcll(r.mask[e]) + kCols - 1) / kCols;
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

__device__ __forceinline__ void load16(const __nv_bfloat16* at, bool wide, uint32_t (&w)[8]) {
  uint4 lo, hi;
  if (wide) {
    ld_nc_256(at, lo, hi);
  } else {
    lo = __ldg(reinterpret_cast<const uint4*>(at));
    hi = __ldg(reinterpret_cast<const uint4*>(at) + 1);
  }
  w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
  w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
}

// One activation row through its quantizer into shared memory, by one warp; zeros behind K.
__device__ __forceinline__ void stage_row(const __nv_bfloat16* row, uint4* dst, int K, int aq, int lane) {
  const uint4* src = reinterpret_cast<const uint4*>(row);
  const int nblk = K / 16, padded = (K + kChunk - 1) / kChunk * (kChunk / 16);
  float s_row = 0.0f;
  if (act_needs_row(aq)) {
    float amax = 0.0f;
    for (int b = lane; b < nblk; b += 32) {
      float f[16];
      unpack8(src[2 * b], f);
      unpack8(src[2 * b + 1], f + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
    }
    amax = warp_max(amax);
    s_row = aq == kQE4M3   ? __fdiv_rn(amax, 448.0f)
            : aq == kQInt8 ? __fdiv_rn(amax, 127.0f)
                           : deploy_tensor_scale(__fdiv_rn(amax, 6.0f));
  }
  for (int b = lane; b < padded; b += 32) {
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (b < nblk) {
      u0 = src[2 * b];
      u1 = src[2 * b + 1];
      if (aq != kQNone) {
        float f[16];
        unpack8(u0, f);
        unpack8(u1, f + 8);
        if (aq == kQE4M3) {
          fakequant_act_inplace<kQE4M3, 16>(f, s_row);
        } else if (aq == kQInt8) {
          fakequant_act_inplace<kQInt8, 16>(f, s_row);
        } else {
          float amax = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
          float sc = __fdiv_rn(amax, 6.0f);
          if (aq == kQE2M1G) sc = deployed_scale(sc, s_row);
          fakequant_act_inplace<kQE2M1, 16>(f, sc);
        }
        u0 = pack8(f);
        u1 = pack8(f + 8);
      }
    }
    dst[2 * b] = u0;
    dst[2 * b + 1] = u1;
  }
}

// Tiles of 16 weight rows: fc1 8 gate rows and the 8 up rows that go with them, fc2 16 output rows.  A block takes a
// consecutive share of all (pass, tile) pairs, passes outermost, so that it stages few passes' tokens.
template <int WK, bool FC1>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(FewParams q) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_mask[1024];
  __shared__ uint32_t s_live[64];
  __shared__ uint16_t s_first[1025];
  __shared__ float s_part[2][kWarps][16][kCols];
  __shared__ int s_row[kCols], s_src[kCols];
  const Route r = {s_mask, s_live, s_first};
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane / 4, t4 = lane & 3;
  const int stride = few_stride(q.K), chunks = (q.K + kChunk - 1) / kChunk;
  const int team = q.team, my_team = warp / team, in_team = warp % team, teams = kWarps / team;
  const int tiles = FC1 ? q.N / 8 : q.N / 16;
  int err;
  const int passes = route(q, r, &err);
  if (FC1 && blockIdx.x == 0) {
    if (tid == 0) *q.err = err;
    for (int i = tid; i < q.d_tiles; i += kThreads) q.arrivals[i] = 0;
  }
  if (!FC1 && passes == 0) {  // every pair was dropped
    for (int i = blockIdx.x * kThreads + tid; i < q.T * q.N / 8; i += gridDim.x * kThreads)
      reinterpret_cast<uint4*>(q.out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t total = (int64_t)passes * tiles;
  const int lo = (int)(total * blockIdx.x / gridDim.x), hi = (int)(total * (blockIdx.x + 1) / gridDim.x);
  const int per_warp = (chunks + team - 1) / team;
  for (int u = lo; u < hi;) {
    const int pass = u / tiles, tile0 = u % tiles, ntiles = min(hi - u, tiles - tile0);
    u += ntiles;
    int e = 0;  // the last expert whose first pass is not behind this one
    for (int b = 512; b; b >>= 1)
      if (e + b < q.E && s_first[e + b] <= pass) e += b;
    const int mine = my_team < ntiles ? (ntiles - my_team + teams - 1) / teams : 0;
    const int steps = mine * per_warp;
    const __nv_bfloat16* we = q.w + (int64_t)e * (FC1 ? 2 * q.N : q.N) * q.K;
    const float* se = q.s + (int64_t)e * (FC1 ? 2 * q.N : q.N) * q.scales;

    uint32_t wa[kDepth][8], wb[kDepth][8];
    float sa[kDepth], sb[kDepth];
    int ld_tile = tile0 + my_team, ld_c = 0;  // the next step to load
    auto load = [&](int slot) {
      const int k0 = (ld_c * team + in_team) * kChunk + 16 * t4;
      const int ra = FC1 ? ld_tile * 8 + g : ld_tile * 16 + g, rb = FC1 ? q.N + ra : ra + 8;
      if (k0 < q.K) {
        load16(we + (int64_t)ra * q.K + k0, q.wide, wa[slot]);
        load16(we + (int64_t)rb * q.K + k0, q.wide, wb[slot]);
        if constexpr (WK != kQNone) {
          const int at = WK == kQE2M1 ? k0 / 16 : WK == kQInt4 ? k0 / 128 : 0;
          sa[slot] = __ldg(se + (int64_t)ra * q.scales + at);
          sb[slot] = __ldg(se + (int64_t)rb * q.scales + at);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) wa[slot][i] = wb[slot][i] = 0;
        sa[slot] = sb[slot] = 0.0f;
      }
      if (++ld_c == per_warp) {
        ld_c = 0;
        ld_tile += teams;
      }
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
      if (i < steps) load(i);

    __syncthreads();  // the tokens of the segment before are no longer read
    if (tid < kCols) {
      uint64_t m = s_mask[e];
      for (int i = (pass - s_first[e]) * kCols + tid; i > 0 && m; --i) m &= m - 1;
      int row = -1, src = -1;
      if (m) {
        const int t = __ffsll((long long)m) - 1;
        for (int j = 0; j < q.k; ++j)
          if ((s_live[t] >> j & 1) && __ldg(q.idx + t * q.k + j) == e) row = t * q.k + j;
        src = FC1 ? t : row;
      }
      s_row[tid] = row;
      s_src[tid] = src;
    }
    __syncthreads();
    if (s_src[warp] >= 0)
      stage_row(q.act + (int64_t)s_src[warp] * q.K, reinterpret_cast<uint4*>(smem + warp * stride), q.K, q.aq, lane);
    __syncthreads();

    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int c = 0, tile = tile0 + my_team, parity = 0;
    for (int base = 0; base < steps; base += kDepth) {
#pragma unroll
      for (int slot = 0; slot < kDepth; ++slot) {
        if (base + slot >= steps) break;
        const int chunk = c * team + in_team;
        if (chunk < chunks) {
          const uint4* xs = reinterpret_cast<const uint4*>(smem + g * stride + (chunk * kChunk + 16 * t4) * 2);
          const uint4 x0 = xs[0], x1 = xs[1];
          uint32_t a[8], b[8];
          if constexpr (WK == kQNone) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              a[i] = wa[slot][i];
              b[i] = wb[slot][i];
            }
          } else {
            fakequant16_packed<WK>(wa[slot], sa[slot], a);
            fakequant16_packed<WK>(wb[slot], sb[slot], b);
          }
          mma_bf16(acc, a[0], b[0], a[1], b[1], x0.x, x0.y);
          mma_bf16(acc, a[2], b[2], a[3], b[3], x0.z, x0.w);
          mma_bf16(acc, a[4], b[4], a[5], b[5], x1.x, x1.y);
          mma_bf16(acc, a[6], b[6], a[7], b[7], x1.z, x1.w);
        }
        if (base + slot + kDepth < steps) load(slot);
        if (++c < per_warp) continue;
        // the tile's end: the team's partial sums are joined in warp order
        c = 0;
        float(*part)[kCols] = s_part[parity][warp];
        part[g][2 * t4] = acc[0];
        part[g][2 * t4 + 1] = acc[1];
        part[g + 8][2 * t4] = acc[2];
        part[g + 8][2 * t4 + 1] = acc[3];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + my_team), "r"(32 * team) : "memory");
        const float(*sum)[16][kCols] = &s_part[parity][my_team * team];
        for (int i = in_team * 32 + lane; i < (FC1 ? 64 : 128); i += 32 * team) {
          if constexpr (FC1) {
            const int col = i / 8, n = i % 8;
            if (s_row[col] >= 0) {
              float zg = 0.0f, zu = 0.0f;
              for (int w = 0; w < team; ++w) {
                zg += sum[w][n][col];
                zu += sum[w][n + 8][col];
              }
              q.rows[(int64_t)s_row[col] * q.N + tile * 8 + n] =
                  __float2bfloat16_rn(__fmul_rn(silu_f(round_bf16(zg)), round_bf16(zu)));
            }
          } else {
            const int col = i / 16, n = i % 16;
            if (s_row[col] >= 0) {
              float y = 0.0f;
              for (int w = 0; w < team; ++w) y += sum[w][n][col];
              q.rows[(int64_t)s_row[col] * q.N + tile * 16 + n] = __float2bfloat16_rn(y);
            }
          }
        }
        parity ^= 1;
        acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
        tile += teams;
      }
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
  for (int w = kWarps; w > 1; w /= 2)
    if ((chunks + w - 1) / w * w * 8 <= chunks * 9) return w;
  return 1;
}

template <int WK, bool FC1>
cudaError_t launch(const FewParams& q, int64_t units, cudaStream_t st) {
  const int bytes = kCols * few_stride(q.K);
  if (cudaError_t e = cudaFuncSetAttribute(few_kernel<WK, FC1>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))
    return e;
  const int64_t slots = 2 * (int64_t)num_sms();
  few_kernel<WK, FC1><<<(unsigned)(units < slots ? units : slots), kThreads, bytes, st>>>(q);
  return cudaGetLastError();
}

template <bool FC1>
cudaError_t launch_kind(int kind, const FewParams& q, int64_t units, cudaStream_t st) {
  switch (kind) {
    case kQE2M1: return launch<kQE2M1, FC1>(q, units, st);
    case kQInt4: return launch<kQInt4, FC1>(q, units, st);
    case kQE4M3: return launch<kQE4M3, FC1>(q, units, st);
    case kQInt8: return launch<kQInt8, FC1>(q, units, st);
    default: return launch<kQNone, FC1>(q, units, st);
  }
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
  q.aq = quant ? act_kind(s.fmt) : kQNone;
  q.d_tiles = (int)(s.d / 16);
  const int64_t pairs = s.T * s.topk;  // no more passes than pairs
  auto wide = [](const void* w) { return (reinterpret_cast<uintptr_t>(w) & 31u) == 0; };

  q.act = static_cast<const __nv_bfloat16*>(x);
  q.w = static_cast<const __nv_bfloat16*>(w13);
  q.s = s13;
  q.rows = reinterpret_cast<__nv_bfloat16*>(ws + L.h);
  q.K = (int)s.d;
  q.N = (int)s.F;
  q.scales = block ? q.K / block : 1;
  q.team = team_of(q.K);
  q.wide = wide(w13);
  prof_begin(QAD_K_MOE_FEW, st);
  cudaError_t e = launch_kind<true>(kind, q, pairs * (q.N / 8), st);
  if (e == cudaSuccess) {
    q.act = reinterpret_cast<const __nv_bfloat16*>(ws + L.h);
    q.w = static_cast<const __nv_bfloat16*>(w2);
    q.s = s2;
    q.rows = reinterpret_cast<__nv_bfloat16*>(ws + L.y);
    q.K = (int)s.F;
    q.N = (int)s.d;
    q.scales = block ? q.K / block : 1;
    q.team = team_of(q.K);
    q.wide = wide(w2);
    note_launches(1);
    e = launch_kind<false>(kind, q, pairs * (q.N / 16), st);
  }
  prof_end(QAD_K_MOE_FEW, st);
  return e;
}

}  // namespace qad
