// Residual addition + root-mean-square norm of token rows, with the activation quantizers of the
// per-row grids (E4M3, INT8) on its output, and the norm's gradient.
//
//   r = bf16(x + res)            the residual stream is stored in bf16, and the norm reads it as stored
//   rstd = 1 / sqrt(mean(r^2) + eps)
//   y = bf16(r * rstd * gamma)   the value the router, the layer and its quantizer read
//   s = fp32(max |y| / Qmax), code = q(y / s), y_hat = bf16(q(y / s) * s)   as the layer's own AQ
// Backward (straight through the quantizer), n = r * rstd, dn = dy * gamma:
//   dx = rstd * (dn - n * mean(dn * n)) + dres,   dgamma = sum over rows of dy * n
// All sums are fp32.  One pass over the data: a row stays in registers between its reductions, so
// both directions are bound by HBM.  16384 x 2048: forward with residual, y and E4M3 codes 49 us for 302 MB
// (6.1 TB/s), backward with the residual's gradient and dgamma 49.4 us for 268 MB: 6.9 TB/s between 8192 and 16384
// rows, 6 us of launch and first rows, 4.5 us for the sum of the partial weight gradients.  Rows wider than 4096 go
// without the ring, one block of the backward per SM: 8192 x 8192 takes 99.6 us (5.4 TB/s), 4096 x 16384 155 us
// (3.5 TB/s, with 76 to 228 bytes of spills); their forward 53.6 us for 4096 x 8192 (5.6 TB/s).
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace qad {
namespace {

// unpack8 by byte moves.  The second use of a row's values unpacks them by other instructions than the
// first: with the same ones the compiler keeps the unpacked values in between, twice the registers.
__device__ __forceinline__ void unpack8_again(const uint4& u, float* f) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(__byte_perm(x[i], 0, 0x1044));
    f[2 * i + 1] = __uint_as_float(__byte_perm(x[i], 0, 0x3244));
  }
}

struct NormFwd {
  const __nv_bfloat16 *x, *res, *gamma;
  __nv_bfloat16 *r, *y, *y_hat;
  uint8_t* codes;
  float *scale, *rstd;
  int64_t T, ldx, ldres;
  int nv, d;  // 16-byte vectors of a row, and its elements
  float eps, inv_d;
};

// Sum over the W warps that share a row; every thread of the group returns it.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* smem, int warp_in_row, int lane, int bar) {
  v = warp_sum(v);
  if constexpr (W > 1) {
    if (lane == 0) smem[warp_in_row] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * W) : "memory");
    v = smem[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v += smem[i];
  }
  return v;
}

// max |y| of a row from its bf16 bits: without their signs, magnitudes compare as integers, two per word, and a NaN
// is above infinity, so that neither is lost on the way to the scale (fmaxf would drop a NaN).
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t pair) { return __vmaxu2(m, pair & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t warp_max_bits(uint32_t m) {
  return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
}
__device__ __forceinline__ float magnitude(uint32_t bits) { return __uint_as_float(bits << 16); }

// rstd from the row's mean square; scaled_mean(f) is that of f r.  Squares that leave fp32's range, at the top (|r| >
// 1e19 / sqrt(d)) or, where next to no eps covers it, at the bottom, are taken again of scaled values: 2^-64 r or 2^100 r.
// A row of zeros without eps has rstd 0, so that y and the gradient are 0; below an rms of 3e-39, whose reciprocal fp32
// does not hold, rstd stays at fp32's largest value.
template <typename F>
__device__ __forceinline__ float inverse_rms(float mean, float eps, F scaled_mean) {
  if (mean == INFINITY || mean + eps < 0x1p-100f) {
    const float f = mean == INFINITY ? 0x1p-64f : 0x1p100f;
    const float s = scaled_mean(f) + eps * f * f;
    return s == 0.0f ? 0.0f : fminf(__fdiv_rn(1.0f, __fsqrt_rn(s)) * f, 3.402823466e38f);
  }
  return __fdiv_rn(1.0f, __fsqrt_rn(mean + eps));
}

// The layer's activation quantizer on 4 values of scale s: their codes, and code value * s in place
template <int KIND>
__device__ __forceinline__ void quantize4(float* a, float s, uint32_t& code) {
  if constexpr (KIND == kQE4M3) {
    uint32_t c[1];
    fakequant_e4m3_codes<4, true>(a, s, c);
    code = c[0];
  } else {
    float x[4];
    act_quotients<4>(a, s, x);
    const float by = s < INFINITY ? s : NAN;  // no INT8 code stands for a NaN quotient: its y_hat says it
    code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = q_int8(x[j]);
      code |= ((uint32_t)(int)q & 0xffu) << (8 * j);
      a[j] = __fmul_rn(copysignf(q, x[j]), by);
    }
  }
}

// Two bf16 pairs (8 bytes) <-> 4 floats
__device__ __forceinline__ void unpack4(const uint2& u, float* f) {
  f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
}
__device__ __forceinline__ uint2 pack4(const float* f) { return make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])); }

// The squares of bf16 values are exact in fp32, so rstd depends on the order of their sum alone.  Up to 4096
// elements that order is fixed: 128 chains (element i in chain i % 128), the four of a group one after the
// other, then the 32 groups pairwise, whatever the kernel that takes the row (and as an evaluation in elementary fp32
// operations sums a row on this GPU); wider rows are summed in their lanes' own order.  A last place of rstd moves y by
// a bf16 step now and then and with it, in the row's largest element, the scale.  The scale is the quotient by
// 448 or 127, as the layer's is: a product with the rounded reciprocal differs in the last place for half the rows.

// Rows of up to 1024 elements: one warp per row, no barrier; lane l keeps the 4-element groups l, l + 32, ...
template <int G, int KIND>
__global__ void __launch_bounds__(128) rmsnorm_fwd_warp_kernel(const NormFwd p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int ng = p.d / 4;  // groups of a row
  if (row >= p.T) return;
  const uint2* xr = reinterpret_cast<const uint2*>(p.x + row * p.ldx);
  const uint2 zero = make_uint2(0, 0);
  uint2 v[G];
#pragma unroll
  for (int i = 0; i < G; ++i) v[i] = lane + 32 * i < ng ? __ldcs(xr + lane + 32 * i) : zero;
  if (p.res) {
    const uint2* rr = reinterpret_cast<const uint2*>(p.res + row * p.ldres);
    uint2 u[G];
#pragma unroll
    for (int i = 0; i < G; ++i) u[i] = lane + 32 * i < ng ? __ldcs(rr + lane + 32 * i) : zero;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      float a[4], b[4];
      unpack4(v[i], a);
      unpack4(u[i], b);
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] += b[j];
      v[i] = pack4(a);
    }
  }
  if (p.r) {
    uint2* ro = reinterpret_cast<uint2*>(p.r + row * p.d);
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (lane + 32 * i < ng) ro[lane + 32 * i] = v[i];
  }
  auto mean_square = [&](float f) {
    float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < G; ++i) {
      float a[4];
      unpack4(v[i], a);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = fmaf(a[j] * f, a[j] * f, q[j]);
    }
    float s = ((q[0] + q[1]) + q[2]) + q[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s * p.inv_d;
  };
  const float rstd = inverse_rms(mean_square(1.0f), p.eps, mean_square);
  if (lane == 0 && p.rstd) p.rstd[row] = rstd;
  const uint2* gr = reinterpret_cast<const uint2*>(p.gamma);
  uint2* yo = reinterpret_cast<uint2*>(p.y + row * p.d);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    float a[4], g[4];
    unpack4(v[i], a);
    unpack4(lane + 32 * i < ng ? __ldg(gr + lane + 32 * i) : zero, g);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = __fmul_rn(__fmul_rn(a[j], rstd), g[j]);
    v[i] = pack4(a);
    if (p.y && lane + 32 * i < ng) yo[lane + 32 * i] = v[i];
    if constexpr (KIND != kQNone) amax = max_bits(max_bits(amax, v[i].x), v[i].y);
  }
  if constexpr (KIND != kQNone) {
    const float s = __fdiv_rn(magnitude(warp_max_bits(amax)), KIND == kQE4M3 ? 448.0f : 127.0f);
    if (lane == 0 && p.scale) p.scale[row] = s;
    if (!p.codes && !p.y_hat) return;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int c = lane + 32 * i;
      if (c >= ng) continue;
      float a[4];
      uint32_t code;
      unpack4(v[i], a);
      quantize4<KIND>(a, s, code);
      if (p.codes) reinterpret_cast<uint32_t*>(p.codes + row * p.d)[c] = code;
      if (p.y_hat) reinterpret_cast<uint2*>(p.y_hat + row * p.d)[c] = pack4(a);
    }
  }
}

// Wider rows: W warps per row, each lane keeping VPL 16-byte vectors of it.  Up to 4096 elements the row also
// passes through shared memory, where thread t of the 128 takes chain t (beyond, the order is the lanes' own).
// For 16384 x 2048 with codes 49 us; a warp per row, which needs no barrier, takes 58: its 102 registers leave 20
// warps per SM, and their loads do not cover each other's reductions.
template <int VPL, int W, int KIND>
__global__ void __launch_bounds__(32 * W) rmsnorm_fwd_kernel(const NormFwd p) {
  __shared__ float red[3][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + row * p.ldx);
  uint4 v[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = i * 32 * W + t;
    v[i] = c < p.nv ? __ldcs(xr + c) : make_uint4(0, 0, 0, 0);
  }
  if (p.res) {
    const uint4* rr = reinterpret_cast<const uint4*>(p.res + row * p.ldres);
    uint4 u[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      u[i] = c < p.nv ? __ldcs(rr + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float a[8], b[8];
      unpack8(v[i], a);
      unpack8(u[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      v[i] = pack8(a);
    }
  }
  if (p.r) {
    uint4* ro = reinterpret_cast<uint4*>(p.r + row * p.d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      if (c < p.nv) ro[c] = v[i];
    }
  }
  constexpr bool CHAINS = W == 4 && VPL <= 4;
  __shared__ __align__(16) __nv_bfloat16 row_copy[CHAINS ? VPL * 1024 : 8];
  if constexpr (CHAINS) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) reinterpret_cast<uint4*>(row_copy)[i * 128 + t] = v[i];  // zeros past the row
    __syncthreads();
  }
  auto mean_square = [&](float f, float* smem) {
    float sum = 0.0f;
    if constexpr (CHAINS) {
#pragma unroll
      for (int i = 0; i < VPL * 8; ++i) {
        const float a = __bfloat162float(row_copy[i * 128 + t]) * f;
        sum = fmaf(a, a, sum);
      }
      // the four chains of a group in turn (lanes 4 k .. 4 k + 3), then the warp's 8 groups pairwise, then the warps
      const float q1 = __shfl_down_sync(0xffffffffu, sum, 1), q2 = __shfl_down_sync(0xffffffffu, sum, 2),
                  q3 = __shfl_down_sync(0xffffffffu, sum, 3);
      sum = ((sum + q1) + q2) + q3;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) smem[warp] = sum;
      __syncthreads();
      sum = (smem[0] + smem[1]) + (smem[2] + smem[3]);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float a[8];
        unpack8(v[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(a[j] * f, a[j] * f, sum);
      }
      sum = row_sum<W>(sum, smem, warp, lane, 1);
    }
    return sum * p.inv_d;
  };
  const float rstd =
      inverse_rms(mean_square(1.0f, red[0]), p.eps, [&](float f) { return mean_square(f, red[2]); });
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
  const uint4* gr = reinterpret_cast<const uint4*>(p.gamma);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = i * 32 * W + t;
    float a[8], g[8];
    unpack8(v[i], a);
    unpack8(c < p.nv ? __ldg(gr + c) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = __fmul_rn(__fmul_rn(a[j], rstd), g[j]);
    v[i] = pack8(a);
    if constexpr (KIND != kQNone) amax = max_bits(max_bits(max_bits(max_bits(amax, v[i].x), v[i].y), v[i].z), v[i].w);
  }
  if (p.y) {
    uint4* yo = reinterpret_cast<uint4*>(p.y + row * p.d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      if (c < p.nv) yo[c] = v[i];
    }
  }
  if constexpr (KIND != kQNone) {
    amax = warp_max_bits(amax);
    uint32_t* tops = reinterpret_cast<uint32_t*>(red[1]);
    if (lane == 0) tops[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) amax = max(amax, tops[i]);
    const float s = __fdiv_rn(magnitude(amax), KIND == kQE4M3 ? 448.0f : 127.0f);
    if (t == 0 && p.scale) p.scale[row] = s;
    if (!p.codes && !p.y_hat) return;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      if (c >= p.nv) continue;
      float a[8];
      uint32_t code[2];
      unpack8(v[i], a);
      quantize4<KIND>(a, s, code[0]);
      quantize4<KIND>(a + 4, s, code[1]);
      if (p.codes) reinterpret_cast<uint2*>(p.codes + row * p.d)[c] = make_uint2(code[0], code[1]);
      if (p.y_hat) reinterpret_cast<uint4*>(p.y_hat + row * p.d)[c] = pack8(a);
    }
  }
}

constexpr int kRing = 4;  // rows of the backward's ring

struct NormBwd {
  const __nv_bfloat16 *dy, *dres, *r, *gamma;
  const float* rstd;
  __nv_bfloat16* dx;
  float* part;      // [gridDim.x, d] partial dgamma, or null
  int32_t* status;  // [gridDim.x] device error bits of each block (the ring's waits), with part
  int64_t T, ldr;
  int64_t stuck;     // a row whose copies are left out (the failure path's self-check), -1: none
  long long budget;  // clock cycles that a wait of the ring may take
  int nv, d;
};

// Rows are taken in turn by groups of W warps on a fixed grid, a row's loads issued before the row ahead
// of it is worked on; each lane keeps the norm-weight gradient of its own columns in registers over
// all rows of its group, so the sum over rows costs one fp32 row per block, added in a fixed order by
// rmsnorm_dgamma_kernel.
template <int VPL, int W, bool DRES>
__global__ void __launch_bounds__(256) rmsnorm_bwd_kernel(const NormBwd p) {
  constexpr int RB = 8 / W;
  extern __shared__ float4 joined[];  // [RB - 1, d]
  __shared__ float red[RB][2][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / W, wr = warp % W, t = wr * 32 + lane;
  const int64_t step = (int64_t)gridDim.x * RB;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 gm[VPL];
  float dg[VPL][8];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = i * 32 * W + t;
    gm[i] = c < p.nv ? __ldg(reinterpret_cast<const uint4*>(p.gamma) + c) : zero;
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
  }
  uint4 n[VPL], g[VPL], e[DRES ? VPL : 1];
  float rstd = 0.0f;
  auto load = [&](int64_t row, uint4 (&nn)[VPL], uint4 (&gg)[VPL], uint4 (&ee)[DRES ? VPL : 1], float& rs) {
    const bool in = row < p.T;
    const uint4* rr = reinterpret_cast<const uint4*>(p.r + row * p.ldr);
    const uint4* dyr = reinterpret_cast<const uint4*>(p.dy + row * p.d);
    const uint4* er = reinterpret_cast<const uint4*>(p.dres + row * p.d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      const bool ok = in && c < p.nv;
      nn[i] = ok ? __ldcs(rr + c) : zero;
      gg[i] = ok ? __ldcs(dyr + c) : zero;
      if constexpr (DRES) ee[i] = ok ? __ldcs(er + c) : zero;
    }
    rs = in ? __ldg(p.rstd + row) : 0.0f;
  };
  int flip = 0;
  int64_t row = (int64_t)blockIdx.x * RB + grp;
  if constexpr (VPL <= 4) load(row, n, g, e, rstd);
  for (; row < p.T; row += step) {
    uint4 n2[VPL], g2[VPL], e2[DRES ? VPL : 1];
    float rstd2 = 0.0f;
    if constexpr (VPL <= 4) load(row + step, n2, g2, e2, rstd2);
    else load(row, n, g, e, rstd);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float a[8], b[8], w[8];
      unpack8(n[i], a);
      unpack8(g[i], b);
      unpack8(gm[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float nn = a[j] * rstd;
        dg[i][j] = fmaf(b[j], nn, dg[i][j]);
        dot = fmaf(b[j] * w[j], nn, dot);
      }
    }
    dot = row_sum<W>(dot, red[grp][flip], wr, lane, 1 + grp);
    flip ^= 1;  // the next row's partial sums must not overwrite what a slower warp still reads
    const float m = dot / (float)p.d;
    uint4* out = reinterpret_cast<uint4*>(p.dx + row * p.d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      float a[8], b[8], w[8], o[8];
      unpack8_again(n[i], a);
      unpack8_again(g[i], b);
      unpack8_again(gm[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (b[j] * w[j] - a[j] * rstd * m);
      if constexpr (DRES) {
        unpack8(e[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += a[j];
      }
      if (c < p.nv) out[c] = pack8(o);
    }
    if constexpr (VPL <= 4) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        n[i] = n2[i];
        g[i] = g2[i];
        if constexpr (DRES) e[i] = e2[i];
      }
      rstd = rstd2;
    }
  }
  if (!p.part) return;
  if constexpr (RB > 1) {
    if (grp > 0)
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = i * 32 * W + t;
        if (c < p.nv) {
          float4* to = joined + ((int64_t)(grp - 1) * p.nv + c) * 2;
          to[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
          to[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
        }
      }
    __syncthreads();
    if (grp > 0) return;
  }
  float4* pr = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * p.d);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = i * 32 * W + t;
    if (c >= p.nv) continue;
#pragma unroll
    for (int q = 0; q < RB - 1; ++q) {
      const float4 a = joined[((int64_t)q * p.nv + c) * 2], b = joined[((int64_t)q * p.nv + c) * 2 + 1];
      dg[i][0] += a.x; dg[i][1] += a.y; dg[i][2] += a.z; dg[i][3] += a.w;
      dg[i][4] += b.x; dg[i][5] += b.y; dg[i][6] += b.z; dg[i][7] += b.w;
    }
    pr[2 * c] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
    pr[2 * c + 1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
  }
}

__device__ __forceinline__ void unpack_pairs(const uint4& u, uint64_t* f) {
  f[0] = f2pack(bf16lo(u.x), bf16hi(u.x));
  f[1] = f2pack(bf16lo(u.y), bf16hi(u.y));
  f[2] = f2pack(bf16lo(u.z), bf16hi(u.z));
  f[3] = f2pack(bf16lo(u.w), bf16hi(u.w));
}

// The same for rows of 513 to 4096 elements, with the rows ahead in shared memory: each group has a ring
// of kRing rows of r, dy and dres, filled by bulk copies that its first lane issues one row after the
// stage's last use (a row's barrier says that every warp is through with the row before).  When a wait
// runs out the leaders issue no more copies, those under way land before the block gives its memory back,
// and the block makes all its rows of dx and its part of the weight gradient NaN and sets its status word:
// nothing of it is in the loop but the leader's look at its wait (a row made NaN where its wait failed cost 2 us
// of 49 for 16384 x 2048).
template <int VPL, int W, bool DRES>
__global__ void __launch_bounds__(256, 2) rmsnorm_bwd_ring_kernel(const NormBwd p) {
  constexpr int RB = 8 / W, PARTS = DRES ? 3 : 2;
  extern __shared__ __align__(128) uint4 ring_all[];
  __shared__ float red[RB][2][W];
  __shared__ __align__(8) uint64_t bars[RB][kRing];
  __shared__ int abort_flag, late;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / W, wr = warp % W, t = wr * 32 + lane;
  const int64_t step = (int64_t)gridDim.x * RB, first = (int64_t)blockIdx.x * RB + grp;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4* ring = ring_all + (size_t)grp * kRing * PARTS * p.nv;
  const bool leader = t == 0;
  int fills = 0;  // the leader's copies so far, in rows
  if (threadIdx.x == 0) abort_flag = late = 0;
  if (leader) {
    for (int s = 0; s < kRing; ++s) mbar_init(smem_u32(&bars[grp][s]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t bytes = (uint32_t)p.d * 2u;
  auto fill = [&](int stage, int64_t row) {  // the leader's
    ++fills;
    const uint32_t bar = smem_u32(&bars[grp][stage]);
    mbar_expect_tx(bar, PARTS * bytes);
    const __nv_bfloat16* src[3] = {p.r + row * p.ldr, p.dy + row * p.d, DRES ? p.dres + row * p.d : nullptr};
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              smem_u32(ring + (size_t)(stage * PARTS + i) * p.nv)),
          "l"(reinterpret_cast<uint64_t>(src[i])), "r"(bytes), "r"(bar)
          : "memory");
  };
  // a row whose copies never come, in the failure path's self-check, ends its group's copies
  const int64_t end = p.stuck >= 0 && p.stuck % step == first ? p.stuck : p.T;
  if (leader)
    for (int s = 0; s < kRing; ++s)
      if (first + s * step < end) fill(s, first + s * step);
  uint64_t gm[VPL][4], dg[VPL][4];  // pairs of columns: packed fp32 arithmetic
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = i * 32 * W + t;
    unpack_pairs(c < p.nv ? __ldg(reinterpret_cast<const uint4*>(p.gamma) + c) : zero, gm[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = f2pack(0.0f, 0.0f);
  }
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  for (int64_t row = first; row < p.T; row += step) {
    const float rstd = __ldg(p.rstd + row);
    const uint4* at = ring + (size_t)stage * PARTS * p.nv;
    // a wait that ran out leaves wrong values, replaced below; the group's barriers stay in step
    const bool ok = mbar_wait(smem_u32(&bars[grp][stage]), phase, &abort_flag, &late, p.budget);
    __syncwarp();
    uint64_t n[VPL][4], dn[VPL][4], dot2 = f2pack(0.0f, 0.0f);
    const uint64_t rs2 = f2pack(rstd, rstd);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      uint64_t b[4];
      unpack_pairs(c < p.nv ? at[c] : zero, n[i]);
      unpack_pairs(c < p.nv ? at[p.nv + c] : zero, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n[i][j] = f2mul(n[i][j], rs2);
        dg[i][j] = f2fma(b[j], n[i][j], dg[i][j]);
        dn[i][j] = f2mul(b[j], gm[i][j]);
        dot2 = f2fma(dn[i][j], n[i][j], dot2);
      }
    }
    const float2 dots = f2unpack(dot2);
    float dot = dots.x + dots.y;
    dot = row_sum<W>(dot, red[grp][flip], wr, lane, 1 + grp);
    flip ^= 1;  // the next row's partial sums must not overwrite what a slower warp still reads
    if constexpr (W == 1) __syncwarp();
    // every warp has passed this row's barrier, so all are through with the row before: its stage takes the row
    // kRing - 1 ahead
    const int64_t ahead = row + (int64_t)(kRing - 1) * step;
    if (leader && row > first && ahead < end && ok) fill(stage == 0 ? kRing - 1 : stage - 1, ahead);
    const float m = -rstd * (dot / (float)p.d);
    const uint64_t m2 = f2pack(m, m);
    uint4* out = reinterpret_cast<uint4*>(p.dx + row * p.d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = i * 32 * W + t;
      if (c >= p.nv) continue;
      uint64_t e[4];
      if constexpr (DRES) unpack_pairs(at[2 * p.nv + c], e);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // rstd dn - rstd mean(dn n) n (+ dres)
        uint64_t v = DRES ? f2fma(dn[i][j], rs2, e[j]) : f2mul(dn[i][j], rs2);
        const float2 x = f2unpack(f2fma(n[i][j], m2, v));
        o[j] = pack_bf16(x.x, x.y);
      }
      out[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (++stage == kRing) {
      stage = 0;
      phase ^= 1u;
    }
  }
  __syncthreads();
  if (abort_flag) {  // alike in the whole block: no wait is left
    volatile int none = 0;
    for (int s = 0; leader && s < kRing; ++s)
      if (fills > s) mbar_wait(smem_u32(&bars[grp][s]), (uint32_t)((fills - 1 - s) / kRing) & 1u, &none, &late);
    const uint32_t nans = 0x7fff7fffu;
    for (int64_t row = first; row < p.T; row += step)
      for (int c = t; c < p.nv; c += 32 * W)
        reinterpret_cast<uint4*>(p.dx + row * p.d)[c] = make_uint4(nans, nans, nans, nans);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) dg[i][j] = f2pack(NAN, NAN);
    __syncthreads();
  }
  if (!p.part) return;
  if (threadIdx.x == 0) p.status[blockIdx.x] = late;
  float4* joined = reinterpret_cast<float4*>(ring_all);  // [RB - 1, d]: every copy has landed and been read
  auto store = [&](float4* to, const uint64_t (&v)[4]) {
    const float2 a = f2unpack(v[0]), b = f2unpack(v[1]), c = f2unpack(v[2]), d = f2unpack(v[3]);
    to[0] = make_float4(a.x, a.y, b.x, b.y);
    to[1] = make_float4(c.x, c.y, d.x, d.y);
  };
  if constexpr (RB > 1) {
    if (grp > 0)
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = i * 32 * W + t;
        if (c < p.nv) store(joined + ((int64_t)(grp - 1) * p.nv + c) * 2, dg[i]);
      }
    __syncthreads();
    if (grp > 0) return;
  }
  float4* pr = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * p.d);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int c = i * 32 * W + t;
    if (c >= p.nv) continue;
#pragma unroll
    for (int q = 0; q < RB - 1; ++q) {
      const float4 a = joined[((int64_t)q * p.nv + c) * 2], b = joined[((int64_t)q * p.nv + c) * 2 + 1];
      dg[i][0] = f2add(dg[i][0], f2pack(a.x, a.y));
      dg[i][1] = f2add(dg[i][1], f2pack(a.z, a.w));
      dg[i][2] = f2add(dg[i][2], f2pack(b.x, b.y));
      dg[i][3] = f2add(dg[i][3], f2pack(b.z, b.w));
    }
    store(pr + 2 * c, dg[i]);
  }
}

// dgamma[c] = sum over the partial rows, in a fixed order: 32 columns per block, each of 32 warps
// adding every 32nd row.  Block 0 joins the status words (null: the backward waits for nothing) into the error word.
// part and status are written while this kernel is already resident: ordinary loads after the wait, not the
// non-coherent ones that const __restrict__ allows.
__global__ void __launch_bounds__(1024) rmsnorm_dgamma_kernel(const float* part, int parts, int d, float* dgamma,
                                                              const int32_t* status, int32_t* err) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched beside the backward's end: its partial rows are complete
  const int late = blockIdx.x == 0 && status && threadIdx.x < parts ? status[threadIdx.x] : 0;
  float v = 0.0f;
  if (c < d)
#pragma unroll 10
    for (int i = warp; i < parts; i += 32) v += part[(int64_t)i * d + c];
  s[warp][lane] = v;
  const int bad = __syncthreads_or(late);
  if (blockIdx.x == 0 && threadIdx.x == 0) *err = bad ? QAD_DEV_TIMEOUT : 0;
  v = warp_sum(s[lane][warp]);
  const int cw = blockIdx.x * 32 + warp;
  if (lane == 0 && cw < d) dgamma[cw] = v;
}

template <int G>
cudaError_t fwd_warp(const NormFwd& p, int kind, cudaStream_t st) {
  const unsigned blocks = (unsigned)((p.T + 3) / 4);
  if (kind == kQE4M3) rmsnorm_fwd_warp_kernel<G, kQE4M3><<<blocks, 128, 0, st>>>(p);
  else if (kind == kQInt8) rmsnorm_fwd_warp_kernel<G, kQInt8><<<blocks, 128, 0, st>>>(p);
  else rmsnorm_fwd_warp_kernel<G, kQNone><<<blocks, 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <int VPL, int W>
cudaError_t fwd_wide(const NormFwd& p, int kind, cudaStream_t st) {
  if (kind == kQE4M3) rmsnorm_fwd_kernel<VPL, W, kQE4M3><<<(unsigned)p.T, 32 * W, 0, st>>>(p);
  else if (kind == kQInt8) rmsnorm_fwd_kernel<VPL, W, kQInt8><<<(unsigned)p.T, 32 * W, 0, st>>>(p);
  else rmsnorm_fwd_kernel<VPL, W, kQNone><<<(unsigned)p.T, 32 * W, 0, st>>>(p);
  return cudaGetLastError();
}

template <int VPL, int W, bool DRES>
cudaError_t bwd_ring(const NormBwd& p, int blocks, cudaStream_t st) {
  auto kern = rmsnorm_bwd_ring_kernel<VPL, W, DRES>;
  constexpr int kMax = 8 / W * kRing * 3 * 512 * W * VPL;  // bytes at the widest row
  static bool ready[64] = {false};  // per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!ready[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMax);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  size_t smem = (size_t)(8 / W) * kRing * (DRES ? 3 : 2) * p.d * 2;
  kern<<<(unsigned)blocks, 256, smem, st>>>(p);
  return cudaGetLastError();
}

template <int VPL, int W>
cudaError_t bwd_launch(const NormBwd& p, int blocks, cudaStream_t st) {
  // rows of 512 elements or fewer stay with loads: their copies of 1 KB or less cost more than they hide (32768
  // x 512: 29 against 33 us, x 256: 20 against 25); from 1024 on the ring wins (16000 x 4096: 83 against 91)
  if constexpr (VPL <= 2 && W >= 2) {
    return p.dres ? bwd_ring<VPL, W, true>(p, blocks, st) : bwd_ring<VPL, W, false>(p, blocks, st);
  } else {
    const size_t smem = p.part ? (size_t)(8 / W - 1) * p.d * 4 : 0;
    if (p.dres) rmsnorm_bwd_kernel<VPL, W, true><<<(unsigned)blocks, 256, smem, st>>>(p);
    else rmsnorm_bwd_kernel<VPL, W, false><<<(unsigned)blocks, 256, smem, st>>>(p);
    return cudaGetLastError();
  }
}

}  // namespace

// Blocks of the backward, and so partial dgamma rows: a constant, so that the workspace size needs no device query.
// (Bounding the registers for three or four blocks spills: 86 and 96 us against 50 for 16384 x 2048.)
constexpr int kNormBlocks = 304;  // two per SM of 152: as many as the registers hold up to 4096 elements, twice as many above

int norm_blocks(int64_t T) { return (int)(T < kNormBlocks ? T : kNormBlocks); }

// The workspace: the error word, the blocks' status words from kNormStatus on, and the partial dgamma rows
constexpr size_t kNormStatus = 256, kNormHeader = 2048;
static_assert(kNormStatus + 4 * kNormBlocks <= kNormHeader, "a status word per block");
size_t norm_workspace(int64_t T, int64_t d) { return kNormHeader + 4 * (size_t)norm_blocks(T) * (size_t)d; }

cudaError_t launch_rmsnorm_fwd(const void* x, int64_t ldx, const void* res, int64_t ldres, const void* gamma, float eps,
                               int kind, void* r, void* y, void* y_hat, void* codes, float* scale, float* rstd,
                               int64_t T, int64_t d, cudaStream_t st) {
  NormFwd p = {};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.res = static_cast<const __nv_bfloat16*>(res);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma);
  p.r = static_cast<__nv_bfloat16*>(r);
  p.y = static_cast<__nv_bfloat16*>(y);
  p.y_hat = static_cast<__nv_bfloat16*>(y_hat);
  p.codes = static_cast<uint8_t*>(codes);
  p.scale = scale;
  p.rstd = rstd;
  p.T = T;
  p.ldx = ldx;
  p.ldres = ldres;
  p.nv = (int)(d / 8);
  p.d = (int)d;
  p.eps = eps;
  p.inv_d = 1.0f / (float)d;
  prof_begin(QAD_K_RMSNORM, st);
  const int groups = (int)((d + 127) / 128);  // 4-element groups per lane of a warp
  cudaError_t e;
  if (groups <= 2) e = fwd_warp<2>(p, kind, st);
  else if (groups <= 4) e = fwd_warp<4>(p, kind, st);
  else if (groups <= 8) e = fwd_warp<8>(p, kind, st);
  else if (groups <= 16) e = fwd_wide<2, 4>(p, kind, st);
  else if (groups <= 24) e = fwd_wide<3, 4>(p, kind, st);
  else if (groups <= 32) e = fwd_wide<4, 4>(p, kind, st);
  else if (groups <= 64) e = fwd_wide<8, 4>(p, kind, st);
  else e = fwd_wide<8, 8>(p, kind, st);
  prof_end(QAD_K_RMSNORM, st);
  return e;
}

cudaError_t launch_rmsnorm_bwd(const void* dy, const void* dres, const void* r, int64_t ldr, const void* gamma,
                               const float* rstd, void* dx, float* dgamma, uint8_t* ws, int64_t T, int64_t d,
                               cudaStream_t st) {
  NormBwd p = {};
  p.dy = static_cast<const __nv_bfloat16*>(dy);
  p.dres = static_cast<const __nv_bfloat16*>(dres);
  p.r = static_cast<const __nv_bfloat16*>(r);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma);
  p.rstd = rstd;
  p.dx = static_cast<__nv_bfloat16*>(dx);
  p.part = dgamma ? reinterpret_cast<float*>(ws + kNormHeader) : nullptr;
  p.status = dgamma ? reinterpret_cast<int32_t*>(ws + kNormStatus) : nullptr;
  const StuckCopy stuck = stuck_copy();
  p.stuck = stuck.row;
  p.budget = stuck.row < 0 ? kWaitCycles : stuck.budget;
  p.T = T;
  p.ldr = ldr;
  p.nv = (int)(d / 8);
  p.d = (int)d;
  const int lanes1 = (p.nv + 31) / 32;
  const int w = lanes1 <= 2 ? 1 : lanes1 <= 4 ? 2 : lanes1 <= 8 ? 4 : 8;  // warps per row
  const int blocks = norm_blocks((T + 8 / w - 1) / (8 / w));
  prof_begin(QAD_K_RMSNORM_BWD, st);
  cudaError_t e;
  if (lanes1 <= 1) e = bwd_launch<1, 1>(p, blocks, st);
  else if (lanes1 <= 2) e = bwd_launch<2, 1>(p, blocks, st);
  else if (lanes1 <= 4) e = bwd_launch<2, 2>(p, blocks, st);
  else if (lanes1 <= 8) e = bwd_launch<2, 4>(p, blocks, st);
  else if (lanes1 <= 16) e = bwd_launch<2, 8>(p, blocks, st);
  else if (lanes1 <= 32) e = bwd_launch<4, 8>(p, blocks, st);
  else e = bwd_launch<8, 8>(p, blocks, st);
  prof_end(QAD_K_RMSNORM_BWD, st);
  if (e != cudaSuccess || !dgamma) return e;
  note_launches(1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((d + 31) / 32), 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  const bool ring = lanes1 > 2 && lanes1 <= 16;  // the others write no status
  return cudaLaunchKernelEx(&cfg, rmsnorm_dgamma_kernel, static_cast<const float*>(p.part), blocks, (int)d, dgamma,
                            static_cast<const int32_t*>(ring ? p.status : nullptr), reinterpret_cast<int32_t*>(ws));
}

}  // namespace qad
