// Root-mean-square norm with the residual's addition and an int8 output with
// one scale a token, in one pass over the activations:
//
//   h = x + residual, rounded once to the activations' type (and stored)
//   r = 1 / sqrt(mean(h^2) + eps)            sum and root in fp64, rounded once to fp32; 0 for a row of zeros
//   y = (h * r) * weight                     fp32, one rounding a product
//   sx = max|y| / 127;  qx = clip(rint(y / sx), -127, 127)
//
// The squares are summed in fp64 (each is exact there), so r does not depend on
// the order of the sum except where its last fp32 bit hangs on the 53rd bit, and
// every later step is one IEEE operation: codes and scales are reproducible bit
// for bit by any implementation of the formula, as quant_per_token_i8's are.
// The normalized row itself is never written: what bounds the kernel is x, the
// residual in and out and one byte a value, 7 bytes an element.  16384 x 4096 bf16
// with residual: 72.4 us = 6.5 TB/s, the rate of a plain copy; one row of 4096:
// 2.6 us, the latency of a launch and two reductions.  Issue slots come next (two
// thirds busy): the exact quotients take three operations instead of a division
// (130 us with divisions, an fp32 copy of the row and one run a thread).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "quotient.cuh"

namespace gwb {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int64_t kManyRows = 592;   // four rows an SM

template <bool F16>
__device__ __forceinline__ float to_f(uint16_t h) {
  if constexpr (F16) return __half2float(__ushort_as_half(h));
  else return __uint_as_float((uint32_t)h << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t from_f(float f) {
  if constexpr (F16) return __half_as_ushort(__float2half_rn(f));
  else return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// The int8 code of y over a row's scale, by the division itself; 0 for rows of zeros and rows that are not finite.
__device__ __forceinline__ int quant_slow(float y, float s) {
  return !(s > 0.0f && s < INFINITY) ? 0 : (int)fminf(fmaxf(rintf(__fdiv_rn(y, s)), -127.0f), 127.0f);
}

// Two values of 16 bits a word, as fp32.
template <bool F16>
__device__ __forceinline__ float2 to_f2(uint32_t w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t from_f2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

struct NormArgs {
  const uint16_t *x, *residual, *weight;
  uint16_t *residual_out;
  int8_t *qx;
  float *sx;
  int64_t K;
  double eps;
};

// Block reductions; `red` holds one slot a warp and one for the result.
__device__ __forceinline__ float block_rstd(double sum, double *red, float *out, int64_t K, double eps) {
  sum = warp_sum(sum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    const double t = warp_sum(lane < nw ? red[lane] : 0.0);
    if (lane == 0) *out = t == 0.0 ? 0.0f : (float)(1.0 / sqrt(t / (double)K + eps));   // (0 * inf is no norm)
  }
  __syncthreads();
  return *out;
}
__device__ __forceinline__ float block_max(float v, float *red) {
  v = warp_max(v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_max(lane < nw ? red[lane] : 0.0f);
}

// One row a block, the row in registers: V runs of 8 elements a thread, 16-byte
// loads where the width is a multiple of 8 (VEC), single elements otherwise.
template <int V, bool VEC, bool F16>
__global__ void __launch_bounds__(V > 2 ? 512 : 1024) k_rmsnorm_row(const NormArgs a) {
  __shared__ double red_d[32];
  __shared__ float red_f[32], rstd_s;
  const int64_t m = blockIdx.x;
  const int K = (int)a.K, nt = blockDim.x, tid = threadIdx.x;
  const uint16_t *x = a.x + m * K, *res = a.residual ? a.residual + m * K : nullptr;
  // element e of run v: a run is contiguous (VEC) or a column of the block's stride
  auto at = [&](int v, int e) { return VEC ? (v * nt + tid) * 8 + e : (v * 8 + e) * nt + tid; };
  auto load = [&](const uint16_t *p, int v) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
      if (at(v, 0) < K) u = *reinterpret_cast<const uint4 *>(p + at(v, 0));
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (at(v, e) < K) w[e / 2] |= (uint32_t)p[at(v, e)] << (e % 2 * 16);
      u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return u;
  };

  uint4 xr[V], rr[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    xr[v] = load(x, v);
    if (res) rr[v] = load(res, v);
  }
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    uint32_t w[4] = {xr[v].x, xr[v].y, xr[v].z, xr[v].w};
    if (res) {
      const uint32_t r4[4] = {rr[v].x, rr[v].y, rr[v].z, rr[v].w};
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float2 f = to_f2<F16>(w[i]), g = to_f2<F16>(r4[i]);
        w[i] = from_f2<F16>(__fadd_rn(f.x, g.x), __fadd_rn(f.y, g.y));
      }
      uint16_t *dst = a.residual_out + m * K;
      if constexpr (VEC) {
        if (at(v, 0) < K) *reinterpret_cast<uint4 *>(dst + at(v, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (at(v, e) < K) dst[at(v, e)] = (uint16_t)(w[e / 2] >> (e % 2 * 16));
      }
    }
    xr[v] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 f = to_f2<F16>(w[i]);
      sum = fma((double)f.x, (double)f.x, sum);
      sum = fma((double)f.y, (double)f.y, sum);
    }
  }
  const float r = block_rstd(sum, red_d, &rstd_s, a.K, a.eps);

  float y[V][8], amax = 0.0f;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const uint4 wv = load(a.weight, v);
    const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w}, h[4] = {xr[v].x, xr[v].y, xr[v].z, xr[v].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 f = to_f2<F16>(h[i]), g = to_f2<F16>(w[i]);
      y[v][2 * i] = __fmul_rn(__fmul_rn(f.x, r), g.x);
      y[v][2 * i + 1] = __fmul_rn(__fmul_rn(f.y, r), g.y);
      amax = max_nan(amax, fabsf(y[v][2 * i]), fabsf(y[v][2 * i + 1]));
    }
  }
  amax = block_max(amax, red_f);
  const float s = __fdiv_rn(amax, 127.0f);
  const Divisor d = make_divisor(s);
  if (tid == 0) a.sx[m] = s;
  int8_t *q = a.qx + m * K;
#pragma unroll
  for (int v = 0; v < V; v++) {
    // |y| <= 127 s (1 + 2^-23), so no code passes 127; the low byte of the rounded quotient is the code
    uint32_t c[8];
    if (d.fast) {
#pragma unroll
      for (int e = 0; e < 8; e++) c[e] = __float_as_uint(round_bits(quotient_fast(y[v][e], d)));
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) c[e] = (uint32_t)quant_slow(y[v][e], s);
    }
    if constexpr (VEC) {
      uint32_t o[2];
#pragma unroll
      for (int i = 0; i < 2; i++)
        o[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
      if (at(v, 0) < K) *reinterpret_cast<uint2 *>(q + at(v, 0)) = make_uint2(o[0], o[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (at(v, e) < K) q[at(v, e)] = (int8_t)c[e];
    }
  }
}

// Rows too wide for the registers of one block (K > 32768): the same steps with
// the row read again for each (from L2 for all but the first).
template <bool F16>
__global__ void __launch_bounds__(1024) k_rmsnorm_wide(const NormArgs a) {
  __shared__ double red_d[32];
  __shared__ float red_f[32], rstd_s;
  const int64_t m = blockIdx.x, K = a.K;
  const uint16_t *x = a.x + m * K;
  const uint16_t *res = a.residual ? a.residual + m * K : nullptr;
  // element i of h; x and residual are read again unless they were overwritten by h
  auto value = [&](int64_t i, bool first) {
    if (!res) return to_f<F16>(x[i]);
    if (!first) return to_f<F16>(a.residual_out[m * K + i]);
    const uint16_t hb = from_f<F16>(__fadd_rn(to_f<F16>(x[i]), to_f<F16>(res[i])));
    a.residual_out[m * K + i] = hb;
    return to_f<F16>(hb);
  };
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < K; i += blockDim.x) {
    const double f = (double)value(i, true);
    sum = fma(f, f, sum);
  }
  const float r = block_rstd(sum, red_d, &rstd_s, K, a.eps);
  float amax = 0.0f;
  for (int64_t i = threadIdx.x; i < K; i += blockDim.x)
    amax = max_nan(amax, fabsf(__fmul_rn(__fmul_rn(value(i, false), r), to_f<F16>(__ldg(a.weight + i)))));
  amax = block_max(amax, red_f);
  const float s = __fdiv_rn(amax, 127.0f);
  if (threadIdx.x == 0) a.sx[m] = s;
  for (int64_t i = threadIdx.x; i < K; i += blockDim.x) {
    const float y = __fmul_rn(__fmul_rn(value(i, false), r), to_f<F16>(__ldg(a.weight + i)));
    a.qx[m * K + i] = (int8_t)quant_slow(y, s);
  }
}

template <bool F16>
void launch(const NormArgs &a, int64_t M, cudaStream_t st) {
  const int64_t runs = (a.K + 7) / 8;                  // 8-element runs of a row
  const bool vec = a.K % 8 == 0;
  const unsigned grid = (unsigned)M;
  auto threads = [&](int V) { return (unsigned)((runs + (int64_t)V * 32 - 1) / ((int64_t)V * 32) * 32); };
  // Few rows: as many threads a row as its runs allow, for the latency of one row.
  // Many rows: up to four runs a thread, for the two reductions' cost a row.
  const int64_t want = M >= kManyRows ? (runs >= 256 ? 4 : (runs >= 64 ? 2 : 1)) : 1;
#define GWB_NORM(V, VEC) k_rmsnorm_row<V, VEC, F16><<<grid, threads(V), 0, st>>>(a)
  if (runs <= 1024 && want == 1) return vec ? GWB_NORM(1, true) : GWB_NORM(1, false);
  if (runs <= 2048 && want <= 2) return vec ? GWB_NORM(2, true) : GWB_NORM(2, false);
  if (runs <= 2048) return vec ? GWB_NORM(4, true) : GWB_NORM(4, false);
  if (runs <= 4096) return vec ? GWB_NORM(8, true) : GWB_NORM(8, false);
#undef GWB_NORM
  k_rmsnorm_wide<F16><<<grid, 1024, 0, st>>>(a);
}

}  // namespace

void launch_rmsnorm_quant_i8(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, int64_t M,
                             int64_t K, double eps, bool f16, uint16_t *residual_out, int8_t *qx, float *sx,
                             cudaStream_t st) {
  NormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight;
  a.residual_out = residual_out; a.qx = qx; a.sx = sx;
  a.K = K; a.eps = eps;
  if (f16) launch<true>(a, M, st);
  else launch<false>(a, M, st);
}

}  // namespace gwb
