// Root-mean-square norm with the residual's addition and an int8 output with
// one scale a token, in one pass over the activations:
//
//   h = x + residual, rounded once to the activations' type (and stored)
//   r = 1 / sqrt(mean(h^2) + eps)            sum and root in fp64, rounded once to fp32
//   y = (h * r) * weight                     fp32, one rounding a product
//   sx = max|y| / 127;  qx = clip(rint(y / sx), -127, 127)
//
// The squares are summed in fp64 (each is exact there), so r does not depend on
// the order of the sum except where its last fp32 bit hangs on the 53rd bit, and
// every later step is one IEEE operation: codes and scales are reproducible bit
// for bit by any implementation of the formula, as quant_per_token_i8's are.
// The normalized row itself is never written: what bounds the kernel is x, the
// residual in and out and one byte a value, 7 bytes an element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace gwb {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxThreads = 1024;

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

// rint(y / s) clipped to +-127, the division correctly rounded.  `inv` is about
// 1 / s: y * inv is within 127 * 2^-22 of the quotient, so away from a rounding
// border (by far more than that) both round to the same integer, and only
// quotients within 2^-12 of one take the division.
__device__ __forceinline__ int quant(float y, float s, float inv) {
  float t = __fmul_rn(y, inv);
  float n = rintf(t);
  if (fabsf(fabsf(__fsub_rn(t, n)) - 0.5f) < 0x1p-12f) n = rintf(__fdiv_rn(y, s));
  return (int)fminf(fmaxf(n, -127.0f), 127.0f);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
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
    if (lane == 0) *out = (float)(1.0 / sqrt(t / (double)K + eps));
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
__global__ void __launch_bounds__(kMaxThreads) k_rmsnorm_row(const NormArgs a) {
  __shared__ double red_d[32];
  __shared__ float red_f[32], rstd_s;
  const int64_t m = blockIdx.x, K = a.K;
  const int nt = blockDim.x, tid = threadIdx.x;
  const uint16_t *x = a.x + m * K;
  const uint16_t *res = a.residual ? a.residual + m * K : nullptr;
  auto at = [&](int v, int e) { return VEC ? ((int64_t)v * nt + tid) * 8 + e : (int64_t)(v * 8 + e) * nt + tid; };

  float h[V][8];
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    uint16_t raw[8], rr[8];
    if constexpr (VEC) {
      uint4 u = make_uint4(0, 0, 0, 0), w = make_uint4(0, 0, 0, 0);
      if (at(v, 0) < K) {
        u = *reinterpret_cast<const uint4 *>(x + at(v, 0));
        if (res) w = *reinterpret_cast<const uint4 *>(res + at(v, 0));
      }
      *reinterpret_cast<uint4 *>(raw) = u;
      *reinterpret_cast<uint4 *>(rr) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const bool in = at(v, e) < K;
        raw[e] = in ? x[at(v, e)] : 0;
        rr[e] = in && res ? res[at(v, e)] : 0;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
      float f = to_f<F16>(raw[e]);
      if (res) {
        raw[e] = from_f<F16>(__fadd_rn(f, to_f<F16>(rr[e])));
        f = to_f<F16>(raw[e]);
      }
      h[v][e] = f;
      sum = fma((double)f, (double)f, sum);
    }
    if (a.residual_out) {
      uint16_t *dst = a.residual_out + m * K;
      if constexpr (VEC) {
        if (at(v, 0) < K) *reinterpret_cast<uint4 *>(dst + at(v, 0)) = *reinterpret_cast<const uint4 *>(raw);
      } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (at(v, e) < K) dst[at(v, e)] = raw[e];
      }
    }
  }
  const float r = block_rstd(sum, red_d, &rstd_s, K, a.eps);

  float amax = 0.0f;
#pragma unroll
  for (int v = 0; v < V; v++) {
    uint16_t w[8];
    if constexpr (VEC) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (at(v, 0) < K) u = __ldg(reinterpret_cast<const uint4 *>(a.weight + at(v, 0)));
      *reinterpret_cast<uint4 *>(w) = u;
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) w[e] = at(v, e) < K ? __ldg(a.weight + at(v, e)) : (uint16_t)0;
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
      h[v][e] = __fmul_rn(__fmul_rn(h[v][e], r), to_f<F16>(w[e]));
      amax = fmaxf(amax, fabsf(h[v][e]));
    }
  }
  amax = block_max(amax, red_f);
  const float s = __fdiv_rn(amax, 127.0f);
  const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  const bool ok = inv <= 3.0e38f;                     // s so small that 1 / s overflows: divide
  if (tid == 0) a.sx[m] = s;
  int8_t *q = a.qx + m * K;
#pragma unroll
  for (int v = 0; v < V; v++) {
    int c[8];
#pragma unroll
    for (int e = 0; e < 8; e++)
      c[e] = s == 0.0f ? 0 : ok ? quant(h[v][e], s, inv) : (int)fminf(fmaxf(rintf(__fdiv_rn(h[v][e], s)), -127.0f), 127.0f);
    if constexpr (VEC) {
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; e++) o[e / 4] |= ((uint32_t)c[e] & 0xffu) << (e % 4 * 8);
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
__global__ void __launch_bounds__(kMaxThreads) k_rmsnorm_wide(const NormArgs a) {
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
    amax = fmaxf(amax, fabsf(__fmul_rn(__fmul_rn(value(i, false), r), to_f<F16>(__ldg(a.weight + i)))));
  amax = block_max(amax, red_f);
  const float s = __fdiv_rn(amax, 127.0f);
  if (threadIdx.x == 0) a.sx[m] = s;
  for (int64_t i = threadIdx.x; i < K; i += blockDim.x) {
    const float y = __fmul_rn(__fmul_rn(value(i, false), r), to_f<F16>(__ldg(a.weight + i)));
    a.qx[m * K + i] = s == 0.0f ? (int8_t)0 : (int8_t)fminf(fmaxf(rintf(__fdiv_rn(y, s)), -127.0f), 127.0f);
  }
}

template <bool F16>
void launch(const NormArgs &a, int64_t M, cudaStream_t st) {
  const int64_t runs = (a.K + 7) / 8;                  // 8-element runs of a row
  const bool vec = a.K % 8 == 0;
  const unsigned grid = (unsigned)M;
  auto threads = [&](int V) { return (unsigned)((runs + (int64_t)V * 32 - 1) / ((int64_t)V * 32) * 32); };
#define GWB_NORM(V, VEC) k_rmsnorm_row<V, VEC, F16><<<grid, threads(V), 0, st>>>(a)
  if (runs <= kMaxThreads) return vec ? GWB_NORM(1, true) : GWB_NORM(1, false);
  if (runs <= 2 * kMaxThreads) return vec ? GWB_NORM(2, true) : GWB_NORM(2, false);
  if (runs <= 4 * kMaxThreads) return vec ? GWB_NORM(4, true) : GWB_NORM(4, false);
#undef GWB_NORM
  k_rmsnorm_wide<F16><<<grid, kMaxThreads, 0, st>>>(a);
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
