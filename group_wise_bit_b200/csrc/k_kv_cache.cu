// Writing tokens' keys and values into the paged, quantized cache, and reading
// rows of it back.
//
// Eight consecutive elements of a row (16 bytes of bf16 or fp16) belong to one
// lane; D / 8 lanes hold a row of one (token, head, key or value), and the
// gs / 8 lanes of a group find its min and max with shuffles.  The arithmetic is
// qpack_affine's (fp32, one IEEE rounding a step, bf16 scale and bias), so codes,
// scales and biases are bit-exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv_layout.cuh"
#include "ptx.cuh"
#include "quotient.cuh"

namespace gwb {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&v)[8]) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if constexpr (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p[j]));
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    } else {
      v[2 * j] = bf16_lo(p[j]);
      v[2 * j + 1] = bf16_hi(p[j]);
    }
  }
}

struct KvArgs {
  const uint16_t *k, *v;       // write: rows [T][H][D], tokens k_stride / v_stride elements apart
  uint16_t *ko, *vo;           // read: dense [T][H][D]
  int64_t k_stride, v_stride;
  const int64_t *slots;
  unsigned char *cache;
  int64_t total_slots;
  uint32_t rows;               // T * H
  int H, page_shift;
};

// This lane's place: row (token, head) and element 8 * l in it; blockIdx.y: keys or values.
struct Place {
  uint32_t row, t;
  int h, l;
};
template <int D>
__device__ __forceinline__ Place place_of(const KvArgs &a) {
  constexpr int LR = D / 8;
  Place p;
  p.row = blockIdx.x * (kThreads / LR) + threadIdx.x / LR;
  p.l = threadIdx.x % LR;
  p.t = p.row / (uint32_t)a.H;
  p.h = (int)(p.row - p.t * (uint32_t)a.H);
  return p;
}

// Start of the granule that holds `slot` of head h, and the token's place in it;
// false for a slot outside the cache (negative: a padded row, else an error).
__device__ __forceinline__ bool granule_of(const KvArgs &a, int64_t slot, int h, int granule, int64_t *off, int *tok) {
  if (slot < 0) return false;
  if (slot >= a.total_slots) {
    atomicOr(&g_device_error, kErrIndex);
    return false;
  }
  const int64_t page = slot >> a.page_shift;
  const int in_page = (int)slot & ((1 << a.page_shift) - 1);
  *off = (((page * a.H + h) << a.page_shift) + in_page) / kv::kTok * granule;
  *tok = in_page % kv::kTok;
  return true;
}

template <int BITS, int D, int GS, bool F16>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvArgs a) {
  constexpr kv::Layout L = kv::layout(BITS, D, GS);
  constexpr int LG = GS / 8;              // lanes of a group
  constexpr float QMAX = (float)((1 << BITS) - 1);
  const Place p = place_of<D>(a);
  const bool val = blockIdx.y != 0;
  int64_t off = 0;
  int tok = 0;
  const bool live = p.row < a.rows && granule_of(a, __ldg(a.slots + p.t), p.h, L.granule, &off, &tok);
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (live) {
    const uint16_t *row = val ? a.v + p.t * a.v_stride : a.k + p.t * a.k_stride;
    unpack8<F16>(__ldg(reinterpret_cast<const uint4 *>(row + p.h * D + p.l * 8)), v);
  }
  // (min and max order -0 below +0, as qpack_affine's keys do)
  float mn = v[0], mx = v[0];
#pragma unroll
  for (int j = 1; j < 8; j++) {
    mn = fminf(mn, v[j]);
    mx = fmaxf(mx, v[j]);
  }
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(kFull, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  }
  if (!live) return;
  const float s = __fdiv_rn(__fsub_rn(mx, mn), QMAX);
  const Divisor d = make_divisor(s);
  uint32_t words[BITS / 4];
  if (d.fast) {
    // integers n in the low bits of the rounded quotients; no code passes QMAX (quotients are within 2^-23 of it)
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; j++) z[j] = round_bits(quotient_fast(__fsub_rn(v[j], mn), d));
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 2; i++)
        words[i] = __byte_perm(__byte_perm(__float_as_uint(z[4 * i]), __float_as_uint(z[4 * i + 1]), 0x0040),
                               __byte_perm(__float_as_uint(z[4 * i + 2]), __float_as_uint(z[4 * i + 3]), 0x0040), 0x5410);
    } else {
      // four nibbles at a time in fp32: exact below 2^16
      uint32_t h[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float n[4];
#pragma unroll
        for (int j = 0; j < 4; j++) n[j] = __fsub_rn(z[4 * i + j], kRoundMagic);
        h[i] = __float_as_uint(round_bits(fmaf(fmaf(n[3], 16.0f, n[2]), 256.0f, fmaf(n[1], 16.0f, n[0]))));
      }
      words[0] = __byte_perm(h[0], h[1], 0x5410);
    }
  } else {
#pragma unroll
    for (int i = 0; i < BITS / 4; i++) words[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      uint32_t q = 0;
      if (s != 0.0f) q = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[j], mn), s)), 0.0f), QMAX);
      words[j * BITS / 32] |= q << (j * BITS % 32);
    }
  }
  unsigned char *gran = a.cache + off;
#pragma unroll
  for (int i = 0; i < BITS / 4; i++) {
    const int w = p.l * (BITS / 4) + i;
    if (!val) {
      *reinterpret_cast<uint32_t *>(gran + kv::key_word(L, tok, w)) = words[i];
    } else {
      *reinterpret_cast<uint16_t *>(gran + kv::val_half(L, tok, 2 * w)) = (uint16_t)words[i];
      *reinterpret_cast<uint16_t *>(gran + kv::val_half(L, tok, 2 * w + 1)) = (uint16_t)(words[i] >> 16);
    }
  }
  if (p.l % LG == 0) {
    const int g = p.l / LG;
    if (!val) {
      *reinterpret_cast<uint32_t *>(gran + kv::key_meta(L, tok, g)) = bf16_bits(s) | (bf16_bits(mn) << 16);
    } else {
      *reinterpret_cast<uint16_t *>(gran + kv::val_scale(L, tok, g)) = (uint16_t)bf16_bits(s);
      *reinterpret_cast<uint16_t *>(gran + kv::val_bias(L, tok, g)) = (uint16_t)bf16_bits(mn);
    }
  }
}

template <int BITS, int D, int GS, bool F16>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvArgs a) {
  constexpr kv::Layout L = kv::layout(BITS, D, GS);
  const Place p = place_of<D>(a);
  if (p.row >= a.rows) return;
  const bool val = blockIdx.y != 0;
  int64_t off = 0;
  int tok = 0;
  uint32_t o[4] = {0, 0, 0, 0};
  if (granule_of(a, __ldg(a.slots + p.t), p.h, L.granule, &off, &tok)) {
    const unsigned char *gran = a.cache + off;
    uint32_t words[BITS / 4];
    const int g = p.l / (GS / 8);
    float s, b;
    if (!val) {
#pragma unroll
      for (int i = 0; i < BITS / 4; i++)
        words[i] = *reinterpret_cast<const uint32_t *>(gran + kv::key_word(L, tok, p.l * (BITS / 4) + i));
      const uint32_t m = *reinterpret_cast<const uint32_t *>(gran + kv::key_meta(L, tok, g));
      s = bf16_lo(m);
      b = bf16_hi(m);
    } else {
#pragma unroll
      for (int i = 0; i < BITS / 4; i++) {
        const int w = p.l * (BITS / 4) + i;
        words[i] = (uint32_t)*reinterpret_cast<const uint16_t *>(gran + kv::val_half(L, tok, 2 * w)) |
                   (uint32_t)*reinterpret_cast<const uint16_t *>(gran + kv::val_half(L, tok, 2 * w + 1)) << 16;
      }
      s = bf16_lo(*reinterpret_cast<const uint16_t *>(gran + kv::val_scale(L, tok, g)));
      b = bf16_lo(*reinterpret_cast<const uint16_t *>(gran + kv::val_bias(L, tok, g)));
    }
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      // a code in the low bits of 2^23's significand, made a number by a subtraction (exact)
      const uint32_t q = ((words[j * BITS / 32] >> (j * BITS % 32)) & ((1u << BITS) - 1u)) | 0x4b000000u;
      f[j] = __fmaf_rn(__fsub_rn(__uint_as_float(q), 8388608.0f), s, b);   // fp32(code * scale + bias)
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if constexpr (F16) {
        const __half2 h = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
  }
  uint16_t *dst = (val ? a.vo : a.ko) + (int64_t)p.row * D + p.l * 8;
  *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <int BITS, int D, int GS>
void launch(const KvArgs &a, bool f16, bool write, cudaStream_t st) {
  constexpr uint32_t per = kThreads / (D / 8);          // rows of a block
  const dim3 grid((a.rows + per - 1) / per, 2);
  if (write) {
    if (f16) k_kv_write<BITS, D, GS, true><<<grid, kThreads, 0, st>>>(a);
    else k_kv_write<BITS, D, GS, false><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (f16) k_kv_read<BITS, D, GS, true><<<grid, kThreads, 0, st>>>(a);
    else k_kv_read<BITS, D, GS, false><<<grid, kThreads, 0, st>>>(a);
  }
}

void dispatch(const KvArgs &a, int D, int bits, int gs, bool f16, bool write, cudaStream_t st) {
#define GWB_KV(B, DD, S) \
  if (bits == B && D == DD && gs == S) return launch<B, DD, S>(a, f16, write, st);
  GWB_KV(4, 64, 32) GWB_KV(4, 64, 64)
  GWB_KV(4, 128, 32) GWB_KV(4, 128, 64) GWB_KV(4, 128, 128)
  GWB_KV(4, 256, 32) GWB_KV(4, 256, 64) GWB_KV(4, 256, 128)
  GWB_KV(8, 64, 32) GWB_KV(8, 64, 64)
  GWB_KV(8, 128, 32) GWB_KV(8, 128, 64) GWB_KV(8, 128, 128)
  GWB_KV(8, 256, 32) GWB_KV(8, 256, 64) GWB_KV(8, 256, 128)
#undef GWB_KV
}

}  // namespace

int64_t kv_granule_bytes(int head_dim, int bits, int gs) { return kv::layout(bits, head_dim, gs).granule; }

void launch_kv_write(const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride, const int64_t *slots,
                     int64_t T, const KvCache &c, bool f16, cudaStream_t st) {
  KvArgs a{};
  a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride;
  a.slots = slots; a.rows = (uint32_t)(T * c.heads);
  a.cache = static_cast<unsigned char *>(c.data);
  a.total_slots = c.pages * c.page_size;
  a.H = (int)c.heads;
  while ((1 << a.page_shift) < c.page_size) a.page_shift++;
  dispatch(a, c.head_dim, c.bits, c.gs, f16, true, st);
}

void launch_kv_read(const KvCache &c, const int64_t *slots, int64_t T, uint16_t *k, uint16_t *v, bool f16,
                    cudaStream_t st) {
  KvArgs a{};
  a.ko = k; a.vo = v;
  a.slots = slots; a.rows = (uint32_t)(T * c.heads);
  a.cache = static_cast<unsigned char *>(c.data);
  a.total_slots = c.pages * c.page_size;
  a.H = (int)c.heads;
  while ((1 << a.page_shift) < c.page_size) a.page_shift++;
  dispatch(a, c.head_dim, c.bits, c.gs, f16, false, st);
}

}  // namespace gwb
