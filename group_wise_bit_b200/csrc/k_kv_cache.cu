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

namespace gwb {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;

// Monotone map of finite floats to int32 under the total order -0 < +0 (as qpack_affine).
__device__ __forceinline__ int order_key(float f) {
  const int i = __float_as_int(f);
  return i >= 0 ? i : (i ^ 0x7fffffff);
}
__device__ __forceinline__ float key_to_float(int k) { return __int_as_float(k >= 0 ? k : (k ^ 0x7fffffff)); }
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
  int64_t T, total_slots;
  int H, page_size;
};

// This lane's place: row (token, head, key / value) and element 8 * l in it.
struct Place {
  int64_t t;
  int h, what, l;
  bool in;
};
template <int D>
__device__ __forceinline__ Place place_of(const KvArgs &a) {
  constexpr int LR = D / 8;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LR;
  Place p;
  p.l = threadIdx.x % LR;
  p.what = (int)(i & 1);
  const int64_t th = i >> 1;
  p.t = th / a.H;
  p.h = (int)(th - p.t * a.H);
  p.in = p.t < a.T;
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
  const int64_t page = slot / a.page_size;
  const int in_page = (int)(slot - page * a.page_size);
  *off = ((page * a.H + h) * (a.page_size / kv::kTok) + in_page / kv::kTok) * (int64_t)granule;
  *tok = in_page % kv::kTok;
  return true;
}

template <int BITS, int D, int GS, bool F16>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvArgs a) {
  constexpr kv::Layout L = kv::layout(BITS, D, GS);
  constexpr int LG = GS / 8;              // lanes of a group
  constexpr float QMAX = (float)((1 << BITS) - 1);
  const Place p = place_of<D>(a);
  int64_t off = 0;
  int tok = 0;
  const bool live = p.in && granule_of(a, __ldg(a.slots + p.t), p.h, L.granule, &off, &tok);
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (live) {
    const uint16_t *row = p.what ? a.v + p.t * a.v_stride : a.k + p.t * a.k_stride;
    unpack8<F16>(*reinterpret_cast<const uint4 *>(row + p.h * D + p.l * 8), v);
  }
  int kmin = order_key(v[0]), kmax = kmin;
#pragma unroll
  for (int j = 1; j < 8; j++) {
    kmin = min(kmin, order_key(v[j]));
    kmax = max(kmax, order_key(v[j]));
  }
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) {
    kmin = min(kmin, __shfl_xor_sync(kFull, kmin, o));
    kmax = max(kmax, __shfl_xor_sync(kFull, kmax, o));
  }
  if (!live) return;
  const float mn = key_to_float(kmin), mx = key_to_float(kmax);
  const float s = __fdiv_rn(__fsub_rn(mx, mn), QMAX);
  uint32_t words[BITS / 4] = {};
#pragma unroll
  for (int j = 0; j < 8; j++) {
    uint32_t q = 0;
    if (s != 0.0f) q = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[j], mn), s)), 0.0f), QMAX);
    words[j * BITS / 32] |= q << (j * BITS % 32);
  }
  unsigned char *gran = a.cache + off;
#pragma unroll
  for (int i = 0; i < BITS / 4; i++) {
    const int w = p.l * (BITS / 4) + i;
    if (p.what == 0) {
      *reinterpret_cast<uint32_t *>(gran + kv::key_word(L, tok, w)) = words[i];
    } else {
      *reinterpret_cast<uint16_t *>(gran + kv::val_half(L, tok, 2 * w)) = (uint16_t)words[i];
      *reinterpret_cast<uint16_t *>(gran + kv::val_half(L, tok, 2 * w + 1)) = (uint16_t)(words[i] >> 16);
    }
  }
  if (p.l % LG == 0) {
    const int g = p.l / LG;
    if (p.what == 0) {
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
  if (!p.in) return;
  int64_t off = 0;
  int tok = 0;
  uint32_t o[4] = {0, 0, 0, 0};
  if (granule_of(a, __ldg(a.slots + p.t), p.h, L.granule, &off, &tok)) {
    const unsigned char *gran = a.cache + off;
    uint32_t words[BITS / 4];
#pragma unroll
    for (int i = 0; i < BITS / 4; i++) {
      const int w = p.l * (BITS / 4) + i;
      if (p.what == 0)
        words[i] = *reinterpret_cast<const uint32_t *>(gran + kv::key_word(L, tok, w));
      else
        words[i] = (uint32_t)*reinterpret_cast<const uint16_t *>(gran + kv::val_half(L, tok, 2 * w)) |
                   (uint32_t)*reinterpret_cast<const uint16_t *>(gran + kv::val_half(L, tok, 2 * w + 1)) << 16;
    }
    const int g = p.l / (GS / 8);
    float s, b;
    if (p.what == 0) {
      const uint32_t m = *reinterpret_cast<const uint32_t *>(gran + kv::key_meta(L, tok, g));
      s = bf16_lo(m);
      b = bf16_hi(m);
    } else {
      s = bf16_lo(*reinterpret_cast<const uint16_t *>(gran + kv::val_scale(L, tok, g)));
      b = bf16_lo(*reinterpret_cast<const uint16_t *>(gran + kv::val_bias(L, tok, g)));
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint32_t q = (words[j * BITS / 32] >> (j * BITS % 32)) & ((1u << BITS) - 1u);
      const float f = __fmaf_rn((float)q, s, b);   // fp32(code * scale + bias), then the output's rounding
      const uint32_t h = F16 ? (uint32_t)__half_as_ushort(__float2half_rn(f)) : bf16_bits(f);
      o[j / 2] |= h << (j % 2 * 16);
    }
  }
  uint16_t *dst = (p.what ? a.vo : a.ko) + (p.t * a.H + p.h) * D + p.l * 8;
  *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <int BITS, int D, int GS>
void launch(const KvArgs &a, bool f16, bool write, cudaStream_t st) {
  const int64_t rows = a.T * a.H * 2;
  const unsigned grid = (unsigned)((rows * (D / 8) + kThreads - 1) / kThreads);
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
  a.slots = slots; a.T = T;
  a.cache = static_cast<unsigned char *>(c.data);
  a.total_slots = c.pages * c.page_size;
  a.H = (int)c.heads; a.page_size = (int)c.page_size;
  dispatch(a, c.head_dim, c.bits, c.gs, f16, true, st);
}

void launch_kv_read(const KvCache &c, const int64_t *slots, int64_t T, uint16_t *k, uint16_t *v, bool f16,
                    cudaStream_t st) {
  KvArgs a{};
  a.ko = k; a.vo = v;
  a.slots = slots; a.T = T;
  a.cache = static_cast<unsigned char *>(c.data);
  a.total_slots = c.pages * c.page_size;
  a.H = (int)c.heads; a.page_size = (int)c.page_size;
  dispatch(a, c.head_dim, c.bits, c.gs, f16, false, st);
}

}  // namespace gwb
