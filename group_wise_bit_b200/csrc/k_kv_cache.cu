// Writing tokens' keys and values into the paged, quantized cache, and reading
// rows of it back.
//
// A block takes 16 tokens, keys or values, and some heads in turn: 16 consecutive
// elements of a row (32 bytes of bf16 or fp16) belong to one thread, D / 16
// threads hold a row, and a thread's token, slot and place in the granule stay the
// same from head to head.  The arithmetic is qpack_affine's (fp32, one IEEE
// rounding a step, bf16 scale and bias): the gs / 16 threads of a group find its
// min and max with shuffles, and codes, scales and biases are bit-exact.
//
// Where a block's 16 slots are one granule, as in a prompt, its codes and metadata
// go through shared memory in the cache's order and move in 16-byte pieces; else
// every thread moves its own 2- and 4-byte units.  8192 tokens of 8 heads x 128 at
// 8 bits, every buffer out of L2: write 13.2 us (13.7 from slices of a fused
// projection), read 13.8, against 7.9 each for their 51 MB; at 4 bits 12.5 and 12.9
// against 6.6; 32768 tokens at 8 bits 44 and 46 against 31.5.  A last tile that is
// no whole granule costs the write 4 us more (8155 tokens: 17.6), its block's small
// units head after head; tiles of padding cost nothing.  The write spends 18 issue
// slots an element, about 8 of them the quantizer's (unpacking, min, max, quotient,
// rounding, packing), the rest addresses, 2-byte staging of the values and barriers,
// and has 69 % of its active cycles' slots busy; the read spends 12 and has 57 %,
// with loads and barriers in front of the rest.  (34 us with 8 elements a thread and
// 2-byte stores.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv_layout.cuh"
#include "ptx.cuh"
#include "quotient.cuh"

namespace gwb {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kE = 16;                    // elements of a thread
// Threads of an SM that the registers are shared out for (64 and 56 a thread).  us at 8192 tokens of 8 x 128, 8 bits:
// write 15.5 with the compiler's 80 registers, 13.9 with 64, 15.9 with 48; read of 20011 tokens of 4 x 64, 4 bits:
// 10.0 with 64, 8.8 with 56 or 48, and of 3000 tokens of 32 x 128, 8 bits: 18.6 with 56, 23.2 with 48.
constexpr int kWriteThreads = 1024, kReadThreads = 1152;
constexpr int kBlockCost = 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &u, float *v) {
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
  int H, page_shift;
  int heads;                   // of a block
};

// A thread's place: token t, element kE * l of a row, heads
// [h0, h1); blockIdx.y: keys or values.
struct Place {
  int64_t t, gran;             // token; granule of its slot in head 0
  int l, h0, h1, tok;          // tok: place in the granule
  bool live, whole;            // the slot is in the cache; the block's slots are one granule
};
template <int D>
__device__ __forceinline__ Place place_of(const KvArgs &a) {
  constexpr int LR = D / kE;
  Place p;
  const int i = threadIdx.x / LR;
  const int64_t t0 = (int64_t)blockIdx.x * kv::kTok;
  p.t = t0 + i;
  p.l = threadIdx.x % LR;
  p.h0 = blockIdx.z * a.heads;
  p.h1 = min(a.H, p.h0 + a.heads);
  // a slot outside the cache is left out: negative (a padded row), or beyond it (an error)
  int64_t slot = -1;
  if (p.t < a.T) slot = __ldg(a.slots + p.t);
  const int64_t first = __ldg(a.slots + t0);
  if (slot >= a.total_slots) {
    atomicOr(&g_device_error, kErrIndex);
    slot = -1;
  }
  p.live = slot >= 0;
  const int64_t page = slot >> a.page_shift;
  const int in_page = (int)slot & ((1 << a.page_shift) - 1);
  p.gran = (page * a.H << (a.page_shift - 4)) + in_page / kv::kTok;
  p.tok = in_page % kv::kTok;
  p.whole = __syncthreads_and(p.live && slot - i == first && first % kv::kTok == 0);
  return p;
}

// The keys' or values' part of a granule as one buffer: codes, then metadata.
template <int BITS, int D, int GS>
struct Part {
  static constexpr int kCode = kv::layout(BITS, D, GS).code_bytes, kMeta = 64 * (D / GS), kBytes = kCode + kMeta;
  static constexpr int kGranule = kv::layout(BITS, D, GS).granule;
  // address of byte i of the buffer in the granule
  static __device__ __forceinline__ unsigned char *at(unsigned char *gran, bool val, int i) {
    return i < kCode ? gran + (val ? kCode : 0) + i : gran + 2 * kCode + (val ? kMeta : 0) + (i - kCode);
  }
  // byte offsets in the codes, and in the metadata
  static __device__ __forceinline__ int word(int tok, int w) {
    constexpr kv::Layout l = kv::layout(BITS, D, GS);
    return kv::key_word(l, tok, w);
  }
  static __device__ __forceinline__ int half(int tok, int h) {
    constexpr kv::Layout l = kv::layout(BITS, D, GS);
    return kv::val_half(l, tok, h) - kCode;
  }
  static __device__ __forceinline__ int kmeta(int tok, int g) {
    constexpr kv::Layout l = kv::layout(BITS, D, GS);
    return kv::key_meta(l, tok, g) - 2 * kCode;
  }
  static __device__ __forceinline__ int vscale(int tok, int g) {
    constexpr kv::Layout l = kv::layout(BITS, D, GS);
    return kv::val_scale(l, tok, g) - 2 * kCode - kMeta;
  }
  static __device__ __forceinline__ int vbias(int tok, int g) {
    constexpr kv::Layout l = kv::layout(BITS, D, GS);
    return kv::val_bias(l, tok, g) - 2 * kCode - kMeta;
  }
};

// Quantizes kE elements of a row whose group lies on LG neighbouring threads.
template <int BITS, int LG>
__device__ __forceinline__ void quantize(const float (&v)[kE], uint32_t (&words)[kE * BITS / 32], float &s, float &mn) {
  constexpr float QMAX = (float)((1 << BITS) - 1);
  // (min and max order -0 below +0, as qpack_affine's keys do; a NaN makes scale and bias NaN, its codes 0)
  float mx = max_nan(v[0], v[1]);
  mn = min_nan(v[0], v[1]);
#pragma unroll
  for (int j = 2; j < kE; j += 2) {
    mn = min_nan(mn, v[j], v[j + 1]);
    mx = max_nan(mx, v[j], v[j + 1]);
  }
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) {
    mn = min_nan(mn, __shfl_xor_sync(kFull, mn, o));
    mx = max_nan(mx, __shfl_xor_sync(kFull, mx, o));
  }
  s = quotient_const<(1 << BITS) - 1>(__fsub_rn(mx, mn));
  const Divisor d = make_divisor(s);
  if (d.fast) {
    // integers in the low bits of the rounded quotients; no code passes QMAX (quotients are within 2^-23 of it)
    float z[kE];
#pragma unroll
    for (int j = 0; j < kE; j++) z[j] = round_bits(quotient_fast(__fsub_rn(v[j], mn), d));
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < kE / 4; i++)
        words[i] = __byte_perm(__byte_perm(__float_as_uint(z[4 * i]), __float_as_uint(z[4 * i + 1]), 0x0040),
                               __byte_perm(__float_as_uint(z[4 * i + 2]), __float_as_uint(z[4 * i + 3]), 0x0040), 0x5410);
    } else {
      // four nibbles at a time in fp32: exact below 2^16
      uint32_t h[kE / 4];
#pragma unroll
      for (int i = 0; i < kE / 4; i++) {
        float n[4];
#pragma unroll
        for (int j = 0; j < 4; j++) n[j] = __fsub_rn(z[4 * i + j], kRoundMagic);
        h[i] = __float_as_uint(round_bits(fmaf(fmaf(n[3], 16.0f, n[2]), 256.0f, fmaf(n[1], 16.0f, n[0]))));
      }
#pragma unroll
      for (int i = 0; i < kE / 8; i++) words[i] = __byte_perm(h[2 * i], h[2 * i + 1], 0x5410);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kE * BITS / 32; i++) words[i] = 0;
#pragma unroll
    for (int j = 0; j < kE; j++) {
      uint32_t q = 0;
      if (s != 0.0f) q = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[j], mn), s)), 0.0f), QMAX);
      words[j * BITS / 32] |= q << (j * BITS % 32);
    }
  }
}

template <int BITS, int D, int GS, bool F16>
__global__ void __launch_bounds__(D, kWriteThreads / D) k_kv_write(const KvArgs a) {
  using P = Part<BITS, D, GS>;
  constexpr int LG = GS / kE;             // threads of a group
  constexpr int W = kE * BITS / 32;       // words of a thread
  __shared__ __align__(16) unsigned char buf[2][P::kBytes];
  const Place p = place_of<D>(a);
  const bool val = blockIdx.y != 0;
  const int64_t head_bytes = ((int64_t)P::kGranule << a.page_shift) / kv::kTok;
  unsigned char *gran = a.cache + p.gran * P::kGranule + p.h0 * head_bytes;
  const uint16_t *row = (val ? a.v + p.t * a.v_stride : a.k + p.t * a.k_stride) + p.l * kE + (int64_t)p.h0 * D;
  uint4 next[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  auto fetch = [&]() {
    next[0] = __ldg(reinterpret_cast<const uint4 *>(row));
    next[1] = __ldg(reinterpret_cast<const uint4 *>(row) + 1);
  };
  if (p.live) fetch();
  for (int h = p.h0; h < p.h1; h++, gran += head_bytes) {
    float v[kE], s, mn;
    unpack8<F16>(next[0], v);
    unpack8<F16>(next[1], v + 8);
    row += D;
    if (p.live && h + 1 < p.h1) fetch();
    uint32_t words[W];
    quantize<BITS, LG>(v, words, s, mn);
    // the units of this thread, into the buffer or straight into the cache
    unsigned char *b = buf[h & 1];
    auto put = [&](unsigned char *codes, unsigned char *meta) {   // where the codes and the metadata begin
      const int g = p.l / LG;
      if (!val) {
#pragma unroll
        for (int i = 0; i < W; i++) *reinterpret_cast<uint32_t *>(codes + P::word(p.tok, p.l * W + i)) = words[i];
        if (p.l % LG == 0)
          *reinterpret_cast<uint32_t *>(meta + P::kmeta(p.tok, g)) = bf16_bits(s) | (bf16_bits(mn) << 16);
      } else {
#pragma unroll
        for (int i = 0; i < W; i++) {
          const int w = p.l * W + i;
          *reinterpret_cast<uint16_t *>(codes + P::half(p.tok, 2 * w)) = (uint16_t)words[i];
          *reinterpret_cast<uint16_t *>(codes + P::half(p.tok, 2 * w + 1)) = (uint16_t)(words[i] >> 16);
        }
        if (p.l % LG == 0) {
          *reinterpret_cast<uint16_t *>(meta + P::vscale(p.tok, g)) = (uint16_t)bf16_bits(s);
          *reinterpret_cast<uint16_t *>(meta + P::vbias(p.tok, g)) = (uint16_t)bf16_bits(mn);
        }
      }
    };
    if (p.whole) {
      put(b, b + P::kCode);
      __syncthreads();                    // (the other buffer's readers have passed the barrier in front)
      for (int i = threadIdx.x; i < P::kBytes / 16; i += D)
        *reinterpret_cast<uint4 *>(P::at(gran, val, i * 16)) = reinterpret_cast<const uint4 *>(b)[i];
    } else if (p.live) {
      put(P::at(gran, val, 0), P::at(gran, val, P::kCode));
    }
  }
}

template <int BITS, int D, int GS, bool F16>
__global__ void __launch_bounds__(D, kReadThreads / D) k_kv_read(const KvArgs a) {
  using P = Part<BITS, D, GS>;
  __shared__ __align__(16) unsigned char buf[2][P::kBytes];
  constexpr int kPer = (P::kBytes / 16 + D - 1) / D, W = kE * BITS / 32;
  const Place p = place_of<D>(a);
  const bool val = blockIdx.y != 0;
  const int64_t head_bytes = ((int64_t)P::kGranule << a.page_shift) / kv::kTok;
  unsigned char *gran = a.cache + p.gran * P::kGranule + p.h0 * head_bytes;
  uint16_t *dst = (val ? a.vo : a.ko) + (p.t * a.H + p.h0) * D + p.l * kE;
  uint4 next[kPer];
  auto fetch = [&]() {
#pragma unroll
    for (int k = 0; k < kPer; k++) {
      const int i = threadIdx.x + k * D;
      if (i < P::kBytes / 16) next[k] = __ldg(reinterpret_cast<const uint4 *>(P::at(gran, val, i * 16)));
    }
  };
  if (p.whole) fetch();
  for (int h = p.h0; h < p.h1; h++, dst += D) {
    unsigned char *b = buf[h & 1];
    const unsigned char *here = gran;
    if (p.whole) {
#pragma unroll
      for (int k = 0; k < kPer; k++) {
        const int i = threadIdx.x + k * D;
        if (i < P::kBytes / 16) reinterpret_cast<uint4 *>(b)[i] = next[k];
      }
    }
    gran += head_bytes;
    if (p.whole) {
      if (h + 1 < p.h1) fetch();
      __syncthreads();                    // (the other buffer's readers have passed the barrier in front)
    }
    uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (p.live) {
      uint32_t words[W];
      float s, m;
      auto get = [&](const unsigned char *codes, const unsigned char *meta) {
        const int g = p.l / (GS / kE);
        if (!val) {
#pragma unroll
          for (int i = 0; i < W; i++) words[i] = *reinterpret_cast<const uint32_t *>(codes + P::word(p.tok, p.l * W + i));
          const uint32_t u = *reinterpret_cast<const uint32_t *>(meta + P::kmeta(p.tok, g));
          s = bf16_lo(u);
          m = bf16_hi(u);
        } else {
#pragma unroll
          for (int i = 0; i < W; i++) {
            const int w = p.l * W + i;
            words[i] = (uint32_t)*reinterpret_cast<const uint16_t *>(codes + P::half(p.tok, 2 * w)) |
                       (uint32_t)*reinterpret_cast<const uint16_t *>(codes + P::half(p.tok, 2 * w + 1)) << 16;
          }
          s = bf16_lo(*reinterpret_cast<const uint16_t *>(meta + P::vscale(p.tok, g)));
          m = bf16_lo(*reinterpret_cast<const uint16_t *>(meta + P::vbias(p.tok, g)));
        }
      };
      if (p.whole) {
        get(b, b + P::kCode);
      } else {
        unsigned char *from = const_cast<unsigned char *>(here);
        get(P::at(from, val, 0), P::at(from, val, P::kCode));
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
          // a code in the low bits of 2^23's significand, made a number by a subtraction (exact)
          const int i = 2 * j + e;
          const uint32_t q = ((words[i * BITS / 32] >> (i * BITS % 32)) & ((1u << BITS) - 1u)) | 0x4b000000u;
          f[e] = __fmaf_rn(__fsub_rn(__uint_as_float(q), 8388608.0f), s, m);   // fp32(code * scale + bias)
        }
        if constexpr (F16) {
          const __half2 x = __floats2half2_rn(f[0], f[1]);
          o[j] = *reinterpret_cast<const uint32_t *>(&x);
        } else {
          const __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]);
          o[j] = *reinterpret_cast<const uint32_t *>(&x);
        }
      }
    }
    if (p.t < a.T) {
      reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// Heads of a block: as many as make the whole launch shortest, where a block costs as much as two heads (its slots
// and first rows have to arrive) and the resident blocks go in rounds.  us, write / read, against as many heads as
// leave 8 blocks an SM: 4096 tokens of 2 x 256, 8 bits 7.3 / 7.2 -> 6.5 / 6.5; 3000 of 32 x 128 20.5 / 20.8 ->
// 18.7 / 18.4; 20011 of 4 x 64, 4 bits 12.3 / 10.3 -> 11.1 / 9.8 (all with 64 registers); a block's cost of one
// head instead of two: 32768 of 8 x 128 46.4 / 46.7, not 44.1 / 46.1.  Few tokens get one head a block.
int heads_of_block(int64_t tiles, int H, int64_t resident) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int h = 1; h <= H && h <= 64; h++) {
    const int64_t blocks = tiles * ((H + h - 1) / h), cost = (blocks + resident - 1) / resident * (2 * h + kBlockCost);
    if (cost < least) {
      least = cost;
      best = h;
    }
  }
  return best;
}

template <int BITS, int D, int GS>
void launch(KvArgs a, bool f16, bool write, cudaStream_t st) {
  const int64_t tiles = (a.T + kv::kTok - 1) / kv::kTok;
  a.heads = heads_of_block(2 * tiles, a.H, 148 * ((write ? kWriteThreads : kReadThreads) / D));
  const dim3 grid((unsigned)tiles, 2, (unsigned)((a.H + a.heads - 1) / a.heads));
  if (write) {
    if (f16) k_kv_write<BITS, D, GS, true><<<grid, D, 0, st>>>(a);
    else k_kv_write<BITS, D, GS, false><<<grid, D, 0, st>>>(a);
  } else {
    if (f16) k_kv_read<BITS, D, GS, true><<<grid, D, 0, st>>>(a);
    else k_kv_read<BITS, D, GS, false><<<grid, D, 0, st>>>(a);
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
  a.H = (int)c.heads;
  while ((1 << a.page_shift) < c.page_size) a.page_shift++;
  dispatch(a, c.head_dim, c.bits, c.gs, f16, true, st);
}

void launch_kv_read(const KvCache &c, const int64_t *slots, int64_t T, uint16_t *k, uint16_t *v, bool f16,
                    cudaStream_t st) {
  KvArgs a{};
  a.ko = k; a.vo = v;
  a.slots = slots; a.T = T;
  a.cache = static_cast<unsigned char *>(c.data);
  a.total_slots = c.pages * c.page_size;
  a.H = (int)c.heads;
  while ((1 << a.page_shift) < c.page_size) a.page_shift++;
  dispatch(a, c.head_dim, c.bits, c.gs, f16, false, st);
}

}  // namespace gwb
