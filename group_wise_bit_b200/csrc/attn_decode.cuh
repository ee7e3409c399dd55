// Attention of one new token a sequence over the paged, quantized cache
// (kv_layout.cuh), the length split over the whole GPU and joined.
//
// For query head h of kv head n, tokens t < len, groups g of the head dimension:
//   key   k[t,d] = ck[t,d] * sk[t,g] + bk[t,g]     (codes, bf16 scale and bias; value v alike)
//   S[t]  = sum_g sk[t,g] * (sum_{d in g} q[d] ck[t,d]) + bk[t,g] * (sum_{d in g} q[d])
//   out   = sum_t p[t] v[t] / sum_t p[t],   p[t] = 2^(S[t] * scale * log2 e - m),  m a running max
//   sum_t p v[t,d] = sum_t (p sv[t,g]) (cv[t,d] - Z) + sum_t p (bv[t,g] + Z sv[t,g]),  Z = 2^(bits-1)
// so neither keys nor values are ever dequantized: the codes are the MMA's
// operand and the group scales multiply 16-token score fragments and P.
//
// Work split.  The unit is two granules (32 tokens of one head, one contiguous
// bulk copy where a page holds both).  The units of all (sequence, head) pairs form one line, cut
// into equal shares, one a CTA; every CTA finds its share from the lengths on
// the device, so ragged batches and lengths that change between graph replays
// are balanced and the host never reads a length.  A (sequence, head) that is
// cut leaves one partial (fp32 sums, max, total) a piece, joined by a second,
// dependent launch in a fixed order (no atomics: results are reproducible).
// In a CTA the warps take units in turn, each streaming its own through a
// private ring of bulk copies, and join through shared memory.
//
// Codes enter the m16n8k16 fp16 MMA as subnormals: code bits in the low bits of
// an fp16 are code * 2^-24, exactly, so unpacking is one AND per register (two
// codes), with a shift for every other pair; the nibble at bits 4..7 stands for
// 16 * code and its q is divided by 16 (exact) or its sum at the end.  The sum of
// uncentred value codes is far larger than the result and the tensor core
// truncates what it adds (toward zero; a subnormal operand at its type's smallest
// normal exponent, 2^-14 of a code here), so every granule's sum is centred at once
// by an MMA with a constant operand of -Z: one issue slot where subtracting Z from
// the unpacked registers takes four.  With PREC the codes do go through 1024 + code
// and a subtraction instead, which makes them normal numbers and the products exact.
//
// What bounds it.  8-bit caches: memory (64 sequences of up to 8192 tokens, 8 kv
// heads x 128, 64 query heads: 132 us = 6.1 TB/s, 0.93 of a plain copy).  4-bit
// caches: the latency of dependent instructions in 12 warps an SM (the same at 4
// bits: 102 us = 4.2 TB/s).  A granule takes 286 issue slots, 80 of them masks and
// shifts of codes, 25 MMAs, where memory's time would leave room for 383; slots are
// 52 % busy, the tensor pipe 34 %, and the first stall is the fixed latency (31 %).
// fp16 outputs (PREC) add MMAs: 126 us at 4 bits, 146 at 8.  Short calls: the chain
// lengths, page ids, codes, queries, join (1 sequence of 128 tokens: 5 us).
// Slower, and left out: e4m3 MMAs for the keys (a nibble is an e4m3 number; 131
// against 112 us, with more instructions and fp16 MMAs counted, not fewer), a
// granule's values beside the next one's scores (117), four CTAs an SM (115), the
// shifts as multiplications (121), shares half or a third as long (118, 124).
//
// Precision.  q is scaled by a power of two per head into fp16 (exact for bf16
// and fp16 but for elements 2^-22 below the largest).  Scores, maxima, totals
// and outputs are fp32; a score's MMA truncates at 2^-14 of a code step of its
// largest |q|, well below what fp16 does to p.  p is rounded to fp16 (2^-11) before it meets the codes,
// p * sv again, and the centred bias bv + Z sv too: 2^-11 of each, against the
// 2^-8 of a bf16 output.  With PREC (fp16 outputs, whose own rounding is 2^-11)
// the remainders of all three roundings take part: p and p * sv through a second
// MMA, the biases' in rows of their MMA that are free.  Value scales and
// biases are normalized by a running power of two a group, so fp16's range
// limits nothing but ratios inside one group's column: a value below 2^-14 of
// the largest that the column has met loses bits (fp16's subnormals), whatever
// the larger one's weight.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv_layout.cuh"
#include "ptx.cuh"

namespace gwb {
namespace {
namespace attn {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLogP = 10.0f;      // P = p * 2^10 in fp16
constexpr float kLogPMax = 14.0f;   // a larger P moves the running max
constexpr int kLogB = 11;           // the remainders of the biases are held times 2^kLogB

struct Args {
  const uint16_t *q;
  int64_t q_stride;             // elements between sequences
  const unsigned char *cache;
  const int32_t *table;         // [B][table_stride] page ids
  int64_t table_stride;
  const int32_t *lens;          // [B]
  uint16_t *out;                // [B][H * G][D]
  float *lse;                   // [B][H * G] or NULL
  float *ws;                    // partials, then records (see Ws)
  int64_t pages;
  int B, H, G, GH;              // GH: query heads of one chunk
  int chunks;                   // chunks of a kv head's G query heads
  int gshift, cap;              // log2 of a page's granules; tokens a table row can name
  int ushift;                   // log2 of a unit's granules
  int depth;                    // ring slots a warp
  int min_per;                  // least places of a share
  int f16;
  int mode;                     // AttnMode
  float scale_log2;             // softmax scale * log2 e * 2^12
};

// One record a CTA, for the join: the pair that the boundary in front of its share cuts, where no
// earlier boundary does.
struct Rec {
  int b, hc, pieces, pad;       // sequence, head chunk, pieces of the pair from share i - 1 on (0: nothing to join)
};
// Workspace: [2 * CTAs] partials of GHP heads x (D sums, max, total), then [CTAs] Rec, then the share size.
template <int D, int GHP>
struct Ws {
  static constexpr int kPart = GHP * (D + 2);   // floats of a partial
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" :::); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D[16 x 8] += A[16 x 16] * B[16 x 8], fp16 operands, fp32 accumulator.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(   // (not volatile: the compiler may interleave independent chains)
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A * B (no registers to clear).
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hadd2u(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                            *reinterpret_cast<const __half2 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// Larger of two pairs of unsigned 16-bit numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// 2^n, n clamped into fp32's normal range.
__device__ __forceinline__ float p2(int n) { return pow2f(max(-126, min(127, n))); }

__device__ __forceinline__ float q_at(const uint16_t *p, int f16) {
  return f16 ? __half2float(__ushort_as_half(*p)) : __uint_as_float((uint32_t)*p << 16);
}

// The line of work.  A pair (sequence, head chunk) of n units takes
// kPieceCost + n places: opening a piece (staging q, joining the warps) costs
// about as much as kPieceCost units do, so shares of many short sequences
// stay level with shares of long ones.  A share that begins inside a pair's first
// kPieceCost places begins at its unit 0; one that ends there leaves the pair
// to the next share.
constexpr int kPieceCost = 16;

// Where the share of a CTA begins, and its length.
struct Start {
  int b, hc, u, pad;             // sequence, head chunk and place in the pair
  long long left, per;           // places of this share (0: nothing to do), of every share but the last
};

// Tokens of sequence b, cut to what its table row can name.
__device__ __forceinline__ int tokens(const Args &a, int b, bool report) {
  const int len = max(0, __ldg(a.lens + b));
  if (len > a.cap && report) atomicOr(&g_device_error, kErrIndex);
  return min(len, a.cap);
}
__device__ __forceinline__ int units(const Args &a, int len) {
  const int s = 4 + a.ushift;
  return (len >> s) + ((len & ((1 << s) - 1)) != 0);
}
__device__ __forceinline__ long long places(int n) { return n > 0 ? n + kPieceCost : 0; }

// Every thread sums a run of the lengths, a scan joins them.
__device__ __forceinline__ void find_start(const Args &a, Start *st, long long *scan) {
  const int tid = threadIdx.x, HC = a.H * a.chunks;
  const int run = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
  long long mine = 0;
  for (int b = b0; b < b1; b++) mine += places(units(a, tokens(a, b, blockIdx.x == 0)));
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(kFull, inc, o);
    if ((tid & 31) >= o) inc += t;
  }
  if ((tid & 31) == 31) scan[tid >> 5] = inc;
  if (tid == 0) st->left = 0;
  __syncthreads();
  long long before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < (tid >> 5)) before += scan[w];
    total += scan[w];
  }
  before *= HC;
  total *= HC;
  const long long per = max((long long)a.min_per, (total + gridDim.x - 1) / gridDim.x);
  const long long first = per * blockIdx.x;
  if (first < total && first >= before && first < before + mine * HC) {
    long long left = first - before;
    for (int b = b0; b < b1; b++) {
      const long long n = places(units(a, tokens(a, b, false)));
      if (left < n * HC) {
        st->b = b;
        st->hc = (int)(left / n);
        st->u = (int)(left - (long long)st->hc * n);
        st->left = min(per, total - first);
        st->per = per;
        break;
      }
      left -= n * HC;
    }
  }
  __syncthreads();
}

// A walk over the pieces of a share.  The CTA has one (step 1); each warp has
// one for its copies, which takes every kWarps-th unit of a piece.
struct Cursor {
  int b, hc, n;                 // pair, units of the sequence
  int g, end;                   // units [g, end) of the piece are left to this walker
  int len;                      // tokens of the sequence
  long long left;               // places of the share behind this piece
  int head;                     // granules of a page in front of the pair's head
  const int32_t *row;           // the sequence's page ids
  int page0, page1;             // page ids of unit g's granules (loaded one unit ahead)
};

// Whether the unit has a second granule with a token in front of the length (else that one's page may not exist).
__device__ __forceinline__ bool cursor_two(const Args &a, const Cursor &c) {
  return a.ushift != 0 && (2 * c.g + 1) * kv::kTok < c.len;
}
__device__ __forceinline__ void cursor_page(const Args &a, Cursor &c) {
  if (c.g < c.end) {
    const int i = c.g << a.ushift;
    c.page0 = c.page1 = __ldg(c.row + (i >> a.gshift));
    if (a.gshift == 0 && cursor_two(a, c)) c.page1 = __ldg(c.row + i + 1);
  }
}
// Opens the piece at place u of (b, hc), skipping empty sequences; false when the share ends in front of it.
template <int GB, bool PAGES = true>
__device__ __forceinline__ bool cursor_open(const Args &a, Cursor &c, int u, int first) {
  c.g = c.end = 0;
  while (c.left > 0 && c.b < a.B) {
    c.len = tokens(a, c.b, false);
    c.n = units(a, c.len);
    if (c.n > 0) {
      const int g = max(0, u - kPieceCost);
      c.left -= max(0, kPieceCost - u);
      const int len = (int)min((long long)(c.n - g), c.left);
      if (len <= 0) break;
      c.left -= len;
      c.end = g + len;
      c.g = g + first;
      c.head = (c.hc / a.chunks) << a.gshift;
      c.row = a.table + (int64_t)c.b * a.table_stride;
      if constexpr (PAGES) cursor_page(a, c);
      return true;
    }
    c.b++;
    c.hc = 0;
  }
  c.left = 0;
  return false;
}
template <int GB, bool PAGES = true>
__device__ __forceinline__ bool cursor_next_piece(const Args &a, Cursor &c, int first) {
  if (++c.hc == a.H * a.chunks) {
    c.hc = 0;
    c.b++;
  }
  return cursor_open<GB, PAGES>(a, c, 0, first);
}
// Leaves a warp's cursor on a granule of its own, or at the end (g >= end, left == 0).
template <int GB>
__device__ __forceinline__ void cursor_settle(const Args &a, Cursor &c, int first) {
  while (c.g >= c.end && c.left > 0) cursor_next_piece<GB>(a, c, first);
}

// Granules of a unit: two, for the sake of what a unit costs besides its tokens and of two independent chains of
// products; one where two rings of two would leave an SM with one CTA (8 bits, head_dim 256).
constexpr int unit_granules(int granule) { return granule > 8192 ? 1 : 2; }

// Resident CTAs an SM that the registers are held to: 12 warps where 168
// registers a thread hold the state, 8 (255 registers) where it takes more.  Shared
// memory may allow fewer: 8 bits at head_dim 128 has ring slots of 35 KB for its
// four warps, and two CTAs fit.
constexpr int min_ctas(int D, int NT) { return D * NT <= 128 ? 3 : 2; }

template <int BITS, int D, int GS, int NT, bool PREC>
struct Kernel {
  static constexpr kv::Layout L = kv::layout(BITS, D, GS);
  static constexpr int NG = L.NG;
  static constexpr int GB = L.granule;
  static constexpr int UG = unit_granules(L.granule);     // granules of a unit
  static constexpr int kUnit = UG * kv::kTok;             // tokens of a unit
  static constexpr int kSlot = UG * GB;                   // bytes of a ring slot
  static constexpr int KM = D / 16;                       // score MMAs a granule and n-tile
  static constexpr int VB = BITS == 4 ? D / 32 : D / 16;  // value blocks (8 lanes x 16 bits a token)
  static constexpr int MPB = BITS == 4 ? 2 : 1;           // MMAs a value block
  static constexpr int DB = D / VB;                       // dimensions of a value block
  static constexpr int GHP = 8 * NT;
  static constexpr int SROW = D + 4;                      // floats of a head's row in the join buffer
  static constexpr int kJoin = kWarps * GHP * (SROW + 2) * 4;

  // Pairs of tokens whose value scale and bias a lane converts a unit: word i = lane + 32 k of the
  // unit's kMW, of granule i / (8 NG), group i / 8 % NG.
  static constexpr int kMW = 8 * NG * UG, MW = (kMW + 31) / 32;
  // One warp's state of the current piece.
  struct State {
    float acc[VB * MPB][NT][4];
    // of row r < NG, group r: [0], [1] sum of P * (bias + Z scale), with PREC [2], [3] of P * 2^kLogB times what
    // the rounding of those biases left
    float bacc[NT][4];
    float m10[NT][2], l[NT][2];   // running max (log2, minus kLogP) and this lane's total, heads 8 nt + 2c, +1
    int E[NG];                    // value scales and biases are held over 2^E
    float fs[MW], fb[MW];         // 2^(BITS - E), 2^-E of the groups this lane converts (convert_meta),
    uint32_t lim_s[MW], lim_b[MW];   // and the largest scale and |bias| (bf16 bits, in both halves) that 2^E holds
  };
  static constexpr int kMeta = (PREC ? 12 : 8) * kMW;   // bytes of a warp's converted scales and biases
  static constexpr int kQ = GHP * D * 2;              // bytes of a piece's queries
  static __device__ __forceinline__ int meta_group(int k) { return (((threadIdx.x & 31) + 32 * k) / 8) % NG; }

  static __device__ __forceinline__ void set_exponent(State &s, int g, int e) {
    s.E[g] = e;
#pragma unroll
    for (int k = 0; k < MW; k++)
      if (meta_group(k) == g) {
        s.fs[k] = p2(BITS - e);
        s.fb[k] = p2(-e);
        s.lim_s[k] = ((uint32_t)(max(0, 127 + e - BITS) << 7) - 1u) * 0x10001u;
        s.lim_b[k] = ((uint32_t)((127 + e) << 7) - 1u) * 0x10001u;
      }
  }

  static __device__ __forceinline__ void reset(State &s) {
#pragma unroll
    for (int i = 0; i < VB * MPB; i++)
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int j = 0; j < 4; j++) s.acc[i][t][j] = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
      for (int j = 0; j < 4; j++) s.bacc[t][j] = 0.0f;
      s.m10[t][0] = s.m10[t][1] = -INFINITY;
      s.l[t][0] = s.l[t][1] = 0.0f;
    }
#pragma unroll
    for (int g = 0; g < NG; g++) set_exponent(s, g, -100);
  }

  // Zeroes the value scales and biases behind the length (the cache may hold
  // anything there, and 0 * NaN is NaN); a fence orders it before the slot's next copy.
  static __device__ __forceinline__ void clear_tail(unsigned char *sm, int valid) {
    uint16_t *meta = reinterpret_cast<uint16_t *>(sm + 2 * L.code_bytes + 64 * NG);
    for (int i = threadIdx.x & 31; i < 2 * NG * 16; i += 32)
      if (i % 16 >= valid) meta[i] = 0;
    fence_proxy_async_smem();
    __syncwarp();
  }

  // Scores of the two granules: 16 tokens x 8 heads a tile, fp32, a group at a
  // time.  The granules' MMA chains are independent and stand side by side (an
  // MMA's result takes 25 cycles, its issue slot 8).
  static __device__ __forceinline__ void scores(const unsigned char *sm, const uint32_t (&qf)[KM][NT][2],
                                                const float (&qsum)[NG][NT][2], float (&sc)[UG][NT][4]) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    constexpr int WG = GS * BITS / 128;             // words (of a lane's row) a group
    const unsigned char *meta = sm + 2 * L.code_bytes + r * NG * 4;
    const unsigned char *row = sm + (r * 4 + c) * L.VW * 4;
    constexpr int MV = NG < 4 ? NG : 4;             // groups of a meta load
    float ga[UG][NT][4];
    uint32_t km[UG][2][MV];
#pragma unroll
    for (int a = 0; a < L.NW / (4 * L.VW); a++) {
      uint32_t w[UG][2][4];                         // [granule][row r, r + 8][word]
#pragma unroll
      for (int h = 0; h < UG; h++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const unsigned char *p = row + h * GB + (a * 16 + 8 * k) * 4 * L.VW * 4;
          if constexpr (L.VW == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[h][k][0] = u.x; w[h][k][1] = u.y; w[h][k][2] = u.z; w[h][k][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[h][k][0] = u.x; w[h][k][1] = u.y;
          }
        }
#pragma unroll
      for (int v = 0; v < L.VW; v++) {
        const int i = a * L.VW + v;                 // word column 4 i + c of the row
        if constexpr (BITS == 4) {
#pragma unroll
          for (int k = 0; k < 2; k++)
#pragma unroll
            for (int h = 0; h < UG; h++) {
              const uint32_t x0 = w[h][0][v] >> (8 * k), x1 = w[h][1][v] >> (8 * k);
              const uint32_t m0 = 0x000f000fu, m1 = 0x00f000f0u;
#pragma unroll
              for (int t = 0; t < NT; t++) {
                const uint32_t(&q)[2] = qf[2 * i + k][t];
                if (i % WG == 0 && k == 0) mma0(ga[h][t], x0 & m0, x1 & m0, x0 & m1, x1 & m1, q[0], q[1]);
                else mma(ga[h][t], x0 & m0, x1 & m0, x0 & m1, x1 & m1, q[0], q[1]);
              }
            }
        } else {
#pragma unroll
          for (int h = 0; h < UG; h++) {
            const uint32_t x0 = w[h][0][v], x1 = w[h][1][v], m0 = 0x00ff00ffu;
#pragma unroll
            for (int t = 0; t < NT; t++) {
              const uint32_t(&q)[2] = qf[i][t];
              if (i % WG == 0) mma0(ga[h][t], x0 & m0, x1 & m0, (x0 >> 8) & m0, (x1 >> 8) & m0, q[0], q[1]);
              else mma(ga[h][t], x0 & m0, x1 & m0, (x0 >> 8) & m0, (x1 >> 8) & m0, q[0], q[1]);
            }
          }
        }
        if (i % WG == WG - 1) {
          const int g = i / WG;
#pragma unroll
          for (int h = 0; h < UG; h++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
              if (g % MV == 0) {
                const unsigned char *p = meta + h * GB + (8 * k * NG + g) * 4;
                if constexpr (MV == 4) {
                  const uint4 u = *reinterpret_cast<const uint4 *>(p);
                  km[h][k][0] = u.x; km[h][k][1] = u.y; km[h][k][2] = u.z; km[h][k][3] = u.w;
                } else if constexpr (MV == 2) {
                  const uint2 u = *reinterpret_cast<const uint2 *>(p);
                  km[h][k][0] = u.x; km[h][k][1] = u.y;
                } else {
                  km[h][k][0] = *reinterpret_cast<const uint32_t *>(p);
                }
              }
              const uint32_t m = km[h][k][g % MV];
              const float ms = bf_lo(m), mb = bf_hi(m);
#pragma unroll
              for (int t = 0; t < NT; t++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                  const float base = g == 0 ? qsum[g][t][e] * mb : fmaf(qsum[g][t][e], mb, sc[h][t][2 * k + e]);
                  sc[h][t][2 * k + e] = fmaf(ga[h][t][2 * k + e], ms, base);
                }
            }
        }
      }
    }
  }

  // The unit's value scales (over 2^(E - BITS)) and centred biases (bias + Z scale, over 2^E) as fp16, each
  // converted once into the warp's buffer: [granule][group][c][bias, scale of tokens 4c, 4c + 1; bias, scale of
  // 4c + 2, 4c + 3], an A operand as it stands: rows r are the biases' sums, rows r + 8 (the scales') are not used.
  // With PREC the remainders of the biases' rounding (bias + Z scale needs more than fp16's 11 bits wherever a
  // group is not nearly symmetric about zero) follow as [granule][group][c][tokens 4c, 4c + 1; 4c + 2, 4c + 3],
  // times 2^kLogB to keep them above fp16's subnormals, and take the scales' place in rows r + 8.
  // Moves a group's power of two first where one of them does not fit.
  static __device__ __forceinline__ void convert_meta(const unsigned char *sm, unsigned char *buf, State &s) {
    const int lane = threadIdx.x & 31;
    uint32_t su[MW], bu[MW];
    bool over = false;
#pragma unroll
    for (int k = 0; k < MW; k++) {
      const int i = lane + 32 * k, h = i / (8 * NG), gp = i % (8 * NG);
      su[k] = bu[k] = 0;
      if (kMW % 32 == 0 || i < kMW) {
        const unsigned char *p = sm + h * GB + 2 * L.code_bytes + 64 * NG + gp * 4;
        su[k] = *reinterpret_cast<const uint32_t *>(p);
        bu[k] = *reinterpret_cast<const uint32_t *>(p + 32 * NG);
      }
      over |= max_u16x2(su[k], s.lim_s[k]) != s.lim_s[k];
      over |= max_u16x2(bu[k] & 0x7fff7fffu, s.lim_b[k]) != s.lim_b[k];
    }
    if (__any_sync(kFull, over)) {
      // exponents that hold scale * 2^BITS and |bias| below 2^E
      int need[MW];
#pragma unroll
      for (int k = 0; k < MW; k++) {
        const uint32_t u = su[k] & 0x7fff7fffu, v = bu[k] & 0x7fff7fffu;
        const uint32_t s1 = max(u & 0xffffu, u >> 16), b1 = max(v & 0xffffu, v >> 16);
        need[k] = min(120, max((int)(s1 >> 7) - 126 + BITS, (int)(b1 >> 7) - 126));
      }
#pragma unroll
      for (int i = 0; i < NG; i++) {
        int e = -126;
#pragma unroll
        for (int k = 0; k < MW; k++)
          if (meta_group(k) == i) e = max(e, need[k]);
        e = __reduce_max_sync(kFull, e);
        if (e > s.E[i]) {
          e += 1;                                    // a little room, so that this stays rare
          const float f = p2(s.E[i] - e);
          set_exponent(s, i, e);
#pragma unroll
          for (int j = 0; j < VB; j++)
            if (j * DB / GS == i)
#pragma unroll
              for (int u2 = 0; u2 < MPB; u2++)
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                  for (int k = 0; k < 4; k++) s.acc[j * MPB + u2][t][k] *= f;
          if ((lane >> 2) == i)
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
              for (int k = 0; k < (PREC ? 4 : 2); k++) s.bacc[t][k] *= f;
        }
      }
    }
    __syncwarp();                                    // the buffer's readers of the unit in front are done
#pragma unroll
    for (int k = 0; k < MW; k++) {
      const int i = lane + 32 * k, hg = i / 8, pair = i % 8;
      const float z = (float)(1 << (BITS - 1)) * s.fb[k];
      const float s0 = bf_lo(su[k]), s1 = bf_hi(su[k]);
      if (kMW % 32 == 0 || i < kMW) {
        const float b0 = fmaf(s0, z, bf_lo(bu[k]) * s.fb[k]), b1 = fmaf(s1, z, bf_hi(bu[k]) * s.fb[k]);
        const uint32_t b = pack_h2(b0, b1);
        *reinterpret_cast<uint2 *>(buf + hg * 64 + pair * 8) = make_uint2(b, pack_h2(s0 * s.fs[k], s1 * s.fs[k]));
        if constexpr (PREC) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&b));
          *reinterpret_cast<uint32_t *>(buf + 8 * kMW + hg * 32 + pair * 4) =
              pack_h2((b0 - f.x) * (float)(1 << kLogB), (b1 - f.y) * (float)(1 << kLogB));
        }
      }
    }
    __syncwarp();
  }

  // Values of a granule: sum of P * (bias + Z scale) a group, and P * scale against the codes.
  // meta, rest: the granule's part of convert_meta's buffer, and of the remainders behind it.
  static __device__ __forceinline__ void values(const unsigned char *sm, const unsigned char *meta,
                                                const unsigned char *rest, const uint32_t (&ph)[NT][2], const uint32_t (&pl)[NT][2], State &s) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    {
      // one MMA: row g of A = group g's (rows of lanes r >= NG repeat them and are not used)
      uint4 m = *reinterpret_cast<const uint4 *>(meta + (r % NG) * 64 + c * 16);
      if constexpr (PREC) {
        const uint2 lo = *reinterpret_cast<const uint2 *>(rest + (r % NG) * 32 + c * 8);
        m.y = lo.x;
        m.w = lo.y;
      }
#pragma unroll
      for (int t = 0; t < NT; t++) {
        mma(s.bacc[t], m.x, m.y, m.z, m.w, ph[t][0], ph[t][1]);
        if constexpr (PREC) mma(s.bacc[t], m.x, m.y, m.z, m.w, pl[t][0], pl[t][1]);
      }
    }
    // !PREC: subnormal codes, and -Z, -16 Z (4-bit) times 2^-24 for the centring MMA
    constexpr uint32_t kC = BITS == 4 ? 0x80088008u : 0x80808080u, kC16 = 0x80808080u;
    // PREC: 1024 + code, and -(1024 + Z), -(1024 + 16 Z): the centred codes as normal numbers
    constexpr uint32_t kM = BITS == 4 ? 0xe408e408u : 0xe480e480u, kM16 = 0xe480e480u;
    const uint4 *vc = reinterpret_cast<const uint4 *>(sm + L.code_bytes) + lane;
    uint32_t b[NG][NT][2];
#pragma unroll
    for (int g = 0; g < NG; g++) {
      const uint4 m = *reinterpret_cast<const uint4 *>(meta + g * 64 + c * 16);
      const uint32_t s0 = m.y, s1 = m.w;
      uint32_t bl[NT][2];
#pragma unroll
      for (int t = 0; t < NT; t++) {
        b[g][t][0] = hmul2u(ph[t][0], s0);
        b[g][t][1] = hmul2u(ph[t][1], s1);
        if constexpr (PREC) {
          bl[t][0] = hfma2u(pl[t][0], s0, hfma2u(ph[t][0], s0, b[g][t][0] ^ 0x80008000u));
          bl[t][1] = hfma2u(pl[t][1], s1, hfma2u(ph[t][1], s1, b[g][t][1] ^ 0x80008000u));
        }
      }
#pragma unroll
      for (int j = g * GS / DB; j < (g + 1) * GS / DB; j++) {
        const uint4 q4 = vc[(j / 2) * 32];           // two blocks share a 16-byte load
        const uint32_t x = j % 2 ? q4.z : q4.x, w = j % 2 ? q4.w : q4.y;
        constexpr uint32_t m0 = BITS == 4 ? 0x000f000fu : 0x00ff00ffu, m1 = BITS == 4 ? 0x00f000f0u : 0x00ff00ffu;
        constexpr uint32_t or_ = PREC ? 0x64006400u : 0u;
        const uint32_t x8 = x >> 8, w8 = w >> 8;
        uint32_t f4[2][4] = {{(x & m0) | or_, ((BITS == 4 ? x : x8) & m1) | or_, (w & m0) | or_, ((BITS == 4 ? w : w8) & m1) | or_},
                             {(x8 & m0) | or_, (x8 & m1) | or_, (w8 & m0) | or_, (w8 & m1) | or_}};
        if constexpr (PREC)
#pragma unroll
          for (int k = 0; k < MPB; k++)
#pragma unroll
            for (int i = 0; i < 4; i++) f4[k][i] = hadd2u(f4[k][i], i % 2 ? kM16 : kM);
#pragma unroll
        for (int k = 0; k < MPB; k++)
#pragma unroll
          for (int t = 0; t < NT; t++) {
            float(&acc)[4] = s.acc[MPB * j + k][t];
            mma(acc, f4[k][0], f4[k][1], f4[k][2], f4[k][3], b[g][t][0], b[g][t][1]);
            if constexpr (PREC) mma(acc, f4[k][0], f4[k][1], f4[k][2], f4[k][3], bl[t][0], bl[t][1]);
          }
      }
    }
    if constexpr (!PREC)                             // minus Z * sum of P * scale
#pragma unroll
      for (int j = 0; j < VB * MPB; j++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          constexpr int per = VB * MPB / NG;
          mma(s.acc[j][t], kC, kC16, kC, kC16, b[j / per][t][0], b[j / per][t][1]);
        }
  }

  // One unit (two granules): scores, running max, P, values of its tokens lo ..
  // valid - 1, lo 0 or 16 and below valid.  Of the others, scores are masked and
  // value scales and biases must be zero (clear_tail).
  static __device__ __forceinline__ void unit(const unsigned char *sm, unsigned char *meta, int lo, int valid, const uint32_t (&qf)[KM][NT][2],
                                              const float (&qsum)[NG][NT][2], const float (&sf)[NT][2], State &s) {
    const int lane = threadIdx.x & 31, r = lane >> 2;
    const int t0 = 4 * (r / 2) + r % 2;             // tokens of rows r and r + 8: t0, t0 + 2
    float sc[UG][NT][4], y[UG][NT][4];
    scores(sm, qf, qsum, sc);
    // ---- running max: moved only when a P would pass 2^14
    auto exponents = [&]() {
#pragma unroll
      for (int h = 0; h < UG; h++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
          for (int j = 0; j < 4; j++) y[h][t][j] = fmaf(sc[h][t][j], sf[t][j & 1], -s.m10[t][j & 1]);
      if (lo > 0 || valid < kUnit)                  // the sequence's last unit, or a page is missing
#pragma unroll
        for (int h = 0; h < UG; h++)
#pragma unroll
          for (int t = 0; t < NT; t++)
#pragma unroll
            for (int j = 0; j < 4; j++)
              if (16 * h < lo || 16 * h + t0 + j / 2 * 2 >= valid) y[h][t][j] = -INFINITY;
    };
    exponents();
    float top = y[0][0][0];
#pragma unroll
    for (int h = 0; h < UG; h++)
#pragma unroll
      for (int t = 0; t < NT; t++) top = fmaxf(fmaxf(fmaxf(y[h][t][0], y[h][t][1]), fmaxf(y[h][t][2], y[h][t][3])), top);
    if (__any_sync(kFull, top > kLogPMax)) {
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < UG; h++)
#pragma unroll
            for (int k = 0; k < 2; k++)
              if (16 * h >= lo && 16 * h + t0 + 2 * k < valid) mx = fmaxf(mx, sc[h][t][e + 2 * k] * sf[t][e]);
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
          const float m = fmaxf(s.m10[t][e], mx - kLogP);
          const float f = ex2(s.m10[t][e] - m);     // 0 the first time
          s.m10[t][e] = m;
          s.l[t][e] *= f;
          s.bacc[t][e] *= f;
          if constexpr (PREC) s.bacc[t][e + 2] *= f;
#pragma unroll
          for (int i = 0; i < VB * MPB; i++) {
            s.acc[i][t][e] *= f;
            s.acc[i][t][e + 2] *= f;
          }
        }
      exponents();
    }
    // ---- P, rounded to fp16 and transposed to the B operand: k = token, n = head
    uint32_t ph[UG][NT][2], pl[UG][NT][2];
#pragma unroll
    for (int h = 0; h < UG; h++)
#pragma unroll
      for (int t = 0; t < NT; t++) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          p[j] = ex2(y[h][t][j]);
          s.l[t][j & 1] += p[j];
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const uint32_t u = pack_h2(p[2 * k], p[2 * k + 1]);
          if constexpr (PREC) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
            pl[h][t][k] = transpose8x8(pack_h2(p[2 * k] - f.x, p[2 * k + 1] - f.y));
          }
          ph[h][t][k] = transpose8x8(u);
        }
      }
    convert_meta(sm, meta, s);
#pragma unroll
    for (int h = 0; h < UG; h++)
      values(sm + h * GB, meta + h * 64 * NG, meta + 8 * kMW + h * 32 * NG, ph[h], pl[h], s);
  }

  // Writes this warp's sums (value units, over 2^kLogP) and max / total to the join buffer.
  static __device__ __forceinline__ void to_join(State &s, float *row_o, float *row_ml) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float l = s.l[t][e];
        l += __shfl_xor_sync(kFull, l, 4);
        l += __shfl_xor_sync(kFull, l, 8);
        l += __shfl_xor_sync(kFull, l, 16);
        const int h = 8 * t + 2 * c + e;
        if (s.m10[t][e] == INFINITY) l = NAN;       // a score beyond fp32: every p is 0 beside it
        if (r == 0) {
          row_ml[2 * h] = s.m10[t][e];
          row_ml[2 * h + 1] = l;
        }
#pragma unroll
        for (int g = 0; g < NG; g++) {
          float b = s.bacc[t][e];
          if constexpr (PREC) b = fmaf(s.bacc[t][e + 2], 1.0f / (1 << kLogB), b);
          const float bias = __shfl_sync(kFull, b, g * 4 + c);
          const float fe = p2(s.E[g]);
#pragma unroll
          for (int j = g * GS / DB; j < (g + 1) * GS / DB; j++) {
            constexpr float f1 = PREC ? 1.0f / (1 << BITS) : (float)(1 << (24 - BITS));
            if constexpr (BITS == 4) {
              float4 v;
              v.x = fmaf(s.acc[2 * j][t][e], f1, bias) * fe;
              v.y = fmaf(s.acc[2 * j][t][e + 2], f1 / 16, bias) * fe;
              v.z = fmaf(s.acc[2 * j + 1][t][e], f1, bias) * fe;
              v.w = fmaf(s.acc[2 * j + 1][t][e + 2], f1 / 16, bias) * fe;
              *reinterpret_cast<float4 *>(row_o + h * SROW + 32 * j + 4 * r) = v;
            } else {
              float2 v;
              v.x = fmaf(s.acc[j][t][e], f1, bias) * fe;
              v.y = fmaf(s.acc[j][t][e + 2], f1, bias) * fe;
              *reinterpret_cast<float2 *>(row_o + h * SROW + 16 * j + 2 * r) = v;
            }
          }
        }
      }
    }
  }
};

// Rounds and stores two output elements (i even).
__device__ __forceinline__ void store_out2(const Args &a, int64_t i, float v0, float v1) {
  uint32_t u;
  if (a.f16) {
    u = pack_h2(v0, v1);
  } else {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v0, v1);
    u = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint32_t *>(a.out + i) = u;
}
// log-sum-exp (natural) from the scaled max and total.
__device__ __forceinline__ float lse_of(float m10, float l) {
  return l > 0.0f ? (m10 + log2f(l)) * 0.6931471805599453f : (l == 0.0f ? -INFINITY : l);
}

template <int BITS, int D, int GS, int NT, bool PREC>
__global__ void __launch_bounds__(kThreads, min_ctas(D, NT)) k_attn_decode(const Args a) {
  using K = Kernel<BITS, D, GS, NT, PREC>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ uint64_t bars[kWarps * 8];
  __shared__ Start start;
  __shared__ long long scan[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  float *join = reinterpret_cast<float *>(smem_raw);                         // [warp][GHP][SROW], then [warp][GHP][2]
  float *join_ml = join + kWarps * K::GHP * K::SROW;
  unsigned char *meta = smem_raw + K::kJoin + warp * K::kMeta;
  unsigned char *qcta = smem_raw + K::kJoin + kWarps * K::kMeta;             // queries of a piece
  unsigned char *ring = qcta + K::kQ + warp * a.depth * K::kSlot;
  uint64_t *bar = bars + warp * 8;

  if (lane == 0)
    for (int i = 0; i < a.depth; i++) mbar_init(bar + i, 1);
  fence_mbar_init();
  pdl_launch_dependents();
  pdl_wait();
  // warps that share a pair, this one's number among them, and their barrier
  const bool alone = a.mode == kAttnWarpPair;
  const int ways = alone ? 1 : kWarps, way = alone ? 0 : warp;
  auto pair_sync = [&]() {
    if (alone) __syncwarp();
    else __syncthreads();
  };
  Start st{};
  if (a.mode == kAttnCut) {
    find_start(a, &start, scan);
    st = start;
  } else {
    const int HC = a.H * a.chunks, pair = alone ? blockIdx.x * kWarps + warp : blockIdx.x;
    st.b = pair / HC;
    st.hc = pair % HC;
    if (st.b < a.B) st.left = places(units(a, tokens(a, st.b, st.hc == 0)));
    pair_sync();
  }                              // (the barriers also publish the mbarriers)

  // rows without a token: zeros, and minus infinity for the log-sum-exp (a warp a row, behind the CTA's share)
  auto empty_rows = [&]() {
    for (int b = blockIdx.x * kWarps + warp; b < a.B; b += gridDim.x * kWarps)
      if (tokens(a, b, false) == 0) {
        const int64_t row = (int64_t)b * a.H * a.G;
        for (int i = lane; i < a.H * a.G * (D / 8); i += 32) reinterpret_cast<uint4 *>(a.out + row * D)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (int i = lane; i < a.H * a.G; i += 32) a.lse[row + i] = -INFINITY;
      }
  };
  constexpr int kPart = Ws<D, K::GHP>::kPart;
  Rec *recs = reinterpret_cast<Rec *>(a.ws + (int64_t)2 * gridDim.x * kPart);
  // pieces walked by the whole CTA (pc), and this warp's copies (cp), ahead of it
  Cursor cp{}, pc{};
  cp.b = pc.b = st.b;
  cp.hc = pc.hc = st.hc;
  cp.left = pc.left = st.left;
  if (!cursor_open<K::GB, false>(a, pc, st.u, 0)) {
    if (tid == 0 && a.mode == kAttnCut) recs[blockIdx.x] = Rec{0, 0, 0, 0};
    empty_rows();
    return;
  }
  cursor_open<K::GB>(a, cp, st.u, way);
  cursor_settle<K::GB>(a, cp, way);
  if (tid == 0 && a.mode == kAttnCut) {
    // this share begins behind the pair's first unit, and the share in front with that unit or before it
    const bool cut = pc.g > 0 && st.u - st.per <= kPieceCost;
    recs[blockIdx.x] = Rec{pc.b, pc.hc, cut ? 1 + (int)((pc.n + kPieceCost - st.u + st.per - 1) / st.per) : 0, 0};
  }

  // The ring: units go in and out in order, slot after slot.  A slot's barrier completes a phase for every
  // unit, also for one without a copy, so that one parity serves all slots of a round.
  int slot_in = 0, slot_out = 0, flying = 0;
  uint32_t parity = 0;
  uint32_t lack0 = 0, lack1 = 0;      // slots without their first / second granule
  bool dead = false;
  const uint32_t page_gran = (uint32_t)a.H << a.gshift;     // granules of a page
  auto issue = [&]() {                // the cursor's unit into slot_in
    if (cp.g >= cp.end) return;
    const bool two = cursor_two(a, cp);
    unsigned char *dst = ring + slot_in * K::kSlot;
    uint64_t *full = bar + slot_in;
    // granule of the cache
    auto gran = [&](int page) {
      return a.cache + ((int64_t)page * page_gran + (cp.head + ((cp.g << a.ushift) & ((1 << a.gshift) - 1)))) * K::GB;
    };
    if (max((uint32_t)cp.page0, (uint32_t)cp.page1) < (uint32_t)a.pages) {
      if (lane == 0) {
        const uint32_t bytes = two ? 2 * K::GB : K::GB;
        mbar_arrive_expect_tx(full, bytes);
        if (a.gshift != 0 || !two) {             // all in one page
          bulk_load(dst, gran(cp.page0), bytes, full);
        } else {
          bulk_load(dst, gran(cp.page0), K::GB, full);
          bulk_load(dst + K::GB, gran(cp.page1), K::GB, full);
        }
      }
    } else {                                     // a granule whose page is outside the cache is left out and reported
      const bool ok0 = (uint32_t)cp.page0 < (uint32_t)a.pages, ok1 = two && (uint32_t)cp.page1 < (uint32_t)a.pages;
      if (lane == 0) {
        atomicOr(&g_device_error, kErrIndex);
        mbar_arrive_expect_tx(full, ok0 || ok1 ? K::GB : 0);
        if (ok0) bulk_load(dst, gran(cp.page0), K::GB, full);      // (gshift 0: else both are bad)
        if (ok1) bulk_load(dst + K::GB, gran(cp.page1), K::GB, full);
      }
      if (!ok0) lack0 |= 1u << slot_in;
      if (!ok1) lack1 |= 1u << slot_in;
    }
    flying++;
    if (++slot_in == a.depth) slot_in = 0;
    cp.g += ways;
    cursor_page(a, cp);
    if (cp.g >= cp.end) cursor_settle<K::GB>(a, cp, way);
  };
  // (a warp alone keeps its queries in its part of the join buffer, which it writes after it has read them)
  unsigned char *qbuf = alone ? reinterpret_cast<unsigned char *>(join + warp * K::GHP * K::SROW) : qcta;
  // queries of a piece into their buffer: heads [h0, h0 + heads) of the kv head's chunk
  auto fetch_q = [&](const Cursor &c) {
    const int chunk = c.hc % a.chunks;
    const int n = min(a.GH, a.G - chunk * a.GH) * (D / 8);
    const uint16_t *src = a.q + (int64_t)c.b * a.q_stride + (int64_t)((c.hc / a.chunks) * a.G + chunk * a.GH) * D;
    for (int i = alone ? lane : tid; i < n; i += 32 * ways) cp_async_16(qbuf + i * 16, src + i * 8, 16);
    cp_async_commit();
  };
  fetch_q(pc);
  issue();
  int rest = a.depth - 1;             // first copies held back until the queries are staged: theirs come sooner

  typename K::State s;
  int g_first = pc.g;
  bool first_piece = true;
  while (true) {
    cp_async_wait<0>();
    pair_sync();                      // this piece's queries are there, and the join buffer is free
    // ---- this piece's queries: chunk of heads [h0, h0 + heads) of kv head pc.hc / chunks
    const int chunk = pc.hc % a.chunks;
    const int h0 = (pc.hc / a.chunks) * a.G + chunk * a.GH;
    const int heads = min(a.GH, a.G - chunk * a.GH);
    uint32_t qf[K::KM][NT][2];
    float qsum[K::NG][NT][2], sf[NT][2];
#pragma unroll
    for (int t = 0; t < NT; t++) {
      // lane r holds head 8t + r; its elements in the order of the score MMAs
      const bool in = 8 * t + r < heads;
      const unsigned char *row = qbuf + (in ? 8 * t + r : 0) * (2 * D);
      float v[D / 4], mx = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; i++) {
        // 4-bit: word 4i + c covers elements 32i + 8c ..+7; 8-bit: words 8i + c and 8i + 4 + c, four each
        uint32_t p[4];
        if constexpr (BITS == 4) {
          *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(row + 64 * i + 16 * c);
        } else {
          *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(row + 64 * i + 8 * c);
          *reinterpret_cast<uint2 *>(p + 2) = *reinterpret_cast<const uint2 *>(row + 64 * i + 32 + 8 * c);
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const uint16_t hb = (uint16_t)(p[e / 2] >> (e % 2 * 16));
          v[8 * i + e] = in ? q_at(&hb, a.f16) : 0.0f;
          mx = fmaxf(mx, fabsf(v[8 * i + e]));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      // q * 2^up has its largest element in [2^12, 2^13)
      const int up = min(120, max(-120, 139 - (int)(__float_as_uint(mx) >> 23)));
      const float fu = pow2f(up);
      float part[K::NG];
#pragma unroll
      for (int g = 0; g < K::NG; g++) part[g] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; i++) {
        float *x = v + 8 * i;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          x[e] *= fu;
          const int g = (BITS == 4 ? 32 * i : 32 * i + 16 * (e / 4)) / GS;
          part[g] += x[e];
        }
        if constexpr (BITS == 4) {
          qf[2 * i][t][0] = pack_h2(x[0], x[4]);
          qf[2 * i][t][1] = pack_h2(x[1] * 0.0625f, x[5] * 0.0625f);
          qf[2 * i + 1][t][0] = pack_h2(x[2], x[6]);
          qf[2 * i + 1][t][1] = pack_h2(x[3] * 0.0625f, x[7] * 0.0625f);
        } else {
          qf[2 * i][t][0] = pack_h2(x[0], x[2]);
          qf[2 * i][t][1] = pack_h2(x[1], x[3]);
          qf[2 * i + 1][t][0] = pack_h2(x[4], x[6]);
          qf[2 * i + 1][t][1] = pack_h2(x[5], x[7]);
        }
      }
      // per-head constants for the score fragment's columns 2c, 2c + 1
      // (2^(24 - up), of which 2^12 came with the scale: 24 - up passes 127 for a query beyond 2^115, and only
      // the product may overflow)
      const float back = a.scale_log2 * pow2f(12 - up);
#pragma unroll
      for (int g = 0; g < K::NG; g++) {
        part[g] += __shfl_xor_sync(kFull, part[g], 1);
        part[g] += __shfl_xor_sync(kFull, part[g], 2);
        part[g] *= 0x1p-24f;
      }
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int src = (2 * c + e) * 4;
        sf[t][e] = __shfl_sync(kFull, back, src);
#pragma unroll
        for (int g = 0; g < K::NG; g++) qsum[g][t][e] = __shfl_sync(kFull, part[g], src);
      }
    }
    K::reset(s);
    Cursor nc = pc;
    const bool more = cursor_next_piece<K::GB, false>(a, nc, 0);
    pair_sync();                      // every warp holds its queries
    if (more) fetch_q(nc);            // (in flight through the piece's loop)
    for (; rest > 0; rest--) issue();

    // ---- this warp's units of the piece
    for (int g = g_first + way; g < pc.end && !dead; g += ways) {
      if (!mbar_wait(bar + slot_out, parity)) {
        dead = true;
        break;
      }
      flying--;
      unsigned char *sm = ring + slot_out * K::kSlot;
      int lo = 0, valid = pc.len - g * K::kUnit;
      if (valid < K::kUnit || (lack0 | lack1)) {        // a last unit, or one of few with a page outside the cache
        const uint32_t bit = 1u << slot_out;
        if (lack0 & bit) lo = kv::kTok;
        if (K::UG == 1 || (lack1 & bit)) valid = min(valid, kv::kTok);
        lack0 &= ~bit;
        lack1 &= ~bit;
        if (lo < valid) {
          if (lo > 0 || valid < kv::kTok) K::clear_tail(sm, lo > 0 ? 0 : valid);
          if (K::UG == 2 && valid < K::kUnit) K::clear_tail(sm + K::GB, valid - kv::kTok);
        }
      }
      if (lo < valid) K::unit(sm, meta, lo, valid, qf, qsum, sf, s);
      __syncwarp();
      if (++slot_out == a.depth) {
        slot_out = 0;
        parity ^= 1u;
      }
      issue();
    }

    // ---- join the warps: row h of every warp's sums, scaled to the common max
    K::to_join(s, join + warp * K::GHP * K::SROW, join_ml + warp * K::GHP * 2);
    if (alone) {
      __syncwarp();
      for (int i = lane; i < heads * (D / 4); i += 32) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        const float l = join_ml[(warp * K::GHP + h) * 2 + 1], inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float4 o = *reinterpret_cast<const float4 *>(join + (warp * K::GHP + h) * K::SROW + d);
        const int64_t row = (int64_t)pc.b * a.H * a.G + h0 + h;
        store_out2(a, row * D + d, o.x * inv, o.y * inv);
        store_out2(a, row * D + d + 2, o.z * inv, o.w * inv);
        if (a.lse && d == 0) a.lse[row] = lse_of(join_ml[(warp * K::GHP + h) * 2], l);
      }
      break;
    }
    __syncthreads();
    const bool whole = g_first == 0 && pc.end == pc.n;
    const int64_t part_id = (int64_t)blockIdx.x * 2 + (first_piece && g_first > 0 ? 0 : 1);
    float *part = a.ws + part_id * kPart;
    for (int i = tid; i < heads * (D / 4); i += kThreads) {
      const int h = i / (D / 4), d = i % (D / 4) * 4;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; w++)
        if (join_ml[(w * K::GHP + h) * 2 + 1] != 0.0f) m = fmaxf(m, join_ml[(w * K::GHP + h) * 2]);
      float l = 0.0f;
      float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const float lw = join_ml[(w * K::GHP + h) * 2 + 1];
        if (lw == 0.0f) continue;                      // a warp without a granule
        const float f = ex2(join_ml[(w * K::GHP + h) * 2] - m);
        const float4 v = *reinterpret_cast<const float4 *>(join + (w * K::GHP + h) * K::SROW + d);
        l = fmaf(lw, f, l);
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
      }
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t row = (int64_t)pc.b * a.H * a.G + h0 + h;
        store_out2(a, row * D + d, o.x * inv, o.y * inv);
        store_out2(a, row * D + d + 2, o.z * inv, o.w * inv);
        if (a.lse && d == 0) a.lse[row] = lse_of(m, l);
      } else {
        *reinterpret_cast<float4 *>(part + h * D + d) = o;
        if (d == 0) {
          part[K::GHP * D + 2 * h] = m;
          part[K::GHP * D + 2 * h + 1] = l;
        }
      }
    }
    if (!more) break;
    pc = nc;
    first_piece = false;
    g_first = 0;
  }
  empty_rows();
  // copies still in flight (only after a wait gave up) land before the CTA's memory is freed
  for (; flying > 0; flying--) {
    mbar_wait(bar + slot_out, parity);
    if (++slot_out == a.depth) {
      slot_out = 0;
      parity ^= 1u;
    }
  }
}

// Joins the pieces of the pairs that shares cut.  Block (i, h) reads the record of
// share i + 1 and, where there is a pair to join, adds head h of the piece that
// ends share i and of those that begin shares i + 1, i + 2, ...: the warps take
// pieces in turn, a lane D / 32 elements, maxima, totals and sums loaded at once.
constexpr int kJoinBatch = 8;

template <int D, int GHP>
__global__ void __launch_bounds__(kThreads) k_attn_join(const Args a, int ctas) {
  constexpr int kPart = Ws<D, GHP>::kPart, E = D / 32;
  __shared__ float so[kWarps][D], sml[kWarps][2];
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x + 1, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (read through L2: nothing of the workspace may come from an earlier launch's lines in L1)
  const int4 rec = __ldcg(reinterpret_cast<const int4 *>(a.ws + (int64_t)2 * ctas * kPart) + i);
  const int b = rec.x, chunk = rec.y % a.chunks, pieces = rec.z;
  const int h0 = (rec.y / a.chunks) * a.G + chunk * a.GH;
  if (pieces == 0 || h >= a.G - chunk * a.GH) return;
  // piece j = 0: end of share i - 1; j > 0: beginning of share i + j - 1
  auto part = [&](int j) { return a.ws + (int64_t)(j == 0 ? 2 * (i - 1) + 1 : 2 * (i + j - 1)) * kPart; };
  float m = -INFINITY, l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; e++) o[e] = 0.0f;
  for (int j0 = warp; j0 < pieces; j0 += kWarps * kJoinBatch) {
    float2 ml[kJoinBatch], v[kJoinBatch][E / 2];
#pragma unroll
    for (int k = 0; k < kJoinBatch; k++) {
      const int j = j0 + k * kWarps;
      ml[k] = make_float2(-INFINITY, 0.0f);
      if (j < pieces) {
        const float *p = part(j);
        ml[k] = __ldcg(reinterpret_cast<const float2 *>(p + GHP * D + 2 * h));
#pragma unroll
        for (int e = 0; e < E / 2; e++) v[k][e] = __ldcg(reinterpret_cast<const float2 *>(p + h * D + lane * E) + e);
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kJoinBatch; k++)
      if (ml[k].y != 0.0f) mn = fmaxf(mn, ml[k].x);                  // (a piece without a token adds nothing)
    const float fo = m == -INFINITY ? 0.0f : ex2(m - mn);
    m = mn;
    l *= fo;
#pragma unroll
    for (int e = 0; e < E; e++) o[e] *= fo;
#pragma unroll
    for (int k = 0; k < kJoinBatch; k++)
      if (ml[k].y != 0.0f) {
        const float f = ex2(ml[k].x - m);
        l = fmaf(ml[k].y, f, l);
#pragma unroll
        for (int e = 0; e < E / 2; e++) {
          o[2 * e] = fmaf(v[k][e].x, f, o[2 * e]);
          o[2 * e + 1] = fmaf(v[k][e].y, f, o[2 * e + 1]);
        }
      }
  }
#pragma unroll
  for (int e = 0; e < E; e++) so[warp][lane * E + e] = o[e];
  if (lane == 0) {
    sml[warp][0] = m;
    sml[warp][1] = l;
  }
  __syncthreads();
  if (threadIdx.x * 2 >= D) return;
  const int d = threadIdx.x * 2;
  float mt = -INFINITY, lt = 0.0f, x0 = 0.0f, x1 = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; w++)
    if (sml[w][1] != 0.0f) mt = fmaxf(mt, sml[w][0]);
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (sml[w][1] == 0.0f) continue;
    const float f = ex2(sml[w][0] - mt);
    lt = fmaf(sml[w][1], f, lt);
    x0 = fmaf(so[w][d], f, x0);
    x1 = fmaf(so[w][d + 1], f, x1);
  }
  const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
  const int64_t row = (int64_t)b * a.H * a.G + h0 + h;
  store_out2(a, row * D + d, x0 * inv, x1 * inv);
  if (a.lse && d == 0) a.lse[row] = lse_of(mt, lt);
}

}  // namespace attn
}  // namespace
}  // namespace gwb

namespace gwb {
namespace {

attn::Args attn_args(const AttnCall &c) {
  attn::Args a{};
  a.q = c.q; a.q_stride = c.q_stride;
  a.cache = static_cast<const unsigned char *>(c.cache.data);
  a.table = c.table; a.table_stride = c.table_stride;
  a.lens = c.lens;
  a.out = c.out; a.lse = c.lse;
  a.ws = static_cast<float *>(c.ws);
  a.pages = c.cache.pages;
  a.B = (int)c.B; a.H = (int)c.cache.heads; a.G = (int)(c.q_heads / c.cache.heads);
  a.chunks = (a.G + 8 * c.tiles - 1) / (8 * c.tiles);
  a.GH = (a.G + a.chunks - 1) / a.chunks;
  int gpp = (int)(c.cache.page_size / kv::kTok);
  while (gpp >>= 1) a.gshift++;
  const int64_t cap = c.max_pages * c.cache.page_size;
  a.cap = (int)(cap < 0x7fffff00 ? cap : 0x7fffff00);          // (a whole number of units)
  a.min_per = attn::kWarps;
  a.f16 = c.f16;
  a.scale_log2 = c.scale * 1.4426950408889634f * 4096.0f;
  return a;
}

// Launches of one instance: the attention, then the join that depends on it.
template <int BITS, int D, int GS, int NT, bool PREC>
gwb_status run_attn(attn::Args a, int64_t ws_bytes, cudaStream_t st) {
  using K = attn::Kernel<BITS, D, GS, NT, PREC>;
  auto kern = attn::k_attn_decode<BITS, D, GS, NT, PREC>;
  constexpr size_t join = K::kJoin + attn::kWarps * K::kMeta + K::kQ;   // (all multiples of 16)
  // ring depth: what lets the CTAs that the registers allow share an SM (228 KB; a CTA takes 1 KB and the
  // kernel's static part besides), at least 2 slots, at most 6
  constexpr size_t slot = (size_t)attn::kWarps * K::kSlot, most = 228 * 1024 / attn::min_ctas(D, NT) - 1536;
  int depth = join < most ? (int)((most - join) / slot) : 0;
  depth = depth < 2 ? 2 : (depth > 6 ? 6 : depth);
  const size_t smem = join + depth * slot;
  AttnSetup su;
  gwb_status s = attn_setup(reinterpret_cast<const void *>(kern), smem, attn::kThreads, &su);
  if (s != GWB_OK) return s;
  const int ctas = su.sms * (su.per_sm < kAttnMaxPerSm ? su.per_sm : kAttnMaxPerSm);
  a.depth = depth;
  a.ushift = K::UG - 1;
  const int64_t pairs = (int64_t)a.B * a.H * a.chunks;
  a.mode = attn_mode(pairs, a.cap, ctas);
  const int64_t need = a.mode != kAttnCut
                           ? 0
                           : (int64_t)ctas * (2 * 4 * attn::Ws<D, K::GHP>::kPart + (int64_t)sizeof(attn::Rec));
  if (ws_bytes < need)
    return fail(GWB_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)ws_bytes, (long long)need);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.mode == kAttnCut ? ctas : a.mode == kAttnCtaPair ? pairs : (pairs + attn::kWarps - 1) / attn::kWarps));
  cfg.blockDim = dim3(attn::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return fail(GWB_ERR_CUDA, "attn_decode launch: %s", cudaGetErrorString(e));
  if (a.mode != kAttnCut) return GWB_OK;
  cfg.gridDim = dim3((unsigned)(ctas - 1), (unsigned)a.GH);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, attn::k_attn_join<D, K::GHP>, a, ctas);
  if (e != cudaSuccess) return fail(GWB_ERR_CUDA, "attn_decode join launch: %s", cudaGetErrorString(e));
  return GWB_OK;
}

}  // namespace
}  // namespace gwb
