// The block layout of the paged, quantized key-value cache, shared by the
// kernels that write it, read it and attend over it.
//
// A cache is [pages][kv heads][block].  A block holds page_size tokens of one
// head as page_size / 16 granules of 16 tokens, so any page size that is a
// multiple of 16 looks the same to a kernel that walks granules, and a granule
// is one contiguous copy.  Codes follow the MLX packing along the head
// dimension (lowest bits = lowest column), with the packed units moved to where
// the attention kernel's m16n8k16 fragments take them, so that it reads
// fragments with 8- and 16-byte shared-memory loads free of bank conflicts:
//
//   key codes     a token's row is NW = D*bits/32 words; word w = 4*(VW*a + v) + c of
//                 the token with MMA row rho is at [a][rho][c][v] (VW = min(4, NW/4))
//   value codes   a row is 2*NW 16-bit halves; half h = 16*a + 8*j + r of token
//                 t = 4*c + 2*y + z is at [a][r][c][j][y][z]: two tokens share a
//                 32-bit word, which is what the P.V product's A operand wants
//   key meta      [rho][group] words, scale (bf16) low, bias (bf16) high
//   value meta    scales bf16 [group][16 tokens], then biases bf16 [group][16 tokens]
//
// rho(t) = 2*(t/4) + t%2 + 8*(t/2%2): rows 2c, 2c+1, 2c+8, 2c+9 of the score
// fragment are then tokens 4c .. 4c+3, the k indices lane c holds in P.V.
#pragma once
#include <cstdint>

namespace gwb {
namespace kv {

constexpr int kTok = 16;   // tokens of a granule

struct Layout {
  int bits, D, gs, NG, NW, VW, code_bytes, granule;
};
__host__ __device__ constexpr Layout layout(int bits, int D, int gs) {
  const int NG = D / gs, NW = D * bits / 32, code = kTok * NW * 4;
  return Layout{bits, D, gs, NG, NW, NW / 4 < 4 ? NW / 4 : 4, code, 2 * code + 128 * NG};
}

__host__ __device__ constexpr int rho(int t) { return 2 * (t / 4) + t % 2 + 8 * (t / 2 % 2); }

// Byte offsets inside a granule.
__host__ __device__ constexpr int key_word(const Layout &l, int t, int w) {
  return 4 * ((((w / (4 * l.VW)) * 16 + rho(t)) * 4 + w % 4) * l.VW + w / 4 % l.VW);
}
__host__ __device__ constexpr int val_half(const Layout &l, int t, int h) {
  return l.code_bytes + 2 * (((((h / 16) * 8 + h % 8) * 4 + t / 4) * 2 + h / 8 % 2) * 4 + t % 4);
}
__host__ __device__ constexpr int key_meta(const Layout &l, int t, int g) {
  return 2 * l.code_bytes + 4 * (rho(t) * l.NG + g);
}
__host__ __device__ constexpr int val_scale(const Layout &l, int t, int g) {
  return 2 * l.code_bytes + 64 * l.NG + 2 * (g * 16 + t);
}
__host__ __device__ constexpr int val_bias(const Layout &l, int t, int g) {
  return 2 * l.code_bytes + 96 * l.NG + 2 * (g * 16 + t);
}

}  // namespace kv
}  // namespace gwb
