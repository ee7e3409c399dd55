"""Oracle of the operators around the linear layers (test infrastructure only): RMS norm with an int8
output, the quantized paged cache and the decode attention over it.

Plain numpy in fp64; fp32 only where a definition rounds to it (each step of the two quantizers and of
the norm's products).  Shares no code with the library.  Arrays of bf16 / fp16 values travel as fp64 or
fp32 numbers that the type represents; `rnd` rounds to either type.
"""
from __future__ import annotations

import numpy as np


def rnd(x, f16):
    """x rounded to nearest even to bf16 or fp16, as fp64."""
    if f16:
        return np.asarray(x, dtype=np.float64).astype(np.float16).astype(np.float64)
    return bf16(x)


def bf16(x):
    """fp64 (or fp32) -> bf16 (nearest even), as fp64; exact double rounding is avoided by working on fp64 bits."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)                               # x = m * 2^e, 0.5 <= |m| < 1
    e = np.maximum(e, -125)                          # below 2^-126 the spacing stays that of the subnormals
    step = np.ldexp(1.0, e - 8)
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(x), np.rint(x / step) * step, x)


def bf16_bits(x):
    """The 16-bit patterns of values that bf16 represents."""
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bits_bf16(u):
    return (np.asarray(u, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# ------------------------------------------------------------------ norm
def rmsnorm_quant_i8(x, residual, weight, eps, f16):
    """(qx int8, sx fp32, h): every step of the definition, fp32 where it says fp32."""
    x = np.asarray(x, dtype=np.float64)
    h = x if residual is None else rnd((x + residual).astype(np.float32), f16)
    r = np.array([1.0 / np.sqrt(np.sum(np.square(row)) / row.size + eps) if row.any() else 0.0 for row in h],
                 dtype=np.float32)
    f32 = np.float32
    with np.errstate(all="ignore"):
        y = (h.astype(f32) * r[:, None]).astype(f32) * np.asarray(weight).astype(f32)
        sx = (np.abs(y).max(1) / f32(127)).astype(f32)
        q = np.rint((y / np.where(sx == 0, f32(1), sx)[:, None]).astype(f32))
    q = np.where(sx[:, None] == 0, 0, np.clip(q, -127, 127))
    return q.astype(np.int8), sx, h


# ------------------------------------------------------------------ quantized rows and the block layout
def quantize_rows(x, bits, gs):
    """x [..., D] -> (codes uint8 [..., D], scales, biases as bf16 values [..., D/gs]); fp32 steps."""
    f32 = np.float32
    g = np.asarray(x, dtype=f32).reshape(*x.shape[:-1], -1, gs)
    # min and max under the total order -0 < +0
    key = g.view(np.int32)
    key = np.where(key >= 0, key, key ^ 0x7fffffff)
    pick = lambda k: np.where(k >= 0, k, k ^ 0x7fffffff).astype(np.int32).view(f32)  # noqa: E731
    mn, mx = pick(key.min(-1)), pick(key.max(-1))
    top = f32((1 << bits) - 1)
    s = ((mx - mn).astype(f32) / top).astype(f32)
    with np.errstate(all="ignore"):
        t = ((g - mn[..., None]).astype(f32) / np.where(s == 0, f32(1), s)[..., None]).astype(f32)
    code = np.where(s[..., None] == 0, 0, np.clip(np.rint(t), 0, top)).astype(np.uint8)
    return code.reshape(x.shape), bf16(s), np.where(mn == 0, np.copysign(0.0, mn), bf16(mn))


class Layout:
    """Where each part of a granule of 16 tokens lies, one element at a time."""

    def __init__(self, bits, D, gs):
        self.bits, self.D, self.gs, self.NG = bits, D, gs, D // gs
        self.NW = D * bits // 32
        self.VW = min(4, self.NW // 4)
        self.code = 64 * self.NW
        self.bytes = 2 * self.code + 128 * self.NG

    @staticmethod
    def rho(t):
        return 2 * (t // 4) + t % 2 + 8 * (t // 2 % 2)

    def key_bits(self, t, d):
        """Bit offset of key code d of token t."""
        w, low = divmod(d * self.bits, 32)
        c, a, v = w % 4, w // (4 * self.VW), w // 4 % self.VW
        return 32 * (((a * 16 + self.rho(t)) * 4 + c) * self.VW + v) + low

    def val_bits(self, t, d):
        h, low = divmod(d * self.bits, 16)
        a, j, r = h // 16, h // 8 % 2, h % 8
        c, y, z = t // 4, t // 2 % 2, t % 2
        return 8 * self.code + 16 * (((((a * 8 + r) * 4 + c) * 2 + j) * 2 + y) * 2 + z) + low

    def key_meta(self, t, g):
        """Byte offset of a key's bf16 scale; its bias follows."""
        return 2 * self.code + 4 * (self.rho(t) * self.NG + g)

    def val_scale(self, t, g):
        return 2 * self.code + 64 * self.NG + 2 * (16 * g + t)

    def val_bias(self, t, g):
        return self.val_scale(t, g) + 32 * self.NG

    def tables(self):
        """Byte and shift of every code, byte of every scale and bias: dicts of [16][D] / [16][NG] arrays."""
        T, Ds, Gs = range(16), range(self.D), range(self.NG)
        kb = np.array([[self.key_bits(t, d) for d in Ds] for t in T])
        vb = np.array([[self.val_bits(t, d) for d in Ds] for t in T])
        ks = np.array([[self.key_meta(t, g) for g in Gs] for t in T])
        return {"k": (kb // 8, kb % 8, ks, ks + 2),
                "v": (vb // 8, vb % 8, np.array([[self.val_scale(t, g) for g in Gs] for t in T]),
                      np.array([[self.val_bias(t, g) for g in Gs] for t in T]))}


def write_rows(cache, slots, rows, what, bits, gs, page):
    """Writes rows [T, H, D] (values) of keys ("k") or values ("v") into cache uint8 [pages, H, block], in place."""
    T, H, D = rows.shape
    lay = Layout(bits, D, gs)
    byte, shift, so, bo = lay.tables()[what]
    code, s, b = quantize_rows(rows, bits, gs)
    sb, bb = bf16_bits(s), bf16_bits(b)
    for i, slot in enumerate(slots):
        if slot < 0 or slot >= cache.shape[0] * page:
            continue
        p, t = divmod(int(slot), page)
        base, t = t // 16 * lay.bytes, t % 16
        for h in range(H):
            blk = cache[p, h, base:base + lay.bytes]
            mask = ((1 << bits) - 1) << shift[t]
            np.bitwise_and.at(blk, byte[t], (~mask & 0xff).astype(np.uint8))
            np.bitwise_or.at(blk, byte[t], (code[i, h].astype(np.int64) << shift[t]).astype(np.uint8))
            blk[so[t]], blk[so[t] + 1] = sb[i, h] & 0xff, sb[i, h] >> 8
            blk[bo[t]], blk[bo[t] + 1] = bb[i, h] & 0xff, bb[i, h] >> 8


def parts_of(cache, slots, what, bits, D, gs, page):
    """(codes [T, H, D], scales, biases [T, H, NG]) at slots, fp64; zeros outside the cache."""
    lay = Layout(bits, D, gs)
    byte, shift, so, bo = lay.tables()[what]
    slots = np.asarray(slots, dtype=np.int64)
    ok = (slots >= 0) & (slots < cache.shape[0] * page)
    at = np.where(ok, slots, 0)
    H = cache.shape[1]
    code = np.zeros((len(at), H, D))
    s, b = np.zeros((len(at), H, D // gs)), np.zeros((len(at), H, D // gs))
    for t in range(16):
        i = np.nonzero(ok & (at % 16 == t))[0]
        if not len(i):
            continue
        gran = cache[at[i] // page][:, :, :].reshape(len(i), H, page // 16, lay.bytes)
        gran = gran[np.arange(len(i)), :, at[i] % page // 16]              # [n, H, bytes]
        code[i] = (gran[:, :, byte[t]].astype(np.int64) >> shift[t]) & ((1 << bits) - 1)
        u16 = lambda o: gran[:, :, o].astype(np.uint16) | (gran[:, :, o + 1].astype(np.uint16) << 8)  # noqa: E731
        s[i], b[i] = bits_bf16(u16(so[t])), bits_bf16(u16(bo[t]))
    return code, s, b


def read_rows(cache, slots, what, bits, D, gs, page):
    """Exact values [T, H, D] of rows (fp64, not rounded); zeros outside the cache."""
    code, s, b = parts_of(cache, slots, what, bits, D, gs, page)
    return code * np.repeat(s, gs, -1) + np.repeat(b, gs, -1)


# ------------------------------------------------------------------ attention
def exact_score_rows(rng, T, H, D, gs, values):
    """(k, v) [T, H, D] as bf16 values for attention whose scores leave no room for an error of their own: column 0
    of every key is n / 64, n whole, in a group that holds 0 and 255 / 64 (an 8-bit scale of 2^-6 and a bias of 0),
    so a query of 2^j in column 0 and zeros elsewhere meets one exact product a token.  `values`: how v is drawn."""
    k = bf16(np.abs(rng.standard_normal((T, H, D)))).clip(0, 3.5)
    k[..., ::gs], k[..., 1::gs], k[..., 2::gs] = 0.0, 255 / 64, 0.0
    k[..., 0] = rng.integers(0, 256, (T, H)) / 64
    v = rng.standard_normal((T, H, D))
    if values != "symmetric":
        v = np.abs(v)                                # the group's minimum is small beside its range
    if values == "outliers":
        v[..., ::40] *= 30
    if values == "shifted":
        v += 33.0                                    # the range is small beside the mean
    return k, bf16(v)


def attn_decode(q, cache, table, lens, bits, gs, page, scale, f16, exact_scores=False):
    """(out, lse, bound, lse_bound): out [B, HQ, D] and lse [B, HQ] in fp64; bound [B, HQ, D]: how far an
    implementation may be off that forms the scores in fp32 and rounds the softmax weights, their product
    with a value scale and the centred bias to fp16 (pairs of fp16 if f16), and its result to the output type.

    With u = 2^-24, weights w_t, value parts a_t = s |code - Z| and b'_t = |bias + Z s| (Z the middle code):
      score    the sum's D + 2 D / gs fp32 steps, truncated by the MMA, each off by at most 2 u of the sum of
               magnitudes T_t = |scale| (sum_d |q_d| (code s + |bias|));  e_t = 2 u (D + 16) T_t + 2^-21
               (no allowance for products that the MMA cuts at 2^-14 of a code step of the largest |q| beside
               them, which T_t outweighs unless one |q| passes the others by far and meets small codes)
      weight   e_t twice (numerator and total), and fp16: 2^-11 (pairs: 2^-21) once for w, once for w * s or b'
      range    weights below 2^-24 of the largest lose bits: N * 2^-29 of the largest value
      sums     fp32, truncated, over at most N / 16 MMAs and 64 joins: 2 u (N / 16 + 64) of the magnitudes
      output   half a step: 2^-8 (bf16), 2^-11 (fp16), of the result
    exact_scores: q and k are such that the sums are exact (exact_score_rows, or a zero query), which leaves the
    roundings of x = scale q . k and of its distance from the maximum (up to 16 in log2 units):
    e_t = 4 u (|x_t| + 16) + 2^-21.
    lse_bound [B, HQ]: log-sum-exp moves by no more than the largest score error (it is 1-Lipschitz in the
    maximum norm), plus its total's fp32 sum, 2 u (N / 32 + 64) relative, and its own roundings, 4 u (|lse| + 16).
    """
    B, HQ, D = q.shape
    H = cache.shape[1]
    G = HQ // H
    out, lse = np.zeros((B, HQ, D)), np.full((B, HQ), -np.inf)
    bound, lse_bound = np.zeros((B, HQ, D)), np.zeros((B, HQ))
    Z = float(1 << (bits - 1))
    u = 2.0 ** -24
    for b in range(B):
        n = int(max(0, min(lens[b], table.shape[1] * page)))
        t = np.arange(n)
        ids = table[b][t // page].astype(np.int64)
        t = t[(ids >= 0) & (ids < cache.shape[0])]
        if not len(t):
            continue
        slots = table[b][t // page].astype(np.int64) * page + t % page
        kc, ks, kb = parts_of(cache, slots, "k", bits, D, gs, page)
        vc, vs, vb = parts_of(cache, slots, "v", bits, D, gs, page)
        rep = lambda x: np.repeat(x, gs, -1)  # noqa: E731
        for h in range(HQ):
            kv = h // G
            k = kc[:, kv] * rep(ks[:, kv]) + rep(kb[:, kv])
            v = vc[:, kv] * rep(vs[:, kv]) + rep(vb[:, kv])
            x = (k @ q[b, h]) * scale
            m = x.max()
            p = np.exp(x - m)
            w = p / p.sum()
            out[b, h], lse[b, h] = w @ v, m + np.log(p.sum())
            T = abs(scale) * ((kc[:, kv] * np.abs(rep(ks[:, kv])) + np.abs(rep(kb[:, kv]))) @ np.abs(q[b, h]))
            e = (4 * u * (np.abs(x) + 16) if exact_scores else 2 * u * (D + 16) * T) + 2.0 ** -21
            lse_bound[b, h] = e.max() + 2 * u * (len(t) / 32 + 64) + 4 * u * (abs(lse[b, h]) + 16)
            a = np.abs(vc[:, kv] - Z) * rep(np.abs(vs[:, kv])) + np.abs(rep(vb[:, kv] + Z * vs[:, kv]))
            mag = np.abs(v) + a
            half = 2.0 ** -21 if f16 else 2.0 ** -11
            bound[b, h] = ((2 * half + 2 * e + 2 * u * (len(t) / 16 + 64)) * w) @ mag + (w @ e) * (w @ mag) \
                + len(t) * 2.0 ** -29 * mag.max() + (2.0 ** -11 if f16 else 2.0 ** -8) * np.abs(out[b, h]) * 1.001 \
                + (2.0 ** -25 if f16 else 0.0)
    return out, lse, bound, lse_bound
