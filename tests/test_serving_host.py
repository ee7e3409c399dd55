"""CPU checks of the norm, the quantized paged cache and the decode attention: what their entry points
refuse on the host, and pins of the oracle the GPU tests compare with."""
import ctypes
import glob
import os
import re

import numpy as np
import pytest
import torch

import group_wise_bit_b200 as gwb
import oracle
from group_wise_bit_b200 import build as gbuild
from oracle import serving as S

NULL = None
OK16 = ctypes.c_void_p(0x1000)     # never dereferenced: every case below fails (or is empty) before a launch
BAD = ctypes.c_void_p(0x1001)
OK8 = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return gwb.lib()


def _st(fn, *args):
    return getattr(gwb.lib(), fn)(*args)


def _msg():
    return gwb.lib().gwb_last_error().decode()


# ------------------------------------------------------------------ refusals
def test_norm_refusals():
    def call(x=OK16, res=NULL, w=OK16, M=2, K=64, eps=1e-5, dt=0, out=NULL, qx=OK16, sx=OK16):
        return _st("gwb_rmsnorm_quant_i8", x, res, w, M, K, eps, dt, out, qx, sx, NULL)
    assert call(M=-1) == 1 and call(K=-1) == 1
    assert call(M=1 << 31) == 2 and call(K=1 << 31) == 2
    assert call(dt=2) == 3
    assert call(eps=-1e-5) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(res=OK16) == 1 and "residual_out" in _msg()
    assert call(out=OK16) == 1
    assert call(x=NULL) == 1 and call(w=NULL) == 1 and call(qx=NULL) == 1 and call(sx=NULL) == 1
    assert call(x=BAD) == 4 and call(w=OK8) == 4 and call(qx=OK8) == 4 and call(sx=OK8) == 4
    assert call(res=OK8, out=OK16) == 4 and call(res=OK16, out=OK8) == 4
    assert call(M=0, x=NULL, w=NULL, qx=NULL, sx=NULL) == 0


def test_dequant_per_token_refusals():
    def call(q=OK16, s=OK16, M=2, K=64, dt=0, out=OK16):
        return _st("gwb_dequant_per_token_i8", q, s, M, K, dt, out, NULL)
    assert call(M=-1) == 1 and call(K=1 << 31) == 2 and call(dt=5) == 3
    assert call(q=NULL) == 1 and call(s=BAD) == 4 and call(out=OK8) == 4
    assert call(M=0, q=NULL, s=NULL, out=NULL) == 0


def _cache_args(**kw):
    d = dict(pages=4, heads=2, page=16, D=64, bits=4, gs=32)
    d.update(kw)
    return d


BAD_CACHES = [(dict(bits=2), 3), (dict(bits=3), 3), (dict(gs=16), 3), (dict(D=96), 3), (dict(D=64, gs=128), 2),
              (dict(page=24), 2), (dict(page=8), 2), (dict(page=8192), 2), (dict(page=-16), 1), (dict(pages=-1), 1),
              (dict(heads=0), 2), (dict(heads=-1), 1), (dict(pages=1 << 31), 2)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refusals(kw, code):
    c = _cache_args(**kw)
    row = c["heads"] * c["D"]
    assert _st("gwb_kv_write", OK16, row, OK16, row, OK16, 3, 0, OK16, c["pages"], c["heads"], c["page"], c["D"],
               c["bits"], c["gs"], NULL) == code
    assert _st("gwb_kv_read", OK16, c["pages"], c["heads"], c["page"], c["D"], c["bits"], c["gs"], OK16, 3, 0, OK16,
               OK16, NULL) == code
    assert _st("gwb_attn_decode", OK16, row, 1, max(1, c["heads"]), 0, OK16, c["pages"], c["heads"], c["page"],
               c["D"], c["bits"], c["gs"], OK16, 4, 4, OK16, 1.0, OK16, NULL, OK16, 1 << 30, NULL) == code


def test_write_and_read_refusals():
    def write(k=OK16, ks=128, v=OK16, vs=128, slots=OK16, T=3, dt=0, cache=OK16, pages=4):
        return _st("gwb_kv_write", k, ks, v, vs, slots, T, dt, cache, pages, 2, 16, 64, 4, 32, NULL)
    assert write(T=-1) == 1 and write(T=1 << 31) == 2
    assert write(dt=7) == 3
    assert write(k=NULL) == 1 and write(v=NULL) == 1 and write(slots=NULL) == 1 and write(cache=NULL) == 1
    assert write(k=OK8) == 4 and write(v=BAD) == 4 and write(cache=OK8) == 4
    assert write(slots=ctypes.c_void_p(0x1004)) == 4
    assert write(ks=120) == 2 and write(vs=0) == 2          # rows that overlap
    assert write(ks=130) == 4 and write(vs=132) == 4        # rows that lose their 16-byte alignment
    assert write(T=0, k=NULL, v=NULL, slots=NULL, cache=NULL) == 0

    def read(k=OK16, v=OK16, slots=OK16, T=3, dt=0, cache=OK16):
        return _st("gwb_kv_read", cache, 4, 2, 16, 64, 4, 32, slots, T, dt, k, v, NULL)
    assert read(T=-1) == 1 and read(T=1 << 31) == 2 and read(dt=-1) == 3
    assert read(k=NULL) == 1 and read(v=NULL) == 1 and read(slots=NULL) == 1 and read(cache=NULL) == 1
    assert read(k=OK8) == 4 and read(v=OK8) == 4 and read(cache=BAD) == 4
    assert read(T=0, k=NULL, v=NULL, slots=NULL, cache=NULL) == 0


def test_attention_refusals():
    def call(q=OK16, qs=512, B=2, HQ=8, dt=0, cache=OK16, pages=4, table=OK16, ts=4, most=4, lens=OK16, scale=0.125,
             out=OK16, lse=NULL, ws=OK16, n=1 << 30):
        return _st("gwb_attn_decode", q, qs, B, HQ, dt, cache, pages, 2, 16, 64, 4, 32, table, ts, most, lens, scale,
                   out, lse, ws, n, NULL)
    assert call(HQ=7, qs=448) == 2 and call(HQ=0) == 2 and call(HQ=65536, qs=65536 * 64) == 2
    assert call(B=-1) == 1 and call(most=-1) == 1 and call(B=1 << 24) == 2 and call(most=1 << 31, ts=1 << 31) == 2
    assert call(ts=3) == 2
    assert call(dt=3) == 3
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    for name in ("q", "cache", "table", "lens", "out"):
        assert call(**{name: NULL}) == 1, name
    assert call(n=-1) == 1
    for name in ("q", "cache", "out", "ws"):
        assert call(**{name: OK8}) == 4, name
    for name in ("table", "lens", "lse"):
        assert call(**{name: ctypes.c_void_p(0x1002)}) == 4, name
    assert call(qs=500) == 2 and call(qs=516) == 4
    assert call(B=0, q=NULL, cache=NULL, table=NULL, lens=NULL, out=NULL, ws=NULL) == 0


def test_block_bytes():
    n = ctypes.c_int64(0)
    for bits in (4, 8):
        for D in (64, 128, 256):
            for gs in (32, 64, 128):
                st = _st("gwb_kv_block_bytes", 64, D, bits, gs, ctypes.byref(n))
                if gs > D:
                    assert st == 2
                else:
                    # codes of keys and values, and a bf16 scale and bias a group of each
                    assert st == 0 and n.value == 64 * 2 * (D * bits // 8 + D // gs * 4)
                    assert n.value == 4 * S.Layout(bits, D, gs).bytes
    assert _st("gwb_kv_block_bytes", 64, 128, 4, 64, NULL) == 1
    assert _st("gwb_attn_decode_workspace", 8, 3, 128, 0, 0, ctypes.byref(n)) == 2
    assert _st("gwb_attn_decode_workspace", 8, 2, 128, 0, 0, NULL) == 1
    assert _st("gwb_attn_decode_workspace", 8, 2, 128, -1, 0, ctypes.byref(n)) == 1


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        gwb.rmsnorm_quant_i8(x, x[0], 1e-5)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16 * 2 * (32 + 8), dtype=torch.uint8)
    slots = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        gwb.kv_write(cache, slots, k, k, 4, 32)
    with pytest.raises(ValueError, match="CUDA"):
        gwb.kv_read(cache, slots, 64, 4, 32)
    with pytest.raises(ValueError, match="CUDA"):
        gwb.attn_decode(k, cache, torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32), 4, 32)
    with pytest.raises(gwb.GwbError, match="UNSUPPORTED"):
        gwb.kv_cache(4, 2, 96, 16, 4, 32, device="cpu")
    with pytest.raises(gwb.GwbError, match="SHAPE"):
        gwb.kv_cache(4, 2, 128, 20, 4, 32, device="cpu")
    c = gwb.kv_cache(4, 2, 64, 16, 4, 32, device="cpu")
    assert c.shape == cache.shape and c.dtype == torch.uint8 and not c.any()


# ------------------------------------------------------------------ pins of the oracle
def test_bf16_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * np.exp(15 * rng.standard_normal(20000))).astype(np.float32)
    x[:4] = [0.0, -0.0, 1.00390625, 3.0e38]           # signed zeros, a tie, the top binade
    assert np.array_equal(S.bf16(x), torch.tensor(x).bfloat16().double().numpy())
    assert np.array_equal(S.bits_bf16(S.bf16_bits(S.bf16(x))), S.bf16(x))


@pytest.mark.parametrize("bits,D,gs", [(b, D, g) for b in (4, 8) for D in (64, 128, 256) for g in (32, 64, 128) if g <= D])
def test_every_bit_of_a_granule_has_one_use(bits, D, gs):
    lay = S.Layout(bits, D, gs)
    used = np.zeros(8 * lay.bytes, dtype=int)
    for t in range(16):
        for d in range(D):
            for o in (lay.key_bits(t, d), lay.val_bits(t, d)):
                used[o:o + bits] += 1
        for g in range(D // gs):
            for o in (lay.key_meta(t, g), lay.key_meta(t, g) + 2, lay.val_scale(t, g), lay.val_bias(t, g)):
                used[8 * o:8 * o + 16] += 1
    assert (used == 1).all()


@pytest.mark.parametrize("bits,gs", [(4, 32), (8, 64)])
def test_rows_quantize_as_the_affine_packer(bits, gs):
    """The cache's quantizer is the oracle's qpack_affine on the row, and rows come back as they were written."""
    rng = np.random.default_rng(bits)
    rows = S.bf16(rng.standard_normal((20, 3, 128)))
    rows[0, 0, :gs] = 0.0
    rows[0, 1, 0] = -0.0                              # a group of both zeros: its bias is -0
    rows[1, 0, :] = 1.5                               # constant groups
    code, s, b = S.quantize_rows(rows, bits, gs)
    wq, sc, bi, _ = oracle.qpack_affine(rows.reshape(60, 128).astype(np.float32), bits, gs)
    packed = np.asarray(wq).view(np.uint32).reshape(60, -1)
    per = 32 // bits
    words = code.reshape(60, -1, per).astype(np.uint32)
    words = np.bitwise_or.reduce(words << (np.arange(per, dtype=np.uint32) * bits), axis=-1)
    assert np.array_equal(words, packed)
    assert np.array_equal(S.bf16_bits(s).reshape(60, -1), sc) and np.array_equal(S.bf16_bits(b).reshape(60, -1), bi)
    cache = rng.integers(0, 256, (3, 3, 16 * S.Layout(bits, 128, gs).bytes // 16), dtype=np.uint8)
    before = cache.copy()
    slots = np.array(list(rng.permutation(48)[:18]) + [-1, 48])
    S.write_rows(cache, slots, rows, "k", bits, gs, 16)
    S.write_rows(cache, slots, rows[::-1], "v", bits, gs, 16)
    exact = code * np.repeat(s, gs, -1) + np.repeat(b, gs, -1)
    exact[18:] = 0
    assert np.array_equal(S.read_rows(cache, slots, "k", bits, 128, gs, 16), exact)
    free = np.setdiff1d(np.arange(48), slots)
    for new, old in zip(S.parts_of(cache, free, "v", bits, 128, gs, 16), S.parts_of(before, free, "v", bits, 128, gs, 16)):
        assert np.array_equal(new, old, equal_nan=True)      # (the untouched rows' scales are any bits)


def test_norm_pins():
    # a row of ones: r = 1 / sqrt(1 + eps), y = r, every code 127
    q, s, h = S.rmsnorm_quant_i8(np.ones((1, 8)), None, np.ones(8), 0.0, False)
    assert (q == 127).all() and s[0] == np.float32(1) / np.float32(127) and np.array_equal(h, np.ones((1, 8)))
    q, s, _ = S.rmsnorm_quant_i8(np.zeros((1, 8)), None, np.ones(8), 1e-6, False)
    assert (q == 0).all() and s[0] == 0
    # codes are the nearest grid points of the norm, and sign symmetric
    rng = np.random.default_rng(3)
    x, w = S.bf16(rng.standard_normal((5, 96))), S.bf16(1 + 0.1 * rng.standard_normal(96))
    q, s, _ = S.rmsnorm_quant_i8(x, None, w, 1e-5, False)
    y = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-5) * w
    assert np.abs(y / s[:, None] - q).max() <= 0.5 + 1e-4 and (np.abs(q).max(1) == 127).all()
    q2, s2, _ = S.rmsnorm_quant_i8(-x, None, w, 1e-5, False)
    assert np.array_equal(q2, -q) and np.array_equal(s2, s)
    # the residual's sum is rounded to the activations' type before the norm
    _, _, h = S.rmsnorm_quant_i8(np.full((1, 4), 256.0), np.full((1, 4), 0.5), np.ones(4), 0.0, False)
    assert (h == 256.0).all()


def test_attention_pins():
    """Against a dense softmax in numpy on the rows as read, a single token, and an empty row."""
    rng = np.random.default_rng(5)
    bits, D, gs, page, H = 8, 64, 32, 32, 2
    cache = np.zeros((4, H, 2 * S.Layout(bits, D, gs).bytes), dtype=np.uint8)
    k, v = S.bf16(rng.standard_normal((128, H, D))), S.bf16(rng.standard_normal((128, H, D)))
    S.write_rows(cache, np.arange(128), k, "k", bits, gs, page)
    S.write_rows(cache, np.arange(128), v, "v", bits, gs, page)
    q = S.bf16(rng.standard_normal((3, 4, D)))
    table = np.array([[2, 0, 3], [1, 9, 1], [0, 0, 0]], dtype=np.int32)
    out, lse, bound, lse_bound = S.attn_decode(q, cache, table, np.array([70, 1, 0]), bits, gs, page, 0.125, False)
    at = np.concatenate([np.arange(64, 96), np.arange(0, 32), np.arange(96, 102)])
    kd, vd = (S.read_rows(cache, at, w, bits, D, gs, page) for w in "kv")
    for h in range(4):
        p = np.exp(0.125 * kd[:, h // 2] @ q[0, h])
        assert np.allclose(out[0, h], p @ vd[:, h // 2] / p.sum(), rtol=1e-12, atol=1e-14)
        assert np.isclose(lse[0, h], np.log(p.sum()), rtol=1e-13)
    one = S.read_rows(cache, [32], "v", bits, D, gs, page)[0]
    assert np.allclose(out[1], np.repeat(one, 2, 0), rtol=1e-15, atol=0)
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all() and (bound[2] == 0).all() and (lse_bound[:2] > 0).all()
    # half a step of a range of up to 8, and the bf16 roundings of scale and bias (2^-9 of range and minimum)
    assert np.abs(kd - k[at]).max() < 8 / 255 / 2 + 8 * 2.0 ** -9 + 4 * 2.0 ** -9 and (bound[:2] > 0).all()


# ------------------------------------------------------------------ what the attention's bound tells apart
def _one_row(values, seed):
    """Largest error over bound of fp16 attention restated in numpy (8 bits, D 128, groups of 64, 3 tokens, one
    head): with the remainders of the weights' and of the biases' fp16 rounding taken along, without the weights',
    without the biases'."""
    rng = np.random.default_rng(seed)
    bits, D, gs, page = 8, 128, 64, 16
    k, v = S.exact_score_rows(rng, 3, 1, D, gs, values)
    cache = np.zeros((1, 1, S.Layout(bits, D, gs).bytes), dtype=np.uint8)
    S.write_rows(cache, np.arange(3), k, "k", bits, gs, page)
    S.write_rows(cache, np.arange(3), v, "v", bits, gs, page)
    q = np.zeros((1, 1, D))
    q[..., 0] = 1.0
    ref, _, bound, _ = S.attn_decode(q, cache, np.zeros((1, 1), dtype=np.int32), [3], bits, gs, page, 1.0, True,
                                     exact_scores=True)
    h = lambda x: np.asarray(x, dtype=np.float16).astype(np.float64)  # noqa: E731
    code, s, b = (x[:, 0] for x in S.parts_of(cache, np.arange(3), "v", bits, D, gs, page))
    x = S.read_rows(cache, np.arange(3), "k", bits, D, gs, page)[:, 0, 0]
    assert np.array_equal(x, k[:, 0, 0])             # the keys' column is exact
    p = 2.0 ** 10 * np.exp(x - x.max())
    # scales and biases over the power of two that holds both
    e = 2.0 ** np.ceil(np.log2(np.maximum(s * 2 ** bits, np.abs(b)).max(0)) + 1)
    sc, bi = s / e * 2 ** bits, (b + 128 * s) / e
    worst = []
    for weights, biases in ((1, 1), (0, 1), (1, 0)):
        hi = h(p)
        lo = weights * h(p - hi)
        ps = h(hi[:, None] * sc)
        pl = weights * h(lo[:, None] * sc + h(hi[:, None] * sc - ps))
        bh = h(bi)
        bl = biases * h((bi - bh) * 2 ** 11) / 2 ** 11
        o = ((np.repeat(ps + pl, gs, 1) * (code - 128)).sum(0) / 2 ** bits
             + np.repeat(((hi + lo)[:, None] * (bh + bl)).sum(0), gs)) * np.repeat(e, gs) / p.sum()
        worst.append((np.abs(h(o) - ref[0, 0]) / bound[0, 0]).max())
    return worst


@pytest.mark.parametrize("values", ["symmetric", "small minimum", "outliers", "shifted"])
def test_attention_bound_sees_a_lost_remainder(values):
    """fp16 outputs keep within the bound of exact scores with every remainder, and leave it without the weights'
    or (where a bias does not fit fp16) the biases'."""
    both, no_weights, no_biases = np.max([_one_row(values, seed) for seed in range(6)], axis=0)
    assert both <= 1.0
    assert no_weights > 1.05
    if values != "symmetric":
        assert no_biases > 1.05


# ------------------------------------------------------------------ shared memory
def test_dynamic_shared_memory_states_its_alignment():
    """Vector accesses, cp.async and bulk copies need 16 bytes: each kernel's dynamic buffer says so, whatever the
    size of the static variables in front of it."""
    found = 0
    for src in sorted(glob.glob(os.path.join(gbuild.CSRC, "*.cu*"))):
        for line in open(src):
            if "extern __shared__" in line:
                m = re.search(r"__align__\((\d+)\)", line)
                assert m and int(m.group(1)) % 16 == 0, f"{os.path.basename(src)}: {line.strip()}"
                found += 1
    assert found >= 8


def test_norm_of_zeros_without_eps_is_zero():
    q, s, _ = S.rmsnorm_quant_i8(np.array([[0.0, -0.0], [3.0, -4.0]]), None, np.ones(2), 0.0, False)
    r = np.float32(1 / np.sqrt(12.5))
    assert s[0] == 0 and not q[0].any() and q[1].tolist() == [95, -127] and s[1] == np.float32(4) * r / np.float32(127)
