"""GPU parity of the norm with an int8 output, the quantized paged cache and the decode attention.

Codes, scales, biases, int8 values and residual sums must be bit-exact with the oracle (fp32 steps as the
definitions state them); attention outputs must lie within the elementwise bound the oracle derives from
fp32 scores, fp16 softmax weights and one output rounding (oracle.serving.attn_decode).
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import serving as S

gwb = pytest.importorskip("group_wise_bit_b200")
pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _t(x, dt):
    return torch.tensor(np.ascontiguousarray(x)).to(DT[dt]).to(DEV)


def _np(t):
    return t.double().cpu().numpy()


def _rand(rng, shape, dt, spread=1.0):
    return S.rnd(spread * rng.standard_normal(shape), dt == "fp16")


# ------------------------------------------------------------------ norm
def _check_norm(x, res, w, dt, eps=1e-5, **kw):
    q, s, h = gwb.rmsnorm_quant_i8(_t(x, dt), _t(w, dt), eps, residual=None if res is None else _t(res, dt), **kw)
    q_o, s_o, h_o = S.rmsnorm_quant_i8(x, res, w, eps, dt == "fp16")
    assert np.array_equal(s.cpu().numpy().view(np.uint32), s_o.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), q_o)
    if res is None:
        assert h is None
    else:
        assert np.array_equal(_np(h), h_o)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 5), (1, 8), (7, 64), (2, 257), (5, 5003), (33, 2048), (2, 8192), (2, 8200),
                                 (3, 12289), (1, 16384), (1, 32768), (2, 32776), (1, 40001)])
def test_norm_bit_exact(M, K, dt):
    rng = np.random.default_rng(M * 100003 + K)
    x, w = _rand(rng, (M, K), dt), _rand(rng, K, dt, 0.2) + 1.0
    w = S.rnd(w, dt == "fp16")
    x[:, :: max(1, K // 5)] *= 16                     # outlier channels
    _check_norm(x, None, w, dt)
    _check_norm(x, _rand(rng, (M, K), dt, 3.0), w, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_norm_edges(dt):
    rng = np.random.default_rng(9)
    x = _rand(rng, (9, 520), dt)
    w = S.rnd(1 + 0.1 * rng.standard_normal(520), dt == "fp16")
    x[0] = 0.0                                        # a zero row: scale 0, codes 0
    x[1, 1:] = 0.0                                    # a single value
    x[2] = S.rnd(x[2] * 1e-6, dt == "fp16")           # small rows (fp16 subnormals): eps takes over
    x[3] = S.rnd(x[3] * 1e4, dt == "fp16")
    x[4] = 1.0
    w[7] = 0.0
    _check_norm(x, None, w, dt)
    _check_norm(x, -x, w, dt)                         # every sum is zero
    _check_norm(x[5:], None, w, dt, eps=0.0)
    _check_norm(x, _rand(rng, x.shape, dt), np.zeros(520), dt)
    if dt == "bf16":                                  # the squares and scales pass fp32's normal range
        big = S.bf16(x * 1e30)
        _check_norm(big, None, w, dt)
        tiny = S.bf16(rng.standard_normal((2, 520)))
        _check_norm(tiny, None, S.bf16(w * 2.0 ** -130), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K", [(5, 72), (5, 77), (700, 4096), (5, 40000)])
def test_norm_rows_that_are_not_finite(M, K, dt):
    """A NaN, an infinity, a sum that overflows: sx is not finite and the codes are 0; other rows keep their results."""
    rng = np.random.default_rng(K)
    x, r, w = _rand(rng, (M, K), dt), _rand(rng, (M, K), dt), S.rnd(1 + 0.1 * rng.standard_normal(K), dt == "fp16")
    q_o, s_o, h_o = S.rmsnorm_quant_i8(x, r, w, 1e-5, dt == "fp16")
    xt, rt = _t(x, dt), _t(r, dt)
    xt[0, K - 1] = float("nan")
    xt[2, 3] = float("-inf")
    xt[3, 0] = rt[3, 0] = torch.finfo(DT[dt]).max
    q, s, h = gwb.rmsnorm_quant_i8(xt, _t(w, dt), 1e-5, residual=rt)
    bad = [0, 2, 3]
    assert torch.isnan(s[bad]).all() and not q[bad].any()
    assert torch.isnan(h[0, -1]) and h[2, 3] == float("-inf") and h[3, 0] == float("inf")
    good = np.setdiff1d(np.arange(M), bad)
    assert np.array_equal(q.cpu().numpy()[good], q_o[good]) and np.array_equal(s.cpu().numpy()[good], s_o[good])
    assert np.array_equal(_np(h)[good], h_o[good])
    # a weight that is not finite: every row
    wt = _t(w, dt)
    wt[K // 2] = float("nan")
    q, s, _ = gwb.rmsnorm_quant_i8(_t(x, dt), wt, 1e-5)
    assert torch.isnan(s).all() and not q.any()


def test_norm_in_place_and_into_given_outputs():
    rng = np.random.default_rng(11)
    M, K = 6, 1000
    x, r, w = _rand(rng, (M, K), "bf16"), _rand(rng, (M, K), "bf16"), _rand(rng, K, "bf16")
    q_o, s_o, h_o = S.rmsnorm_quant_i8(x, r, w, 1e-6, False)
    for alias in ("x", "residual"):
        xt, rt = _t(x, "bf16"), _t(r, "bf16")
        qx, sx = torch.full((M, K), 99, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
        out = xt if alias == "x" else rt
        got = gwb.rmsnorm_quant_i8(xt, _t(w, "bf16"), 1e-6, residual=rt, residual_out=out, qx=qx, sx=sx)
        assert got[0] is qx and got[1] is sx and got[2] is out
        assert np.array_equal(_np(out), h_o) and np.array_equal(qx.cpu().numpy(), q_o)
        assert np.array_equal(sx.cpu().numpy(), s_o)
    q, s, _ = gwb.rmsnorm_quant_i8(_t(x[:0], "bf16"), _t(w, "bf16"), 1e-6)
    assert q.shape == (0, K) and s.shape == (0,)


def test_norm_equals_the_quantizer_where_the_norm_is_exact():
    """Rows whose norm is representable in bf16: the same codes and scales as quant_per_token_i8."""
    x = torch.tensor([[1.0, -1.0, 1.0, 1.0] * 64, [2.0, -2.0, 2.0, -2.0] * 64], dtype=torch.bfloat16, device=DEV)
    w = torch.tensor([0.5, 1.0, 1.5, 2.0] * 64, dtype=torch.bfloat16, device=DEV)
    q, s, _ = gwb.rmsnorm_quant_i8(x, w, 0.0)
    y = torch.sign(x) * w
    q2, s2 = gwb.quant_per_token_i8(y.contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 16), (5, 17), (2, 4096), (300, 144), (7, 5003)])
def test_dequant_per_token_bit_exact(M, K, dt):
    rng = np.random.default_rng(K)
    q = rng.integers(-128, 128, (M, K)).astype(np.int8)
    s = (np.exp(3 * rng.standard_normal(M)) * (rng.random(M) > 0.2)).astype(np.float32)
    got = gwb.dequant_per_token_i8(torch.tensor(q).to(DEV), torch.tensor(s).to(DEV), dtype=DT[dt])
    assert np.array_equal(_np(got), S.rnd(q.astype(np.float32) * s[:, None], dt == "fp16"))


# ------------------------------------------------------------------ cache
LAYOUTS = [(b, D, g) for b in (4, 8) for D in (64, 128, 256) for g in (32, 64, 128) if g <= D]


def _random_cache(rng, pages, H, D, page, bits, gs):
    """Any bytes (NaN scales among them): what an uninitialised cache holds."""
    return rng.integers(0, 256, (pages, H, page // 16 * S.Layout(bits, D, gs).bytes), dtype=np.uint8)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,D,gs", LAYOUTS)
def test_cache_write_and_read_bit_exact(bits, D, gs, dt):
    rng = np.random.default_rng(bits * D + gs)
    H, page, pages = 3, 16 if D == 64 else 32, 5
    T = 37
    k, v = _rand(rng, (T, H, D), dt), _rand(rng, (T, H, D), dt, 5.0)
    k[0, 0] = 0.0
    k[0, 0, 5] = -0.0                                 # a group of both zeros: its bias is -0
    k[1, 1, 3] = -0.0
    v[2, 2] = 1.25                                    # constant groups
    v[3, 0, ::7] *= 100
    k, v = S.rnd(k, dt == "fp16"), S.rnd(v, dt == "fp16")   # what the cast to dt hands to the kernel
    slots = rng.permutation(pages * page)[:T]
    slots[[5, 36]] = -1                               # padded rows, one behind the last
    cache = _random_cache(rng, pages, H, D, page, bits, gs)
    dev = torch.tensor(cache).to(DEV)
    st = torch.tensor(slots).to(DEV)
    gwb.kv_write(dev, st, _t(k, dt), _t(v, dt), bits, gs)
    S.write_rows(cache, slots, k, "k", bits, gs, page)
    S.write_rows(cache, slots, v, "v", bits, gs, page)
    assert np.array_equal(dev.cpu().numpy(), cache)   # untouched rows keep their bytes
    for out in DT:
        kr, vr = gwb.kv_read(dev, st, D, bits, gs, dtype=DT[out])
        for got, what in ((kr, "k"), (vr, "v")):
            code, s, b = S.parts_of(cache, slots, what, bits, D, gs, page)
            ref = (code * np.repeat(s, gs, -1) + np.repeat(b, gs, -1)).astype(np.float32)
            assert np.array_equal(_np(got), S.rnd(ref, out == "fp16"))
    gwb.check_device_error()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,D,gs", LAYOUTS)
def test_cache_groups_that_are_not_finite(bits, D, gs, dt):
    """A group with a NaN or an infinity reads back as NaN; every other byte of the cache is what it was without."""
    rng = np.random.default_rng(bits * D + gs)
    T, H, page = 32, 2, 32
    k, v = _t(_rand(rng, (T, H, D), dt), dt), _t(_rand(rng, (T, H, D), dt), dt)
    for order in (torch.arange(T), torch.randperm(T)):          # whole granules, single rows
        slots = order.to(DEV)
        ref = gwb.kv_cache(1, H, D, page, bits, gs)
        gwb.kv_write(ref, slots, k, v, bits, gs)
        for what, x in enumerate((k, v)):
            bad = x.clone()
            hit = torch.zeros(T, H, D // gs, dtype=torch.bool, device=DEV)
            for i, value in enumerate((float("nan"), float("inf"), float("-inf"))):
                at = (5 * i + 1, i % H, (37 * i) % D)
                bad[at] = value
                hit[at[0], at[1], at[2] // gs] = True
            cache = gwb.kv_cache(1, H, D, page, bits, gs)
            gwb.kv_write(cache, slots, *((bad, v) if what == 0 else (k, bad)), bits, gs)
            rows, clean = gwb.kv_read(cache, slots, D, bits, gs), gwb.kv_read(ref, slots, D, bits, gs)
            cols = hit.repeat_interleave(gs, 2)
            assert torch.isnan(rows[what][cols]).all()
            assert torch.equal(rows[what][~cols], clean[what][~cols]) and torch.equal(rows[1 - what], clean[1 - what])


def test_cache_rows_are_the_affine_packers():
    """Codes, scales and biases of a written row are qpack_affine's of the same row."""
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn(50, 2, 128, device=DEV, generator=g).bfloat16()
    cache = gwb.kv_cache(4, 2, 128, 16, 4, 64)
    slots = torch.randperm(64, device=DEV, generator=g)[:50]
    gwb.kv_write(cache, slots, k, k, 4, 64)
    kr, vr = gwb.kv_read(cache, slots, 128, 4, 64)
    wq, sc, bi = gwb.qpack_affine(k.float().reshape(100, 128).contiguous(), 4, 64)
    ref = gwb.dequant_affine(wq, sc, bi, 128, 4, 64).view(50, 2, 128)
    assert torch.equal(kr, ref) and torch.equal(vr, ref)


@pytest.mark.parametrize("bits", [4, 8])
def test_cache_codes_on_the_border(bits):
    """Rows of few distinct bf16 values put many quotients halfway between two codes, and scales over all
    exponents and significands: the same codes as the packer, which divides."""
    g = torch.Generator(device=DEV).manual_seed(bits)
    T, D, gs = 6000, 128, 32
    k = torch.randint(-24, 25, (T, 1, D), device=DEV, generator=g).float()
    step = torch.exp2(torch.randint(-60, 60, (T, 1, 1), device=DEV, generator=g).float())
    step *= 1 + torch.randint(0, 128, (T, 1, 1), device=DEV, generator=g) / 128
    k = (k * step).bfloat16()
    v = torch.randn(T, 1, D, device=DEV, generator=g).mul_(step).bfloat16()
    cache = gwb.kv_cache(-(-T // 16), 1, D, 16, bits, gs)
    gwb.kv_write(cache, torch.arange(T, device=DEV), k, v, bits, gs)
    for x, what in ((k, "k"), (v, "v")):
        wq, sc, bi = gwb.qpack_affine(x.float().reshape(T, D).contiguous(), bits, gs)
        code, s, b = S.parts_of(cache.cpu().numpy(), np.arange(T), what, bits, D, gs, 16)
        words = wq.cpu().numpy().view(np.uint32)
        ref = (words[:, :, None] >> (np.arange(32 // bits, dtype=np.uint32) * bits)) & ((1 << bits) - 1)
        assert np.array_equal(code.reshape(T, D), ref.reshape(T, D))
        assert np.array_equal(s.reshape(T, -1), _np(sc)) and np.array_equal(b.reshape(T, -1), _np(bi))


@pytest.mark.parametrize("T", [1, 2, 300])
def test_cache_strided_rows_and_odd_slot_views(T):
    rng = np.random.default_rng(T)
    H, Hq, D, bits, gs, page = 5, 15, 64, 8, 64, 64
    qkv = _rand(rng, (T, (Hq + 2 * H) * D), "fp16")
    pages = T // page + 2
    cache = gwb.kv_cache(pages, H, D, page, bits, gs)
    t = _t(qkv, "fp16")
    k, v = t[:, Hq * D:(Hq + H) * D].view(T, H, D), t[:, (Hq + H) * D:].view(T, H, D)
    slots = np.concatenate([[0], rng.permutation(pages * page)[:T]])
    st = torch.tensor(slots).to(DEV)[1:]              # 8-byte aligned only
    gwb.kv_write(cache, st, k, v, bits, gs)
    ref = np.zeros(tuple(cache.shape), dtype=np.uint8)
    S.write_rows(ref, slots[1:], qkv[:, Hq * D:(Hq + H) * D].reshape(T, H, D), "k", bits, gs, page)
    S.write_rows(ref, slots[1:], qkv[:, (Hq + H) * D:].reshape(T, H, D), "v", bits, gs, page)
    assert np.array_equal(cache.cpu().numpy(), ref)
    out = torch.full((T, H, D), 7.0, dtype=torch.float16, device=DEV)
    kr, vr = gwb.kv_read(cache, st, D, bits, gs, dtype=torch.float16, k=out)
    assert kr is out
    assert np.array_equal(_np(kr), S.rnd(S.read_rows(ref, slots[1:], "k", bits, D, gs, page).astype(np.float32), True))


def test_cache_slots_outside_are_left_out_and_reported():
    cache = gwb.kv_cache(2, 1, 64, 16, 4, 32)
    k = torch.ones(4, 1, 64, dtype=torch.bfloat16, device=DEV)
    k[:, :, ::2] = 2.0
    slots = torch.tensor([3, 32, -5, 1 << 40], device=DEV)
    gwb.kv_write(cache, slots, k, k, 4, 32)
    with pytest.raises(gwb.GwbError, match="INVALID_ARG"):
        gwb.check_device_error()
    gwb.check_device_error()                          # reading it cleared it
    ref = np.zeros(tuple(cache.shape), dtype=np.uint8)
    S.write_rows(ref, [3], _np(k[:1]), "k", 4, 32, 16)
    S.write_rows(ref, [3], _np(k[:1]), "v", 4, 32, 16)
    assert np.array_equal(cache.cpu().numpy(), ref)
    kr, vr = gwb.kv_read(cache, slots, 64, 4, 32)
    with pytest.raises(gwb.GwbError, match="INVALID_ARG"):
        gwb.check_device_error()
    assert torch.equal(kr[0], k[0]) and not kr[1:].any() and not vr[1:].any()
    kr, _ = gwb.kv_read(cache, slots[[0, 2, 0]].contiguous(), 64, 4, 32)      # repeats, and padding alone: no error
    assert torch.equal(kr[0], k[0]) and torch.equal(kr[2], k[0]) and not kr[1].any()
    gwb.check_device_error()
    assert gwb.kv_read(cache, slots[:0], 64, 4, 32)[0].shape == (0, 1, 64)
    gwb.kv_write(cache, slots[:0], k[:0], k[:0], 4, 32)


def test_a_slot_named_twice_touches_nothing_else():
    """Slots must be distinct; one named twice holds some mixture, and every other row is what it should be."""
    rng = np.random.default_rng(40)
    T, H, D = 64, 2, 128
    k, v = _rand(rng, (T, H, D), "bf16"), _rand(rng, (T, H, D), "bf16")
    slots = np.arange(T)
    slots[[3, 20, 47]] = [50, 50, 21]
    ref = _random_cache(rng, 5, H, D, 16, 4, 64)
    cache = torch.tensor(ref).to(DEV)
    gwb.kv_write(cache, torch.tensor(slots).to(DEV), _t(k, "bf16"), _t(v, "bf16"), 4, 64)
    S.write_rows(ref, slots, k, "k", 4, 64, 16)
    S.write_rows(ref, slots, v, "v", 4, 64, 16)
    got = cache.cpu().numpy()
    rest = np.setdiff1d(np.arange(80), [50, 21])
    for what in "kv":
        for a, b in zip(S.parts_of(got, rest, what, 4, D, 64, 16), S.parts_of(ref, rest, what, 4, D, 64, 16)):
            assert np.array_equal(a, b, equal_nan=True)
    gwb.check_device_error()


def test_binding_refusals_on_the_gpu():
    cache = gwb.kv_cache(4, 2, 64, 16, 4, 32)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(3, device=DEV)
    with pytest.raises(ValueError, match="heads"):
        gwb.kv_write(cache, slots, k[:, :1].contiguous(), k[:, :1].contiguous(), 4, 32)
    with pytest.raises(ValueError, match="contiguous"):
        gwb.kv_write(cache, slots, k.transpose(1, 2).contiguous().transpose(1, 2), k, 4, 32)
    with pytest.raises(TypeError, match="v"):
        gwb.kv_write(cache, slots, k, k.half(), 4, 32)
    with pytest.raises(TypeError, match="slots"):
        gwb.kv_write(cache, slots.int(), k, k, 4, 32)
    with pytest.raises(ValueError, match="block"):
        gwb.kv_write(cache[:, :, :-16].contiguous(), slots, k, k, 4, 32)
    with pytest.raises(gwb.GwbError, match="ALIGN"):
        gwb.kv_write(cache, slots, torch.zeros(3 * 132, dtype=torch.bfloat16, device=DEV).view(3, 132)[:, :128].view(3, 2, 64),
                     k, 4, 32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    long = torch.zeros(2, 64, dtype=torch.int32, device=DEV)          # 1024 tokens: such tables are cut
    with pytest.raises(gwb.GwbError, match="workspace"):
        gwb.attn_decode(q, cache, long, lens, 4, 32, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert gwb.attn_decode_workspace(4, 2, 64, 2, 512) == 0
    assert 0 < gwb.attn_decode_workspace(4, 2, 64, 2, 1024) == gwb.attn_decode_workspace(4, 2, 64)
    with pytest.raises(gwb.GwbError, match="SHAPE"):
        gwb.attn_decode(q[:, :3].contiguous(), cache, table, lens, 4, 32)
    with pytest.raises(TypeError, match="page_table"):
        gwb.attn_decode(q, cache, table.long(), lens, 4, 32)
    with pytest.raises(ValueError, match="page_table"):
        gwb.attn_decode(q, cache, table[:1], lens, 4, 32)
    with pytest.raises(ValueError, match="seq_lens"):
        gwb.attn_decode(q, cache, table, lens[:1], 4, 32)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="residual_out"):
        gwb.rmsnorm_quant_i8(x, x[0], 1e-5, residual_out=x)
    with pytest.raises(TypeError, match="weight"):
        gwb.rmsnorm_quant_i8(x, x[0].float(), 1e-5)
    gwb.check_device_error()


# ------------------------------------------------------------------ attention
class Batch:
    """Sequences of given lengths in a paged cache whose other rows are any bytes."""

    def __init__(self, lens, H, G, D, bits, gs, page, dt, seed=0, k_spread=1.0, v_spread=1.0, q_spread=1.0, v_shift=0.0):
        rng = np.random.default_rng(seed)
        self.H, self.G, self.D, self.bits, self.gs, self.page, self.dt = H, G, D, bits, gs, page, dt
        self.lens = np.asarray(lens, dtype=np.int32)
        need = -(-np.maximum(self.lens, 0) // page)
        most = max(1, int(need.max()))
        pages = int(need.sum()) + 2
        order = rng.permutation(pages)
        self.table = rng.integers(0, pages, (len(lens), most)).astype(np.int32)   # unused entries name any page
        at = 0
        slots = []
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            t = np.arange(max(0, self.lens[b]))
            slots.append(self.table[b][t // page].astype(np.int64) * page + t % page)
        slots = np.concatenate(slots)
        self.k = _rand(rng, (len(slots), H, D), "bf16", k_spread)
        self.v = S.bf16(_rand(rng, (len(slots), H, D), "bf16", v_spread) + v_shift)
        self.q = _rand(rng, (len(lens), H * G, D), dt, q_spread)
        cache = torch.tensor(_random_cache(rng, pages, H, D, page, bits, gs)).to(DEV)
        self.slots = torch.tensor(slots).to(DEV)
        if len(slots):
            gwb.kv_write(cache, self.slots, _t(self.k, "bf16"), _t(self.v, "bf16"), bits, gs)
        self.cache = cache
        self.args = (_t(self.q, dt), cache, torch.tensor(self.table).to(DEV), torch.tensor(self.lens).to(DEV), bits, gs)

    def run(self, **kw):
        lse = torch.full(self.q.shape[:2], 123.0, device=DEV)
        out = torch.full(self.q.shape, float("nan"), dtype=DT[self.dt], device=DEV)
        assert gwb.attn_decode(*self.args, out=out, lse=lse, **kw) is out
        return out, lse

    def oracle(self, scale=None):
        s = np.float64(np.float32(1.0 / self.D ** 0.5 if scale is None else scale))
        return S.attn_decode(self.q, self.cache.cpu().numpy(), self.table, self.lens, self.bits, self.gs, self.page, s,
                             self.dt == "fp16")

    def check(self, got=None, scale=None, **kw):
        out, lse = got or self.run(scale=scale, **kw)
        ref = self.oracle(scale)
        _compare(_np(out), _np(lse), *ref)


def _compare(out, lse, ref, ref_lse, bound, lse_bound):
    err = np.abs(out - ref)
    assert np.isfinite(out).all()
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), f"off by {err[worst]:.3e} at {worst}, bound {bound[worst]:.3e}, value {ref[worst]:.3e}"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    # The log-sum-exp is off by no more than the largest score error, and a score's error scales with the
    # sum of the magnitudes it adds (q spread 30: 1e3 and more), not with the log-sum-exp itself, which those
    # terms may cancel to: the bound is the oracle's, from the same e_t as the outputs'.
    assert np.all(np.abs(lse[~empty] - ref_lse[~empty]) <= lse_bound[~empty])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,D,gs", LAYOUTS)
def test_attention_layouts(bits, D, gs, dt):
    lens = [0, 1, 15, 16, 17, 64, 100, 333]
    Batch(lens, 2, 4, D, bits, gs, 16 if gs == 32 else 64, dt, seed=bits + D + gs).check()


@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 9, 12, 16, 17, 33])
@pytest.mark.parametrize("D", [128, 256])
def test_attention_shared_heads(G, D):
    Batch([70, 5, 0, 130], 2, G, D, 4 if G % 2 else 8, 64, 32, "bf16", seed=G).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 4096])
def test_attention_page_sizes(page):
    Batch([page - 1, page, page + 1, 3 * page + 5 if page < 1000 else 7], 1, 4, 64, 4, 64, page, "bf16", seed=page).check()


@pytest.mark.parametrize("H,lens", [(1, [20000]), (3, [9000, 1, 0, 4097]), (8, [2500]), (1, [1] * 300),
                                    (2, [0] * 140 + [777] + [0] * 140 + [33]), (1, [0, 0, 0])])
def test_attention_long_ragged_and_wide_batches(H, lens):
    """Sequences cut over many shares, and shares that hold many sequences."""
    Batch(lens, H, 4, 128, 4, 64, 64, "bf16", seed=len(lens) + H).check()
    Batch(lens[:40], H, 2, 64, 8, 32, 16, "fp16", seed=len(lens)).check()


@pytest.mark.parametrize("B,H,G,D,bits,gs,page,most", [
    (3, 2, 4, 128, 4, 64, 16, 512),        # a CTA a pair
    (1, 1, 1, 64, 8, 32, 512, 512),        # one pair
    (150, 8, 2, 64, 4, 32, 16, 96),        # a warp a pair, a last CTA with idle warps
    (37, 16, 20, 128, 8, 64, 32, 128),     # the same with three chunks of heads
    (90, 7, 9, 256, 4, 128, 64, 64),
    (230, 8, 1, 64, 4, 64, 128, 1500),     # a CTA a pair, many pairs of middling length
])
def test_attention_uncut_pairs(B, H, G, D, bits, gs, page, most):
    """Short tables go a pair a CTA or a pair a warp; rows are empty, of one token, full and between."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, most + 1, B)
    lens[: min(B, 3)] = [most, 0, 1][: min(B, 3)]
    if B > 100:
        lens[rng.permutation(B)[: B // 2]] %= 40      # (keeps the oracle quick)
    b = Batch(lens, H, G, D, bits, gs, page, "bf16", seed=B)
    first = b.run()
    b.check(first)
    again = b.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    b.lens[:] = 0                                      # nothing but empty rows
    b.args[3].zero_()
    b.check()
    gwb.check_device_error()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("kw", [dict(q_spread=30.0), dict(k_spread=20.0), dict(v_spread=1e-3), dict(v_spread=300.0),
                                dict(v_shift=50.0), dict(k_spread=0.0, v_spread=0.0), dict(q_spread=0.0)],
                         ids=["peaked", "wide keys", "small values", "large values", "shifted values", "zeros", "zero query"])
def test_attention_value_ranges(kw, dt):
    Batch([500, 40, 1], 2, 4, 128, 4, 32, 64, dt, seed=3, **kw).check()
    Batch([500, 40, 1], 2, 4, 128, 8, 128, 64, dt, seed=4, **kw).check()


def test_attention_values_far_outside_fp16():
    """bf16 caches hold 1e+-20: the values' powers of two are kept aside."""
    for spread in (1e20, 1e-20):
        Batch([300, 17], 1, 8, 64, 8, 32, 32, "bf16", seed=8, v_spread=spread).check()
    # a late token whose values dwarf the earlier ones, and one whose score does
    b = Batch([700], 1, 4, 128, 4, 64, 64, "bf16", seed=9)
    big = torch.full((1, 1, 128), 3e4, dtype=torch.bfloat16, device=DEV)
    big[:, :, ::3] = -1e4
    gwb.kv_write(b.cache, b.slots[650:651], torch.zeros_like(big), big, 4, 64)
    b.check()
    b = Batch([700], 1, 4, 128, 4, 64, 64, "bf16", seed=10)
    gwb.kv_write(b.cache, b.slots[688:689], 40 * b.args[0][:, :1].contiguous(), big, 4, 64)
    b.check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 0.01])
def test_attention_scales(scale):
    Batch([200, 3], 2, 4, 64, 8, 64, 16, "bf16", seed=6).check(scale=scale)


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("lens,dt,bits", [([40, 700, 3], "bf16", 4), ([40, 700, 3], "fp16", 8), ([40, 300, 3], "bf16", 8),
                                          ([40, 300, 3], "fp16", 4)])
def test_attention_rows_that_are_not_finite_stay_among_themselves(lens, dt, bits, value):
    """In a sequence: a key makes its kv head's rows NaN, a value its group of columns.  Behind the end: nothing."""
    H, G, D, gs = 2, 4, 128, 32
    b = Batch(lens, H, G, D, bits, gs, 64, dt, seed=21)
    good, good_lse = b.run()
    k, v = _t(b.k, "bf16"), _t(b.v, "bf16")
    for place in (0, lens[1] // 2, lens[1] - 1):
        i = lens[0] + place                            # a token of sequence 1
        bad = k[i:i + 1].clone()
        bad[0, 1, 70] = float(value)
        gwb.kv_write(b.cache, b.slots[i:i + 1], bad, v[i:i + 1], bits, gs)
        out, lse = b.run()
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[1, G:] = True
        assert torch.equal(torch.isnan(out), hit) and torch.equal(out[~hit], good[~hit])
        assert torch.equal(torch.isnan(lse), hit[..., 0]) and torch.equal(lse[~hit[..., 0]], good_lse[~hit[..., 0]])
        bad = v[i:i + 1].clone()
        bad[0, 0, 33] = float(value)
        gwb.kv_write(b.cache, b.slots[i:i + 1], k[i:i + 1], bad, bits, gs)
        out, lse = b.run()
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[1, :G, gs:2 * gs] = True
        assert torch.equal(torch.isnan(out), hit) and torch.equal(out[~hit], good[~hit]) and torch.equal(lse, good_lse)
        gwb.kv_write(b.cache, b.slots[i:i + 1], k[i:i + 1], v[i:i + 1], bits, gs)
    # the row behind a sequence's last, in its last page
    slot = b.slots[lens[0] - 1:lens[0]] + 1
    both = torch.full((1, H, D), float(value), dtype=torch.bfloat16, device=DEV)
    gwb.kv_write(b.cache, slot, both, both, bits, gs)
    out, lse = b.run()
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


def test_attention_strided_queries_tables_and_given_workspace():
    b = Batch([90, 0, 257], 2, 4, 64, 8, 32, 32, "fp16", seed=12)
    q, cache, table, lens, bits, gs = b.args
    wide = torch.full((3, 20, 64), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, :8] = q
    tw = torch.full((3, table.shape[1] + 5), 1 << 30, dtype=torch.int32, device=DEV)
    tw[:, 1:1 + table.shape[1]] = table
    lens_odd = torch.cat([lens[:1], lens])[1:]        # 4-byte aligned only
    ws = torch.randint(0, 256, (gwb.attn_decode_workspace(8, 2, 64),), dtype=torch.uint8, device=DEV)
    ref = b.run()
    got_lse = torch.empty(3, 8, device=DEV)
    got = gwb.attn_decode(wide[:, :8], cache, tw[:, 1:1 + table.shape[1]], lens_odd, bits, gs, lse=got_lse, workspace=ws)
    assert torch.equal(got, ref[0]) and torch.equal(got_lse, ref[1])
    assert torch.equal(gwb.attn_decode(*b.args), ref[0])          # without lse
    gwb.check_device_error()


def test_attention_bad_pages_and_lengths_are_left_out_and_reported():
    b = Batch([64, 100, 48], 2, 4, 64, 4, 32, 16, "bf16", seed=13)
    q, cache, table, lens, bits, gs = b.args
    good = b.run()
    gwb.check_device_error()
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        b.table[1, 2] = bad                           # tokens 32 .. 47 of sequence 1
        table.copy_(torch.tensor(b.table))
        got = b.run()
        with pytest.raises(gwb.GwbError, match="INVALID_ARG"):
            gwb.check_device_error()
        b.check(got)
        for i in (0, 2):
            assert torch.equal(got[0][i], good[0][i])
    # every page of a sequence is bad: an empty row
    b.table[1, :] = -7
    table.copy_(torch.tensor(b.table))
    got = b.run()
    with pytest.raises(gwb.GwbError, match="INVALID_ARG"):
        gwb.check_device_error()
    assert not got[0][1].any() and torch.isneginf(got[1][1]).all()


def test_attention_negative_lengths_are_empty_rows():
    b = Batch([64, 100, 48], 2, 4, 64, 4, 32, 16, "bf16", seed=13)
    b.lens[2] = -4
    b.args[3].copy_(torch.tensor(b.lens))
    b.check()
    gwb.check_device_error()


def test_attention_length_beyond_the_table():
    b = Batch([64, 30], 1, 2, 64, 4, 32, 16, "bf16", seed=14)
    ref = b.run()
    b.args[3].copy_(torch.tensor(np.array([2 ** 31 - 1, 30], dtype=np.int32)))
    got = b.run()
    with pytest.raises(gwb.GwbError, match="INVALID_ARG"):
        gwb.check_device_error()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_attention_cache_offsets_beyond_32_bits():
    page, H, D, bits, gs = 256, 8, 128, 8, 64
    block = gwb.kv_block_bytes(page, D, bits, gs)
    pages = (5 << 30) // (H * block) + 1
    cache = torch.empty(pages, H, block, dtype=torch.uint8, device=DEV)
    assert cache.numel() > 5 << 30
    rng = np.random.default_rng(15)
    ids = np.array([[pages - 1, 0, pages - 2]], dtype=np.int32)
    n = 2 * page + 100
    t = np.arange(n)
    slots = ids[0][t // page].astype(np.int64) * page + t % page
    k, v, q = (_rand(rng, s, "bf16") for s in ((n, H, D), (n, H, D), (1, 4 * H, D)))
    gwb.kv_write(cache, torch.tensor(slots).to(DEV), _t(k, "bf16"), _t(v, "bf16"), bits, gs)
    kr, _ = gwb.kv_read(cache, torch.tensor(slots).to(DEV), D, bits, gs)
    small = torch.cat([cache[-2:], cache[:1]])        # pages - 2, pages - 1, 0
    ids_small = np.array([[1, 2, 0]], dtype=np.int32)
    lse = torch.empty(1, 4 * H, device=DEV)
    out = gwb.attn_decode(_t(q, "bf16"), cache, torch.tensor(ids).to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                          bits, gs, lse=lse)
    small = small.cpu().numpy()
    at = ids_small[0][t // page].astype(np.int64) * page + t % page
    assert np.array_equal(_np(kr), S.bf16(S.read_rows(small, at, "k", bits, D, gs, page).astype(np.float32)))
    _compare(_np(out), _np(lse), *S.attn_decode(q, small, ids_small, [n], bits, gs, page, np.float64(np.float32(D ** -0.5)),
                                                False))


def test_attention_is_reproducible():
    b = Batch([3000, 17, 5000, 900], 2, 8, 128, 4, 64, 64, "bf16", seed=16)
    first = b.run()
    for _ in range(3):
        again = b.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_captured_step_follows_lengths_and_cache():
    """Write, attend and norm captured once; replays see new tokens, slots and lengths in the same buffers."""
    b = Batch([100, 0, 31, 2000], 2, 4, 64, 8, 32, 16, "bf16", seed=17)
    q, cache, table, lens, bits, gs = b.args
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    v, slots = torch.zeros_like(k), torch.full((4,), -1, dtype=torch.int64, device=DEV)
    w = torch.ones(8 * 64, dtype=torch.bfloat16, device=DEV)

    def step():
        gwb.kv_write(cache, slots, k, v, bits, gs)
        out = gwb.attn_decode(q, cache, table, lens, bits, gs)
        return (out, *gwb.rmsnorm_quant_i8(out.view(4, -1), w, 1e-5))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    rng = np.random.default_rng(18)
    for n in ([100, 0, 31, 2000], [101, 0, 32, 1999], [64, 0, 1, 16]):
        n = np.array(n, dtype=np.int32)
        at = np.where(n > 0, n - 1, 0)
        new = b.table[np.arange(4), at // 16].astype(np.int64) * 16 + at % 16
        slots.copy_(torch.tensor(np.where(n > 0, new, -1)))
        lens.copy_(torch.tensor(n))
        k.copy_(_t(_rand(rng, (4, 2, 64), "bf16"), "bf16"))
        v.copy_(_t(_rand(rng, (4, 2, 64), "bf16"), "bf16"))
        g.replay()
        torch.cuda.synchronize()
        graph = [t.clone() for t in got[:3]]
        eager = step()
        for a, e in zip(graph, eager):
            assert torch.equal(a, e)
        ref, _, bound, _ = S.attn_decode(b.q, cache.cpu().numpy(), b.table, n, bits, gs, 16, np.float64(np.float32(0.125)), False)
        assert (np.abs(_np(graph[0]) - ref) <= bound).all()
    gwb.check_device_error()


def test_a_first_call_may_be_a_captured_one():
    """A fresh process whose first calls of the library are made under stream capture."""
    code = """
import torch, group_wise_bit_b200 as gwb
d = "cuda"
cache = gwb.kv_cache(40, 2, 128, 32, 4, 64)
k = torch.randn(3, 2, 128, device=d).bfloat16()
slots = torch.tensor([0, 32, 1200], device=d)
table = torch.arange(40, dtype=torch.int32, device=d)[None].repeat(3, 1).contiguous()
lens = torch.tensor([1, 33, 1201], dtype=torch.int32, device=d)
q = torch.randn(3, 8, 128, device=d).bfloat16()
w = torch.ones(1024, dtype=torch.bfloat16, device=d)
def step():
    gwb.kv_write(cache, slots, k, k, 4, 64)
    a = gwb.attn_decode(q, cache, table, lens, 4, 64)
    b = gwb.attn_decode(q, cache, table[:, :4], lens.clamp(max=128), 4, 64)
    return a, b, *gwb.rmsnorm_quant_i8(a.view(3, -1), w, 1e-5), *gwb.kv_read(cache, slots, 128, 4, 64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
for x, y in zip(got, step()):
    assert (x is None and y is None) or torch.equal(x, y)
gwb.check_device_error()
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_calls_on_two_streams_and_two_graphs_do_not_share_a_workspace():
    bs = [Batch([4000, 300], 2, 8, 128, 4, 64, 64, "bf16", seed=20 + i) for i in range(2)]
    refs = [b.run()[0].clone() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    graphs, outs = [], []
    for b, s in zip(bs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(gwb.attn_decode(*b.args))
        graphs.append(g)
    for _ in range(20):
        eager = []
        for b, s, g in zip(bs, streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
                eager.append(gwb.attn_decode(*b.args))
        torch.cuda.synchronize()
        for o, e, r in zip(outs, eager, refs):
            assert torch.equal(o, r) and torch.equal(e, r)


def test_a_long_chain_without_synchronisation():
    """Back-to-back dependent calls on one workspace (each launch may start before the one in front has ended)."""
    b = Batch([2600, 40, 777], 2, 4, 64, 4, 32, 16, "bf16", seed=25)
    ws = torch.empty(gwb.attn_decode_workspace(8, 2, 64), dtype=torch.uint8, device=DEV)
    q, cache, table, lens, bits, gs = b.args
    ref = [q]
    for _ in range(6):
        ref.append(gwb.attn_decode(ref[-1], cache, table, lens, bits, gs))
        torch.cuda.synchronize()
    for _ in range(10):
        x = q
        for i in range(6):
            x = gwb.attn_decode(x, cache, table, lens, bits, gs, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(x, ref[-1])


# ------------------------------------------------------------------ a decoder layer's attention half, as it is used
def test_a_decode_step_through_the_layer():
    """norm -> W8A8 q/k/v projection -> cache write -> attention -> W4A8 output projection -> norm with residual,
    every stage against fp64 on what the stage in front really produced."""
    rng = np.random.default_rng(30)
    B, E, H, G, D, page, bits, gs = 6, 1024, 2, 4, 128, 32, 4, 64
    HQ = H * G
    past = Batch([50, 1, 333, 64, 0, 127], H, G, D, bits, gs, page, "bf16", seed=31)
    x, res = _rand(rng, (B, E), "bf16"), _rand(rng, (B, E), "bf16")
    w1, w2 = S.bf16(1 + 0.1 * rng.standard_normal(E)), S.bf16(1 + 0.1 * rng.standard_normal(E))
    wqkv = torch.tensor(0.03 * rng.standard_normal(((HQ + 2 * H) * D, E)), dtype=torch.float32, device=DEV)
    wo = torch.tensor(0.03 * rng.standard_normal((E, HQ * D)), dtype=torch.float32, device=DEV)
    qkv_w, o_w = gwb.qpack_sym_i8(wqkv), gwb.qpack_sym_i4(wo)

    qx, sx, h = gwb.rmsnorm_quant_i8(_t(x, "bf16"), _t(w1, "bf16"), 1e-5, residual=_t(res, "bf16"))
    qkv, _ = gwb.gemm_i8i8(qx, sx, *qkv_w)
    q = qkv[:, :HQ * D].view(B, HQ, D)
    k, v = qkv[:, HQ * D:(HQ + H) * D].view(B, H, D), qkv[:, (HQ + H) * D:].view(B, H, D)
    # room for one more token each
    table = np.concatenate([past.table, np.zeros((B, 1), dtype=np.int32)], 1)
    free = np.setdiff1d(np.arange(past.cache.shape[0] + B), table[:, :-1])[-B:]
    cache = torch.cat([past.cache, torch.zeros(B, *past.cache.shape[1:], dtype=torch.uint8, device=DEV)])
    lens = past.lens + 1
    for b in range(B):
        if past.lens[b] % page == 0:
            table[b, past.lens[b] // page] = free[b]
    slots = table[np.arange(B), past.lens // page].astype(np.int64) * page + past.lens % page
    gwb.kv_write(cache, torch.tensor(slots).to(DEV), k, v, bits, gs)
    a = gwb.attn_decode(q, cache, torch.tensor(table).to(DEV), torch.tensor(lens).to(DEV), bits, gs)
    qa, sa = gwb.quant_per_token_i8(a.view(B, -1))
    o, _ = gwb.gemm_i8i4(qa, sa, *o_w)
    q2, s2, h2 = gwb.rmsnorm_quant_i8(o, _t(w2, "bf16"), 1e-5, residual=h)
    torch.cuda.synchronize()
    gwb.check_device_error()

    q_o, s_o, h_o = S.rmsnorm_quant_i8(x, res, w1, 1e-5, False)
    assert np.array_equal(qx.cpu().numpy(), q_o) and np.array_equal(sx.cpu().numpy(), s_o)
    wv = qkv_w[0].double().cpu().numpy() * qkv_w[1].double().cpu().numpy()[:, None]
    ref = (q_o * s_o[:, None].astype(np.float64)) @ wv.T
    assert np.all(np.abs(_np(qkv) - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + 1e-30)   # exact int32, one rounding (and two fp32 products)
    cache_np = past.cache.cpu().numpy()
    cache_np = np.concatenate([cache_np, np.zeros((B, *cache_np.shape[1:]), dtype=np.uint8)])
    S.write_rows(cache_np, slots, _np(k), "k", bits, gs, page)
    S.write_rows(cache_np, slots, _np(v), "v", bits, gs, page)
    assert np.array_equal(cache.cpu().numpy(), cache_np)
    ref, _, bound, _ = S.attn_decode(_np(q), cache_np, table, lens, bits, gs, page, np.float64(np.float32(D ** -0.5)), False)
    assert (np.abs(_np(a) - ref) <= bound).all()
    q_o, s_o, h_o = S.rmsnorm_quant_i8(_np(o), _np(h), w2, 1e-5, False)
    assert np.array_equal(q2.cpu().numpy(), q_o) and np.array_equal(s2.cpu().numpy(), s_o) and np.array_equal(_np(h2), h_o)


# ------------------------------------------------------------------ what fp16 outputs promise
@pytest.mark.parametrize("values", ["symmetric", "small minimum", "outliers", "shifted"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,D,gs,G", [(8, 64, 32, 4), (8, 128, 64, 3), (8, 128, 128, 12), (8, 256, 64, 8)])
def test_attention_weights_and_values_where_scores_are_exact(bits, D, gs, G, dt, values):
    """Scores without an error of their own, few tokens: what is left is how weights, their products with the value
    scales and the centred biases are rounded (oracle.serving.attn_decode, exact_scores)."""
    _exact_scores([1, 2, 3, 5, 2, 3], 2, G, D, bits, gs, dt, values, 1.0)


@pytest.mark.parametrize("values", ["symmetric", "small minimum", "outliers", "shifted"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,D,gs,G", [(4, 64, 64, 4), (4, 128, 32, 9), (4, 256, 128, 2), (8, 128, 32, 8), (8, 64, 64, 16)])
def test_attention_values_under_a_zero_query(bits, D, gs, G, dt, values):
    """Equal weights: the mean of the rows, exact but for the biases, the products with the scales and the output."""
    _exact_scores([1, 500, 2, 17, 700], 2, G, D, bits, gs, dt, values, 0.0)


def _exact_scores(lens, H, G, D, bits, gs, dt, values, q0):
    rng = np.random.default_rng(1000 * bits + D + gs + G)
    page = 32
    need = [-(-n // page) for n in lens]
    table = np.zeros((len(lens), max(need)), dtype=np.int32)
    order, at, slots = rng.permutation(sum(need)), 0, []
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        t = np.arange(lens[b])
        slots.append(table[b][t // page].astype(np.int64) * page + t % page)
    slots = np.concatenate(slots)
    k, v = S.exact_score_rows(rng, len(slots), H, D, gs, values)
    q = np.zeros((len(lens), H * G, D))
    q[..., 0] = q0 * 2.0 ** -rng.integers(0, 2, q.shape[:2])
    cache = gwb.kv_cache(sum(need), H, D, page, bits, gs)
    gwb.kv_write(cache, torch.tensor(slots).to(DEV), _t(k, "bf16"), _t(v, "bf16"), bits, gs)
    args = (_t(q, dt), cache, torch.tensor(table).to(DEV), torch.tensor(np.array(lens, dtype=np.int32)).to(DEV), bits, gs)
    lse = torch.empty(q.shape[:2], device=DEV)
    out = gwb.attn_decode(*args, scale=1.0, lse=lse)
    ref = S.attn_decode(q, cache.cpu().numpy(), table, lens, bits, gs, page, 1.0, dt == "fp16", exact_scores=True)
    _compare(_np(out), _np(lse), *ref)


# ------------------------------------------------------------------ queries and scores at the end of fp32's range
@pytest.mark.parametrize("D,bits,G", [(64, 8, 4), (128, 8, 9), (256, 8, 2)])
@pytest.mark.parametrize("lens", [[3, 40, 300], [700, 1, 0, 90]])
def test_attention_of_very_large_queries(lens, D, bits, G):
    """Queries times 2^117 over keys over 2^117 are the same scores, bit for bit."""
    rng = np.random.default_rng(D)
    k, v = S.exact_score_rows(rng, sum(lens), 1, D, 64, "symmetric")
    q = np.zeros((len(lens), G, D))
    q[..., 0] = 2.0 ** -rng.integers(0, 3, q.shape[:2])
    got = []
    for up in (0, 117):
        args = _one_head_batch(k * 2.0 ** -up, v, q * 2.0 ** up, lens, bits, 64)
        lse = torch.empty(q.shape[:2], device=DEV)
        got.append((gwb.attn_decode(*args, lse=lse), lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][0]).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("lens", [[3, 40, 300], [700, 1, 0, 90]])
def test_attention_scores_beyond_fp32_are_not_silently_zeros(lens, sign):
    """Every score overflows: NaN rows and log-sum-exps, not the zeros of an empty row."""
    rng = np.random.default_rng(3)
    k, v = S.exact_score_rows(rng, sum(lens), 1, 128, 64, "symmetric")
    k[..., 0] = np.maximum(k[..., 0], 1 / 64)
    q = np.zeros((len(lens), 4, 128))
    q[..., 0] = sign * 2.0 ** 100
    lse = torch.empty(q.shape[:2], device=DEV)
    out = gwb.attn_decode(*_one_head_batch(k * 2.0 ** 40, v, q, lens, 8, 64), lse=lse)
    full = torch.tensor([n > 0 for n in lens], device=DEV)
    assert torch.isnan(out[full]).all() and torch.isnan(lse[full]).all()
    assert not out[~full].any() and torch.isneginf(lse[~full]).all()


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("lens,dt,bits,G", [([40, 700, 3], "bf16", 4, 4), ([40, 300, 3], "fp16", 8, 4),
                                            ([40, 700, 3], "fp16", 4, 12), ([40, 300, 3], "bf16", 8, 2)])
def test_attention_queries_that_are_not_finite_make_their_rows_nan(lens, dt, bits, G, value):
    b = Batch(lens, 2, G, 128, bits, 64, 64, dt, seed=22)
    good, good_lse = b.run()
    for i, h in ((1, 0), (0, G), (2, 2 * G - 1)):
        b.args[0][i, h, 37] = float(value)
    out, lse = b.run()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[1, 0] = hit[0, G] = hit[2, 2 * G - 1] = True
    assert torch.equal(torch.isnan(lse), hit) and torch.equal(torch.isnan(out), hit[..., None].expand_as(out))
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])


def _one_head_batch(k, v, q, lens, bits, gs, page=32):
    """Arguments of attn_decode for rows k, v [sum(lens), 1, D] in consecutive pages, bf16."""
    need = [-(-n // page) for n in lens]
    table = np.zeros((len(lens), max(need)), dtype=np.int32)
    at, slots = 0, []
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        slots.append(at * page + np.arange(lens[b]))
        at += n
    cache = gwb.kv_cache(sum(need), 1, q.shape[2], page, bits, gs)
    gwb.kv_write(cache, torch.tensor(np.concatenate(slots)).to(DEV), _t(k, "bf16"), _t(v, "bf16"), bits, gs)
    return (_t(q, "bf16"), cache, torch.tensor(table).to(DEV), torch.tensor(np.array(lens, dtype=np.int32)).to(DEV), bits, gs)


# ------------------------------------------------------------------ rows of zeros without eps
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K", [(4, 1), (4, 77), (5, 4096), (700, 520), (3, 40000)])
def test_norm_of_a_zero_row_with_eps_zero(M, K, dt):
    """Scale 0 and codes 0, as with any other eps; the rows beside it keep their results."""
    rng = np.random.default_rng(K)
    x, w = _rand(rng, (M, K), dt), S.rnd(1 + 0.1 * rng.standard_normal(K), dt == "fp16")
    x[0], x[2] = 0.0, -0.0
    r = _rand(rng, (M, K), dt)
    r[0], r[2] = 0.0, 0.0
    r[1] = -x[1]                                      # a sum of zeros
    for res in (None, r):
        q, s, h = gwb.rmsnorm_quant_i8(_t(x, dt), _t(w, dt), 0.0, residual=None if res is None else _t(res, dt))
        zero = [0, 2] if res is None else [0, 1, 2]
        assert not s[zero].any() and not q[zero].any()
    _check_norm(x, None, w, dt, eps=0.0)
    _check_norm(x, r, w, dt, eps=0.0)


def test_attention_refuses_a_workspace_that_is_no_tensor():
    b = Batch([3], 1, 1, 64, 4, 32, 16, "bf16")
    for bad, error in ((1 << 20, TypeError), (torch.empty(1 << 20, device=DEV), TypeError),
                       (torch.empty(1 << 20, dtype=torch.uint8), ValueError)):
        with pytest.raises(error, match="workspace"):
            gwb.attn_decode(*b.args, workspace=bad)


# ------------------------------------------------------------------ every instance with 16-head tiles
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,D,gs", [x for x in LAYOUTS if x[1] <= 128])
def test_attention_layouts_with_more_than_eight_heads(bits, D, gs, dt):
    """Groups of 9 to 16 query heads a kv head share a tile of 16; 12 and 20 leave rows of it empty or take two."""
    seed = bits + D + gs
    Batch([700, 1, 0, 33, 16], 2, 12, D, bits, gs, 16, dt, seed=seed).check()          # cut
    Batch([0, 1, 31, 300], 1, 16, D, bits, gs, 64, dt, seed=seed).check()              # a CTA a pair
    lens = np.random.default_rng(seed).integers(0, 40, 260)
    b = Batch(lens, 1, 20, D, bits, gs, 32, dt, seed=seed)                             # a warp a pair
    b.check()
    gwb.check_device_error()


@pytest.mark.parametrize("bits,D,gs", [x for x in LAYOUTS if x[1] <= 128])
def test_sixteen_head_tiles_round_as_eight_head_ones(bits, D, gs):
    """fp16, exact scores: the bound of the roundings alone (see above) on every 16-head instance."""
    for q0 in ((1.0, 0.0) if bits == 8 else (0.0,)):
        _exact_scores([1, 2, 3, 5], 1, 16, D, bits, gs, "fp16", "outliers", q0)
        _exact_scores([600, 3], 1, 9, D, bits, gs, "fp16", "small minimum", q0)
