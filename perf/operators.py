"""What is measured of the serving operators: their cases, plain forms and definitions.

Three operators that stand around the low-bit linear layers of a decoder:

- ``norm``: root-mean-square norm with the residual's addition and an int8 output with one scale
  a token, the activations of the W8A8 and W4A8 products;
- ``store`` / ``load``: quantising keys and values into a paged cache as they are written, and
  reading rows of the cache back;
- ``attend``: attention of one new token a sequence over that paged, quantised cache.

The cache is a uint8 tensor [pages, kv heads, block].  A block holds page_size tokens of one head
as page_size / 16 granules of 16 tokens; a granule is, in this order,

- key codes, 32-bit words [words/row/(4 VW)][16 rows][4][VW], VW = min(4, words a row / 4): row
  rho(t) = 2 (t // 4) + t % 2 + 8 (t // 2 % 2) of token t holds its MLX-packed words, word
  w = 4 (VW a + v) + c at [a][rho][c][v];
- value codes, 16-bit halves [halves a row / 16][8][4][2][2][2]: half h = 16 a + 8 j + r of the
  MLX-packed row of token t = 4 c + 2 y + z at [a][r][c][j][y][z];
- key scales and biases, bf16 [16 rows][groups][2];
- value scales, bf16 [groups][16 tokens], then value biases, bf16 [groups][16 tokens].
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5


def listed():
    return [
        # one decode step of one user: the norm in front of a layer's projections, latency alone
        dict(name="norm_one_token", op="norm", M=1, K=4096, dtype="bf16", residual=True),
        # a decode batch in fp16, a width that is no multiple of a vector's elements, first norm (no residual)
        dict(name="norm_odd_width", op="norm", M=77, K=5003, dtype="fp16", residual=False),
        # a long prompt batch
        dict(name="norm_prompt", op="norm", M=16384, K=4096, dtype="bf16", residual=True),
        # a decode step of a batch writes one token a sequence; keys and values are slices of a fused projection
        dict(name="store_decode", op="store", T=64, H=8, Hq=32, D=128, page=64, bits=4, gs=64, dtype="bf16", pad=0),
        # a prompt chunk, 8-bit cache, the projection's last rows are padding
        dict(name="store_prompt", op="store", T=8192, H=8, Hq=32, D=128, page=32, bits=8, gs=64, dtype="bf16", pad=37),
        # a context read back for a path that wants dense keys and values, fp16, small heads and pages
        dict(name="load_context", op="load", T=20011, H=4, D=64, page=16, bits=4, gs=32, dtype="fp16"),
        dict(name="load_short", op="load", T=300, H=8, D=128, page=64, bits=8, gs=128, dtype="bf16"),
        # a chat's first answers: one short sequence
        dict(name="attend_short", op="attend", B=1, L=100, H=8, G=4, D=128, page=64, bits=4, gs=64, dtype="bf16", lse=False),
        # an ordinary serving batch: ragged lengths, empty rows among them
        dict(name="attend_batch", op="attend", B=32, L=4096, H=8, G=4, D=128, page=64, bits=4, gs=64, dtype="bf16", lse=False),
        # one user with a very long context
        dict(name="attend_long", op="attend", B=1, L=131072, H=8, G=8, D=128, page=64, bits=8, gs=64, dtype="bf16", lse=True),
        # few wide heads shared by many queries, small groups and pages, fp16
        dict(name="attend_shared", op="attend", B=9, L=5000, H=1, G=12, D=256, page=16, bits=8, gs=32, dtype="fp16", lse=True),
        # a full machine: many sequences of thousands of tokens
        dict(name="attend_full", op="attend", B=64, L=8192, H=8, G=8, D=128, page=128, bits=4, gs=64, dtype="bf16", lse=False),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["norm", "store", "load", "attend", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm":
        K = log(64, 16384)
        if rng.random() < 0.7:
            K = max(64, K // 64 * 64)
        M = log(1, max(2, min(16384, 60_000_000 // K)))
        return dict(op=op, M=M, K=K, dtype=dtype, residual=rng.random() < 0.7)
    bits = rng.choice([4, 8])
    D = rng.choice([64, 128, 128, 256])
    gs = rng.choice([g for g in (32, 64, 128) if g <= D])
    page = rng.choice([16, 32, 64, 128, 256])
    H = rng.choice([1, 2, 4, 5, 8, 16])
    if op in ("store", "load"):
        T = log(1, max(2, 8_000_000 // (H * D)))
        if op == "load":
            return dict(op=op, T=T, H=H, D=D, page=page, bits=bits, gs=gs, dtype=dtype)
        return dict(op=op, T=T, H=H, Hq=H * rng.choice([1, 4, 7]), D=D, page=page, bits=bits, gs=gs, dtype=dtype,
                    pad=rng.choice([0, 0, min(T, 5)]))
    B = log(1, 256)
    L = log(1, min(131072, 400_000_000 // (B * H * D)))
    return dict(op=op, B=B, L=L, H=H, G=rng.choice([1, 2, 4, 5, 8, 12, 16, 20]), D=D, page=page, bits=bits, gs=gs,
                dtype=dtype, lse=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _granule_parts(D, bits, gs):
    """Bytes of a granule's key codes, value codes, key scales and biases, value scales and biases."""
    return [2 * D * bits, 2 * D * bits, 64 * (D // gs), 64 * (D // gs)]


def _cache(pages, H, D, page, bits, gs, g, keys):
    """A cache whose rows are independent draws: codes around the middle, scales of a spread of ranges."""
    kc, vc, km, vm = _granule_parts(D, bits, gs)
    n = pages * H * (page // 16)
    cache = torch.empty(n, kc + vc + km + vm, dtype=torch.uint8, device="cuda")
    top = (1 << bits) - 1
    for lo in range(0, n, 1 << 15):                                  # codes, a slice at a time
        m = min(n, lo + (1 << 15)) - lo
        c = torch.randn(m, (kc + vc) * 8 // bits, device="cuda", generator=g, dtype=torch.float16)
        c = c.mul_(top / 5.2).add_(top / 2).round_().clamp_(0, top).to(torch.uint8)
        cache[lo:lo + m, :kc + vc] = c if bits == 8 else c[:, ::2] | (c[:, 1::2] << 4)
    for lo, width, pairs in ((kc + vc, km // 4, True), (kc + vc + km, vm // 4, False)):
        spread = torch.randn(n, width, device="cuda", generator=g).mul_(0.25).exp_()
        scale = (spread * (5.2 * (keys if pairs else 1.0) / top)).to(torch.bfloat16)
        bias = (spread * -2.6 * (keys if pairs else 1.0) * (1 + 0.1 * torch.randn(n, width, device="cuda", generator=g)))
        bias = bias.to(torch.bfloat16)
        meta = torch.stack([scale, bias], 2) if pairs else torch.stack([scale, bias], 1)
        cache[:, lo:lo + 4 * width] = meta.reshape(n, -1).view(torch.uint8)
    return cache.view(pages, H, -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case)
    if case["op"] == "norm":
        M, K, dt = case["M"], case["K"], DT[case["dtype"]]
        channel = torch.ones(K, device="cuda")
        channel[torch.randperm(K, device="cuda", generator=g)[:max(1, K // 100)]] = 8.0      # outlier channels
        s["x"] = (torch.randn(M, K, device="cuda", generator=g) * channel).to(dt)
        s["residual"] = (2 * torch.randn(M, K, device="cuda", generator=g)).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(dt)
        return s
    H, D, page, bits, gs, dt = (case[k] for k in ("H", "D", "page", "bits", "gs", "dtype"))
    dt = DT[dt]
    if case["op"] in ("store", "load"):
        T = case["T"]
        pages = -(-T // page) + 3
        table = rng.permutation(pages)[:-(-T // page)]
        at = np.arange(T)
        slots = table[at // page] * page + at % page
        if case["op"] == "store":
            if case["pad"]:
                slots[T - case["pad"]:] = -1
            s["qkv"] = torch.randn(T, (case["Hq"] + 2 * H) * D, device="cuda", generator=g).to(dt)
            s["k"] = s["qkv"][:, case["Hq"] * D:(case["Hq"] + H) * D].view(T, H, D)
            s["v"] = s["qkv"][:, (case["Hq"] + H) * D:].view(T, H, D)
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
        s["cache"] = _cache(pages, H, D, page, bits, gs, g, 2.0)
        return s
    B, L = case["B"], case["L"]
    lens = rng.integers((L + 1) // 2, L + 1, B)
    lens[rng.integers(0, B)] = L
    if B >= 16:
        lens[rng.integers(0, B, B // 16)] = 0                         # rows that wait for a request
        lens[rng.integers(0, B)] = 1
    need = -(-lens // page)
    most = -(-L // page)
    pages = int(need.sum()) + 1
    order = rng.permutation(pages)
    table = np.zeros((B, most), dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["table"] = torch.from_numpy(table).cuda()
    s["q"] = (1.5 * torch.randn(B, H * case["G"], D, device="cuda", generator=g)).to(dt)
    s["cache"] = _cache(pages, H, D, page, bits, gs, g, 1.0)
    return s


# ---------------------------------------------------------------- the plain forms
def _unpack(cache, D, bits, gs):
    """Dense keys and values fp32 [pages, H, page, D] of a cache, by reshaping its parts."""
    P, H, _ = cache.shape
    kc, vc, km, vm = _granule_parts(D, bits, gs)
    gr = cache.reshape(P, H, -1, kc + vc + km + vm)
    n, NG = gr.shape[2], D // gs
    shifts = torch.arange(0, 8, bits, device=cache.device, dtype=torch.uint8)
    codes = lambda b: ((b.unsqueeze(-1) >> shifts) & ((1 << bits) - 1)).flatten(-2)  # noqa: E731
    vw = min(4, D * bits // 128)
    # row 2 a + z + 8 y holds token 4 a + 2 y + z
    k = gr[..., :kc].reshape(P, H, n, -1, 2, 4, 2, 4, vw, 4).permute(0, 1, 2, 5, 4, 6, 3, 8, 7, 9)
    k = codes(k.reshape(P, H, n * 16, -1)).float()
    v = gr[..., kc:kc + vc].reshape(P, H, n, -1, 8, 4, 2, 2, 2, 2).permute(0, 1, 2, 5, 7, 8, 3, 6, 4, 9)
    v = codes(v.reshape(P, H, n * 16, -1)).float()
    m = gr[..., kc + vc:kc + vc + km].contiguous().view(torch.bfloat16).float()
    m = m.reshape(P, H, n, 2, 4, 2, NG, 2).permute(0, 1, 2, 4, 3, 5, 6, 7).reshape(P, H, n * 16, NG, 2)
    k = torch.addcmul(m[..., 1:], k.view(P, H, n * 16, NG, gs), m[..., :1]).flatten(-2)
    m = gr[..., kc + vc + km:].contiguous().view(torch.bfloat16).float()
    m = m.reshape(P, H, n, 2, NG, 16).permute(0, 1, 2, 5, 4, 3).reshape(P, H, n * 16, NG, 2)
    v = torch.addcmul(m[..., 1:], v.view(P, H, n * 16, NG, gs), m[..., :1]).flatten(-2)
    return k, v


def _quantise(x, bits, gs):
    """The values a row's codes stand for: min / max a group, one fp32 rounding a step, bf16 scale and bias."""
    x = x.float().unflatten(-1, (-1, gs))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    top = (1 << bits) - 1
    step = (high - low) / torch.full_like(low, top)     # (a division by a plain number would be a product)
    code = torch.where(step > 0, ((x - low) / step).round().clamp(0, top), 0.0)
    return torch.addcmul(low.bfloat16().float(), code, step.bfloat16().float()).flatten(-2)


def _rows(dense, slots, page):
    """Rows [T, H, D] of a dense cache at slots; a negative slot is a row of zeros."""
    at = slots.clamp(min=0)
    rows = dense[at // page, :, at % page]
    return torch.where((slots >= 0)[:, None, None], rows, 0.0)


def run(s):
    if own:
        return _own(s)
    if s["op"] == "norm":
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        f = h.double()
        r = torch.rsqrt(f.square().mean(1, keepdim=True) + EPS).float()
        y = h.float() * r * s["weight"].float()
        sx = y.abs().amax(1, keepdim=True) / torch.full_like(r, 127)
        codes = torch.where(sx > 0, (y / sx).round().clamp(-127, 127), 0.0)
        out = {"values": (codes * sx).to(h.dtype), "scale": sx[:, 0]}
        if s["residual"] is not None:
            out["residual"] = h
        return out
    if s["op"] == "store":
        keep = (s["slots"] >= 0)[:, None, None]
        return [torch.where(keep, _quantise(x, s["bits"], s["gs"]), 0.0).to(x.dtype) for x in (s["k"], s["v"])]
    if s["op"] == "load":
        used = torch.unique(s["slots"] // s["page"], return_inverse=True)
        k, v = _unpack(s["cache"][used[0]], s["D"], s["bits"], s["gs"])
        at = used[1] * s["page"] + s["slots"] % s["page"]
        return [_rows(x, at, s["page"]).to(DT[s["dtype"]]) for x in (k, v)]
    B, L, H, G, D = (s[k] for k in "BLHGD")
    k, v = _unpack(s["cache"], D, s["bits"], s["gs"])
    k = k[s["table"].long()].transpose(1, 2).flatten(2, 3)                     # [B, H, tokens, D]
    v = v[s["table"].long()].transpose(1, 2).flatten(2, 3)
    q = s["q"].float().view(B, H, G, D)
    scores = (q @ k.transpose(2, 3)) * (1 / math.sqrt(D))
    there = torch.arange(k.shape[2], device=k.device) < s["lens"][:, None]
    scores = scores.masked_fill(~there[:, None, None], -math.inf)
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - top.clamp(min=-3e38))
    total = p.sum(3, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0.0)
    out = out.view(B, H * G, D).to(s["q"].dtype)
    return [out, (top + total.log()).view(B, H * G)] if s["lse"] else out


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import group_wise_bit_b200 as gwb
    if s["op"] == "norm":
        qx, sx, h = gwb.rmsnorm_quant_i8(s["x"], s["weight"], EPS, residual=s["residual"])
        out = {"values": gwb.dequant_per_token_i8(qx, sx, dtype=s["x"].dtype), "scale": sx}
        if s["residual"] is not None:
            out["residual"] = h
        return out
    if s["op"] == "store":
        gwb.kv_write(s["cache"], s["slots"], s["k"], s["v"], s["bits"], s["gs"])
        return list(gwb.kv_read(s["cache"], s["slots"], s["D"], s["bits"], s["gs"], dtype=s["k"].dtype))
    if s["op"] == "load":
        return list(gwb.kv_read(s["cache"], s["slots"], s["D"], s["bits"], s["gs"], dtype=DT[s["dtype"]]))
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if s["lse"] else None
    out = gwb.attn_decode(s["q"], s["cache"], s["table"], s["lens"], s["bits"], s["gs"], lse=lse)
    return [out, lse] if s["lse"] else out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        n = case["M"] * case["K"]
        return {"bytes": n * (2 + 1 + (4 if case["residual"] else 0)) + 2 * case["K"] + 4 * case["M"], "flops": 8 * n}
    row = 2 * (case["D"] * case["bits"] // 8 + 4 * (case["D"] // case["gs"]))     # a token's keys and values of one head
    if case["op"] == "store":     # read, quantise, write; and the rows read back
        n = (case["T"] - case["pad"]) * case["H"]
        return {"bytes": n * (4 * case["D"] + 2 * row) + case["T"] * (case["H"] * 4 * case["D"] + 16),
                "flops": n * 2 * case["D"] * 8}
    if case["op"] == "load":
        n = case["T"] * case["H"]
        return {"bytes": n * (row + 4 * case["D"]) + 8 * case["T"], "flops": 4 * n * case["D"]}
    # lengths are uniform between half of L and L; a sixteenth of the rows is empty where there are many
    B = case["B"]
    tokens = case["L"] + (B - 1) * case["L"] * 0.75 * (15 / 16 if B >= 16 else 1.0)
    heads = case["H"] * case["G"]
    return {"bytes": int(tokens * case["H"] * row + B * heads * 4 * case["D"] + 4 * tokens / case["page"]),
            "flops": int(4 * tokens * heads * case["D"])}


# ---------------------------------------------------------------- the definitions in 64 bits
def _element(cache, page, H, D, bits, gs, slot, head, what):
    """Row [.., D] of keys ("k") or values ("v") at slots and heads, each byte looked up by its offset."""
    kc, vc, km, vm = _granule_parts(D, bits, gs)
    size = kc + vc + km + vm
    flat = cache.reshape(-1)
    t = slot % 16
    base = ((slot // page * H + head) * (page // 16) + slot % page // 16) * size
    d = torch.arange(D, device=cache.device)
    rho = 2 * torch.div(t, 4, rounding_mode="floor") + t % 2 + 8 * (t // 2 % 2)
    grp = d // gs
    if what == "k":
        vw = min(4, D * bits // 128)
        w = d * bits // 32
        c, v, a = w % 4, w // 4 % vw, w // (4 * vw)
        byte = 4 * (((a * 16 + rho) * 4 + c) * vw + v) + d * bits % 32 // 8
        scale = kc + vc + ((rho * (D // gs) + grp) * 2) * 2
        bias = scale + 2
    else:
        h = d * bits // 16
        r, j, a = h % 8, h // 8 % 2, h // 16
        byte = kc + 2 * ((((a * 8 + r) * 4 + t // 4) * 2 + j) * 4 + t % 4) + d * bits % 16 // 8
        scale = kc + vc + km + (grp * 16 + t) * 2
        bias = scale + (D // gs) * 32
    code = (flat[base + byte].to(torch.int64) >> (d * bits % 8)) & ((1 << bits) - 1)
    halves = flat.view(torch.bfloat16)
    return code.double() * halves[torch.div(base + scale, 2, rounding_mode="floor")].double() \
        + halves[torch.div(base + bias, 2, rounding_mode="floor")].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()        # the sum is stored, rounded once
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].double()
        sx = y.abs().amax(1, keepdim=True) / 127
        values = torch.where(sx > 0, torch.round(y / sx) * sx, 0.0)
        out = {"values": values, "scale": sx[:, 0]}
        if s["residual"] is not None:
            out["residual"] = h
        return out
    H, D, page, bits, gs = (case[k] for k in ("H", "D", "page", "bits", "gs"))
    if case["op"] == "store":
        out = []
        for x in (s["k"], s["v"]):
            w = x.double().reshape(case["T"], H, D // gs, gs)
            low, high = w.min(3, keepdim=True)[0], w.max(3, keepdim=True)[0]
            top = 2.0 ** bits - 1
            # the quantiser's definition rounds every step to 32 bits
            r32 = lambda z: z.float().double()  # noqa: E731
            step = r32(r32(high - low) / top)
            code = torch.round(r32(r32(w - low) / torch.where(step == 0, 1.0, step))).clamp(0, top)
            code = torch.where(step == 0, 0.0, code)
            val = code * step.bfloat16().double() + low.bfloat16().double()
            val = val.reshape(case["T"], H, D)
            out.append(torch.where((s["slots"] < 0)[:, None, None], 0.0, val))
        return out
    if case["op"] == "load":
        head = torch.arange(H, device="cuda")[None, :, None]
        return [_element(s["cache"], page, H, D, bits, gs, s["slots"][:, None, None], head, w) for w in "kv"]
    B, G = case["B"], case["G"]
    out = torch.zeros(B, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H * G), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(B):
        at = torch.arange(lens[b], device="cuda")
        if not lens[b]:
            continue
        slot = s["table"][b].long()[at // page] * page + at % page
        for h in range(H):
            k = _element(s["cache"], page, H, D, bits, gs, slot[:, None], h, "k")
            v = _element(s["cache"], page, H, D, bits, gs, slot[:, None], h, "v")
            sc = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(sc, 1)
            out[b, h * G:(h + 1) * G] = torch.softmax(sc, 1) @ v
    return [out, lse] if case["lse"] else out
