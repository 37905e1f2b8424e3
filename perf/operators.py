"""The layer operators around the attention core: the cases they are measured on, and their plain forms.

Three operators of one attention sub-layer, in the order a layer calls them:

* "linear8": a linear layer in 8-bit integers.  Every token's row of x gets a scale s = amax|x| / 127 and the codes
  round(x / s); the product with a weight held as codes and a scale for each output channel; plus a bias.
* "rope" / "rope_bwd": RMSNorm of every query and key head, then the rotation by position, in one pass; and its
  gradients for the inputs and the norm's weights.
* "xattn" / "xattn_bwd": softmax cross-attention of the tokens to an encoder's states of another length, with a length
  for each batch element and key heads shared by groups of query heads; and its gradients.

`run` computes the plain form with elementary torch operations in 32 bits (64 where 32 lose), or, where `own` is set,
calls the package's operators.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a stream, all heads: the latency of a call
        {"name": "rope_token", "kind": "rope", "tokens": 1, "hq": 24, "hk": 24, "d": 128, "rot": 128, "pair": "split",
         "axes": 1, "dtype": "bf16", "per_head": False, "packed": True},
        # the video tokens of one 768p block (90 frames of 24 x 42), three position axes, in a packed projection
        {"name": "rope_768p", "kind": "rope", "tokens": 90720, "hq": 24, "hk": 24, "d": 128, "rot": 128, "pair": "inter",
         "axes": 3, "dtype": "bf16", "per_head": True, "packed": True},
        # the exact (float32) mode at the small workload's size, odd token count, shared key heads, part of d rotated
        {"name": "rope_bwd_small_f32", "kind": "rope_bwd", "tokens": 4799, "hq": 8, "hk": 2, "d": 64, "rot": 32, "pair": "split",
         "axes": 1, "dtype": "f32", "gdtype": "f32", "per_head": False, "packed": False},
        # training at 768p: the core's float32 gradients of q and k taken back to the projection's output
        {"name": "rope_bwd_768p", "kind": "rope_bwd", "tokens": 90720, "hq": 24, "hk": 24, "d": 128, "rot": 128, "pair": "inter",
         "axes": 3, "dtype": "bf16", "gdtype": "f32", "per_head": True, "packed": True},
        # serving: one query token for each of 8 requests over long encoder states of different lengths
        {"name": "xattn_token", "kind": "xattn", "B": 8, "Tq": 1, "L": 4096, "H": 24, "Hkv": 8, "d": 128, "dtype": "bf16",
         "ragged": True, "empty": False},
        # the exact (float32) mode: a ragged batch with one empty prompt
        {"name": "xattn_small_f32", "kind": "xattn", "B": 3, "Tq": 4800, "L": 77, "H": 8, "Hkv": 8, "d": 64, "dtype": "f32",
         "ragged": True, "empty": True},
        # the video tokens of one 768p block over a prompt of 512 tokens
        {"name": "xattn_768p", "kind": "xattn", "B": 1, "Tq": 90720, "L": 512, "H": 24, "Hkv": 24, "d": 128, "dtype": "bf16",
         "ragged": False, "empty": False},
        # a ragged training batch of short clips, shared key heads, a prompt length that ends inside a tile
        {"name": "xattn_bwd_ragged", "kind": "xattn_bwd", "B": 3, "Tq": 5040, "L": 300, "H": 8, "Hkv": 4, "d": 64, "dtype": "bf16",
         "ragged": True, "empty": True},
        # training at 768p
        {"name": "xattn_bwd_768p", "kind": "xattn_bwd", "B": 1, "Tq": 90720, "L": 512, "H": 24, "Hkv": 24, "d": 128, "dtype": "bf16",
         "ragged": False, "empty": False},
        # one token through the layer's concatenated branches (K = 24 heads x 2 branches x 128)
        {"name": "linear8_token", "kind": "linear8", "M": 1, "K": 6144, "N": 4096, "dtype": "bf16", "bias": True},
        # a few hundred tokens (one small latent frame), ragged in every tile
        {"name": "linear8_frame", "kind": "linear8", "M": 237, "K": 1280, "N": 784, "dtype": "bf16", "bias": True},
        # the tokens of one 768p block
        {"name": "linear8_768p", "kind": "linear8", "M": 90720, "K": 6144, "N": 4096, "dtype": "bf16", "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_bwd", "xattn", "xattn", "xattn_bwd", "linear8"])
    if kind in ("rope", "rope_bwd"):
        d = rng.choice([32, 64, 96, 128, 256])
        hk = rng.choice([1, 2, 3, 4, 8, 24])
        hq = hk * rng.choice([1, 1, 2, 3, 5])
        most = 90720 * 48 * 128 // ((hq + hk) * d)
        rot = rng.choice([d, d, d // 2])
        c = {"kind": kind, "tokens": _log(rng, 1, min(90720, most)), "hq": hq, "hk": hk, "d": d, "rot": rot - rot % 16,
             "pair": rng.choice(["split", "inter"]), "axes": rng.choice([1, 3]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
             "per_head": rng.random() < 0.5, "packed": rng.random() < 0.5}
        if c["dtype"] == "f32":
            c["tokens"] = max(1, c["tokens"] // 2)
        if kind == "rope_bwd":
            c["gdtype"] = "f32" if c["dtype"] == "f32" else rng.choice(["bf16", "f32"])
        return c
    if kind in ("xattn", "xattn_bwd"):
        exact32 = rng.random() < 0.2
        d = rng.choice([32, 64, 128]) if exact32 else rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        H = hkv * rng.choice([1, 1, 2, 3])
        B = rng.choice([1, 1, 2, 3, 5])
        # one key alone leaves gradients of zero for q and k, which have no relative error
        L = _log(rng, 8 if kind == "xattn_bwd" else 1, 512 if exact32 else 8192)
        most = (1 << 27 if exact32 else 1 << 30) // (B * H * L)
        return {"kind": kind, "B": B, "Tq": _log(rng, 1, max(1, min(2000 if exact32 else 60000, most))), "L": L, "H": H, "Hkv": hkv,
                "d": d, "dtype": "f32" if exact32 else "bf16", "ragged": B > 1 or rng.random() < 0.3, "empty": B > 2 and rng.random() < 0.3}
    K, N = 16 * _log(rng, 4, 384), 16 * _log(rng, 4, 256)
    return {"kind": kind, "M": _log(rng, 1, 60000), "K": K, "N": N, "dtype": rng.choice(["bf16", "bf16", "f32"]), "bias": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _sections(c):
    """Rotated pairs of each position axis: the whole half for one axis; frame, row and column for three."""
    half = c["rot"] // 2
    if c["axes"] == 1:
        return [half]
    side = half * 3 // 8
    return [half - 2 * side, side, side]


def _positions(c):
    """Position of every token on every axis: a run far from the start, or a (frame, row, column) grid."""
    i = torch.arange(c["tokens"], device="cuda")
    if c["axes"] == 1:
        return (i % 4096 + 28000).unsqueeze(1).int().contiguous(), 32768
    return torch.stack([i // 1008 % 128, i // 42 % 24, i % 42], 1).int().contiguous(), 128


def _table(c, rows):
    """(cos, sin) of position times frequency, [rows, rot / 2, 2], the angles in 64 bits."""
    freq = torch.cat([10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / max(n, 1)) for n in _sections(c)])
    a = torch.arange(rows, device="cuda", dtype=torch.float64).unsqueeze(1) * freq
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _lengths(c):
    """Valid encoder states of every batch element: a spread from L down to a quarter of it, and an empty one."""
    n = [max(1, c["L"] - b * c["L"] * 3 // (4 * c["B"])) - (1 if c["B"] == 1 and c["L"] > 1 else 0) for b in range(c["B"])]
    if c["empty"]:
        n[-1] = 0
    return n if c["ragged"] else [c["L"]] * c["B"]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[c["dtype"]]
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    s = {"case": c}
    if c["kind"] in ("rope", "rope_bwd"):
        t, hq, hk, d = c["tokens"], c["hq"], c["hk"], c["d"]
        if c["packed"]:  # the query and key heads of one projection's output [tokens, hq + 2 hk, d]
            x = torch.randn((t, hq + 2 * hk, d), device="cuda", generator=g, dtype=dt).mul_(1.5)
            s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
        else:
            s["q"], s["k"] = (1.5 * rand(t, hq, d)).to(dt), (1.5 * rand(t, hk, d)).to(dt)
        shape = (lambda h: (h, d)) if c["per_head"] else (lambda h: (d,))
        s["wq"], s["wk"] = 1 + 0.2 * rand(*shape(hq)), 1 + 0.2 * rand(*shape(hk))
        s["pos"], rows = _positions(c)
        s["table"] = _table(c, rows)
        if c["kind"] == "rope_bwd":
            gt = TYPES[c["gdtype"]]
            s["gq"] = torch.randn((t, hq, d), device="cuda", generator=g, dtype=gt)
            s["gk"] = torch.randn((t, hk, d), device="cuda", generator=g, dtype=gt)
        if own:
            from video_diffusion_hybrid_b200.api import QKNormRope
            s["op"] = QKNormRope(hq, hk, d, rot=c["rot"], pairing="split" if c["pair"] == "split" else "interleaved",
                                 sections=_sections(c), per_head=c["per_head"], eps=1e-6)
    elif c["kind"] in ("xattn", "xattn_bwd"):
        B, Tq, L, H, Hkv, d = c["B"], c["Tq"], c["L"], c["H"], c["Hkv"], c["d"]
        s["q"] = torch.randn((B, Tq, H, d), device="cuda", generator=g, dtype=dt).mul_(1.5)
        kv = rand(B, L, 2, Hkv, d).to(dt)  # one projection of the encoder's states
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        s["len"] = torch.tensor(_lengths(c), device="cuda", dtype=torch.int32) if c["ragged"] else None
        if c["kind"] == "xattn_bwd":
            s["dy"] = torch.randn((B, Tq, H, d), device="cuda", generator=g, dtype=dt)
            s["y"], s["lse"] = _attend(s)  # kept from the forward pass
            s["y"] = s["y"].to(dt)
        if own:
            from video_diffusion_hybrid_b200.api import CrossAttention
            s["op"] = CrossAttention(B, Tq, L, H, Hkv, d, dtype=c["dtype"])
    else:
        M, K, N = c["M"], c["K"], c["N"]
        x = torch.randn((M, K), device="cuda", generator=g, dtype=dt)
        s["x"] = x.mul_((1 + 4 * (torch.rand(K, device="cuda", generator=g) < 0.02)).to(dt))  # a few large channels
        w = rand(N, K) / math.sqrt(K)
        s["ws"] = w.abs().amax(1) / 127
        s["w"] = (w.double() / s["ws"].double().unsqueeze(1)).round().to(torch.int8)
        s["b"] = 0.1 * rand(N) if c["bias"] else None
        if own:
            from video_diffusion_hybrid_b200.api import Int8Linear
            s["op"] = Int8Linear(s["w"], s["ws"], s["b"], out_dtype=c["dtype"])
    return s


# ------------------------------------------------------------ plain forms
def _angles(s, f=torch.float32):
    """cos and sin of every token's rotated pairs [tokens, 1, rot / 2]: the table's row of the pair's own axis."""
    c = s["case"]
    n = _sections(c)
    axis = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
    p = s["pos"].long()[:, axis]
    cs = s["table"][p, torch.arange(c["rot"] // 2, device="cuda")].to(f)
    return cs[..., 0].unsqueeze(1), cs[..., 1].unsqueeze(1)


def _turn(x, cos, sin, c):
    """The rotated pairs of x's first `rot` columns; the others as they are."""
    r, half = c["rot"], c["rot"] // 2
    a, b = (x[..., :half], x[..., half:r]) if c["pair"] == "split" else (x[..., 0:r:2], x[..., 1:r:2])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([u, v], -1) if c["pair"] == "split" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _rope(x, w, cos, sin, c):
    x = x.float()
    return _turn(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w, cos, sin, c)


def _rope_bwd(x, w, g, cos, sin, c):
    x = x.float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    xh = x * rstd
    dz = _turn(g.float(), cos, -sin, c)
    dw = (dz * xh).sum(0, dtype=torch.float64)
    dh = dz * w
    return rstd * (dh - xh * (dh * xh).mean(-1, keepdim=True)), (dw if c["per_head"] else dw.sum(0)).float()


def _grouped(s):
    """q as [B, Hkv, G, Tq, d]; k and v as [B, Hkv, 1, L, d]; 32 bits."""
    c = s["case"]
    heads = lambda x: x.float().unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4)  # noqa: E731
    return heads(s["q"]), heads(s["k"]), heads(s["v"]), heads


def _weights(s, q, k):
    """Unnormalised softmax weights, their sum and the maximum they are relative to; all zero where nothing is valid."""
    c = s["case"]
    z = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(c["d"]))
    if s["len"] is not None:
        gone = torch.arange(c["L"], device="cuda") >= s["len"].view(-1, 1, 1, 1, 1)
        z = z.masked_fill(gone, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(z - m)
    return e, e.sum(-1, keepdim=True), m


def _attend(s):
    """o [B, Tq, H, d] and the log-sum-exp [B, Tq, H], 32 bits."""
    q, k, v, _ = _grouped(s)
    e, l, m = _weights(s, q, k)
    o = torch.matmul(e, v) / torch.where(l == 0, torch.ones_like(l), l)
    back = lambda x: x.permute(0, 3, 1, 2, 4).flatten(2, 3)  # noqa: E731
    return back(o).contiguous(), back(m + torch.log(l)).squeeze(-1).contiguous()


def _attend_bwd(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    q, k, v, heads = _grouped(s)
    dy = heads(s["dy"])
    e, l, _ = _weights(s, q, k)
    p = e / torch.where(l == 0, torch.ones_like(l), l)
    del e
    delta = (dy * heads(s["y"])).sum(-1, keepdim=True)
    dv = torch.matmul(p.transpose(-1, -2), dy).sum(2)
    ds = p * (torch.matmul(dy, v.transpose(-1, -2)) - delta) * (1 / math.sqrt(c["d"]))
    del p
    dq = torch.matmul(ds, k).permute(0, 3, 1, 2, 4).flatten(2, 3)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return {"dq": dq.to(dt), "dk": dk.transpose(1, 2).to(dt), "dv": dv.transpose(1, 2).to(dt)}


def run(s):
    c = s["case"]
    dt = TYPES[c["dtype"]]
    if own:
        if c["kind"] == "rope":
            q, k = s["op"](s["q"], s["k"], s["wq"], s["wk"], s["table"], s["pos"])
            return {"q": q, "k": k}
        if c["kind"] == "rope_bwd":
            return s["op"].backward(s["q"], s["k"], s["wq"], s["wk"], s["table"], s["gq"], s["gk"], s["pos"])
        if c["kind"] == "xattn":
            return {"y": s["op"](s["q"], s["k"], s["v"], s["len"])}
        if c["kind"] == "xattn_bwd":
            return s["op"].backward(s["q"], s["k"], s["v"], s["y"], s["lse"], s["dy"], s["len"])
        return {"out": s["op"](s["x"])}
    if c["kind"] == "rope":
        cos, sin = _angles(s)
        return {"q": _rope(s["q"], s["wq"], cos, sin, c).to(dt), "k": _rope(s["k"], s["wk"], cos, sin, c).to(dt)}
    if c["kind"] == "rope_bwd":
        cos, sin = _angles(s)
        dq, dwq = _rope_bwd(s["q"], s["wq"], s["gq"], cos, sin, c)
        dk, dwk = _rope_bwd(s["k"], s["wk"], s["gk"], cos, sin, c)
        return {"dq": dq.to(dt), "dk": dk.to(dt), "dwq": dwq, "dwk": dwk}
    if c["kind"] == "xattn":
        return {"y": _attend(s)[0].to(dt)}
    if c["kind"] == "xattn_bwd":
        return _attend_bwd(s)
    x = s["x"].float()
    sx = (x.abs().amax(1, keepdim=True).double() / 127).float()  # one rounding of the quotient: ties among the codes go by it
    codes = (x.double() / sx.double()).round().float()
    out = torch.matmul(codes, s["w"].float().t()) * sx * s["ws"]
    return {"out": (out if s["b"] is None else out + s["b"]).to(dt)}


# ------------------------------------------------------------------ work
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] in ("rope", "rope_bwd"):
        h = c["hq"] + c["hk"]
        n = c["tokens"] * h * c["d"]
        w = 4 * c["d"] * (h if c["per_head"] else 2)
        rows = 4096 if c["axes"] == 1 else 128
        pos = 4 * c["tokens"] * c["axes"] + 4 * c["rot"] * min(rows, c["tokens"])
        if c["kind"] == "rope":
            return {"bytes": 2 * n * e + w + pos, "flops": 9 * n}
        return {"bytes": n * (2 * e + (2 if c["gdtype"] == "bf16" else 4)) + 2 * w + pos, "flops": 16 * n}
    if c["kind"] in ("xattn", "xattn_bwd"):
        keys = sum(_lengths(c))
        rows = c["B"] * c["Tq"] * c["H"]
        kv = keys * c["Hkv"] * c["d"]
        prod = 2 * c["Tq"] * c["H"] * keys * c["d"]
        if c["kind"] == "xattn":
            return {"bytes": e * (2 * rows * c["d"] + 2 * kv), "flops": 2 * prod}
        return {"bytes": e * (4 * rows * c["d"] + 2 * kv + 2 * c["B"] * c["L"] * c["Hkv"] * c["d"]) + 4 * rows, "flops": 5 * prod}
    return {"bytes": c["M"] * c["K"] * e + c["K"] * c["N"] + 4 * c["N"] * (2 if c["bias"] else 1) + c["M"] * c["N"] * e,
            "flops": 2 * c["M"] * c["N"] * c["K"]}


# ----------------------------------------------------------------- exact
def _exact_rotation(case, s):
    """The rotation of each token as complex numbers, in 64 bits: [tokens, 1, rot / 2]."""
    n = _sections(case)
    cols, at = [], 0
    for axis, pairs in enumerate(n):
        cols.append(s["table"][:, at:at + pairs].double().index_select(0, s["pos"][:, axis].long()))
        at += pairs
    return torch.view_as_complex(torch.cat(cols, 1).contiguous()).unsqueeze(1)


def _exact_pairs(x, case):
    r = case["rot"]
    x = x[..., :r]
    x = x.unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["pair"] == "split" else x.unflatten(-1, (r // 2, 2))
    return torch.view_as_complex(x.contiguous())


def _exact_unpair(z, rest, case):
    x = torch.view_as_real(z)
    x = x.transpose(-1, -2).flatten(-2) if case["pair"] == "split" else x.flatten(-2)
    return torch.cat([x, rest], -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] in ("rope", "rope_bwd"):
        e = _exact_rotation(c, s)
        out = {}
        for n in ("q", "k"):
            x, w = s[n].double(), s["w" + n].double()
            norm = (x.square().sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt()
            if c["kind"] == "rope":
                z = x / norm * w
                out[n] = _exact_unpair(_exact_pairs(z, c) * e, z[..., c["rot"]:], c)
                continue
            g = s["g" + n].double()
            g = _exact_unpair(_exact_pairs(g, c) * e.conj(), g[..., c["rot"]:], c)
            dw = (g * x / norm).sum(0)
            out["dw" + n] = dw if c["per_head"] else dw.sum(0)
            g = g * w
            out["d" + n] = g / norm - x * (g * x).sum(-1, keepdim=True) / (c["d"] * norm ** 3)
        return out
    if c["kind"] in ("xattn", "xattn_bwd"):
        G, n = c["H"] // c["Hkv"], _lengths(c)
        q = s["q"].double()
        y = torch.zeros_like(q)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(s["k"], dtype=torch.float64), torch.zeros_like(s["v"], dtype=torch.float64)
        for b in range(c["B"]):
            for h in range(c["H"]):
                k, v = s["k"][b, :n[b], h // G].double(), s["v"][b, :n[b], h // G].double()
                if n[b] == 0:
                    continue
                p = torch.softmax(q[b, :, h] @ k.t() / math.sqrt(c["d"]), -1)
                y[b, :, h] = p @ v
                if c["kind"] == "xattn":
                    continue
                g = s["dy"][b, :, h].double()
                t = g @ v.t()
                t = p * (t - (t * p).sum(-1, keepdim=True)) / math.sqrt(c["d"])
                dq[b, :, h] = t @ k
                dk[b, :n[b], h // G] += t.t() @ q[b, :, h]
                dv[b, :n[b], h // G] += p.t() @ g
        return {"y": y} if c["kind"] == "xattn" else {"dq": dq, "dk": dk.contiguous(), "dv": dv.contiguous()}
    x = s["x"].double()
    top = (x.abs().amax(1, keepdim=True) / 127).float().double()  # the scale is held in 32 bits
    out = torch.round(x / top) @ s["w"].double().t() * (top * s["ws"].double())
    return {"out": out if s["b"] is None else out + s["b"].double()}
