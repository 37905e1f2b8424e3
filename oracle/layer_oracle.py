"""fp64 oracle (torch, any device) of the layer's operators around the core: norm
and rotation of queries and keys, cross-attention to an encoder's states, the
8-bit integer linear layer; and error bounds of their kernels.

The functions are written from the definitions, with loops over what the
kernels handle at once.  The bounds are what the kernels' roundings can add up
to; `EPS` is half a step of float32, `step(dtype)` of an output type.
"""
import math

import torch

EPS = 2.0 ** -24


def step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------- norm and rotation
def _rotate(z, table, pos, rot, pairing, sections, sign):
    """Rotates the first `rot` columns of z [tokens, H, d]; pos [tokens, axes] inside the table."""
    out = z.clone()
    half, j = rot // 2, 0
    for axis, pairs in enumerate(sections):
        for _ in range(pairs):
            a, b = (2 * j, 2 * j + 1) if pairing == "interleaved" else (j, j + half)
            c = table[pos[:, axis].long(), j].double()
            cos, sin = c[:, :1], sign * c[:, 1:]
            out[..., a] = z[..., a] * cos - z[..., b] * sin
            out[..., b] = z[..., a] * sin + z[..., b] * cos
            j += 1
    return out


def qk_norm_rope(x, w, table, pos, rot, pairing, sections, eps):
    """One of q and k: x [tokens, H, d], w [d] or [H, d] or None."""
    z = x.double()
    z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        z = z * w.double()
    return _rotate(z, table, pos, rot, pairing, sections, 1.0) if rot else z


def qk_norm_rope_bwd(x, w, table, pos, rot, pairing, sections, eps, g):
    """dx and dw (one row for each head: the caller sums them for a shared weight); also what bounds their
    errors: the scale of dx's terms for each row, and the sum of |terms| of dw."""
    x = x.double()
    rstd = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xh = x * rstd
    dz = _rotate(g.double(), table, pos, rot, pairing, sections, -1.0) if rot else g.double()
    dh = dz if w is None else dz * w.double()
    dx = rstd * (dh - xh * (dh * xh).mean(-1, keepdim=True))
    # a rotated element is bounded by the sum of its pair, a row by twice its largest
    scale = 2 * rstd * (dh.abs().amax(-1, keepdim=True) + xh.abs() * (dh * xh).abs().mean(-1, keepdim=True))
    return dx, (dz * xh).sum(0), scale, 2 * (dz.abs().amax(-1, keepdim=True) * xh.abs()).sum(0)


# --------------------------------------------------------- cross-attention
def cross_attn(q, k, v, kv_len=None, scale=None):
    """o [B, Tq, H, d] and lse [B, Tq, H], float64."""
    B, Tq, H, d = q.shape
    Hkv, s = k.shape[2], scale or 1 / math.sqrt(d)
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = k.shape[1] if kv_len is None else min(max(int(kv_len[b]), 0), k.shape[1])
        for h in range(H if n else 0):
            z = s * (q[b, :, h].double() @ k[b, :n, h * Hkv // H].double().t())
            lse[b, :, h] = torch.logsumexp(z, -1)
            o[b, :, h] = torch.exp(z - lse[b, :, h, None]) @ v[b, :n, h * Hkv // H].double()
    return o, lse


def cross_attn_bound(q, k, v, o, kv_len, scale, operand, out):
    """Bounds of the errors of o and lse: `operand` and `out` are half a step of the type that P is rounded to
    (0: none) and of y.  A score is a sum of d products (the tensor cores may drop a bit of each sum), its
    exponential's relative error is the score's absolute one plus a few steps; P's relative errors move o by at
    most their size times sum_j p_j (|v_j| + |o|)."""
    B, Tq, H, d = q.shape
    Hkv, s = k.shape[2], scale or 1 / math.sqrt(d)
    bo, bl = torch.zeros_like(o), torch.zeros(o.shape[:3], dtype=torch.float64, device=q.device)
    for b in range(B):
        n = k.shape[1] if kv_len is None else min(max(int(kv_len[b]), 0), k.shape[1])
        for h in range(H if n else 0):
            kb, vb, qb = k[b, :n, h * Hkv // H].double(), v[b, :n, h * Hkv // H].double(), q[b, :, h].double()
            z = s * (qb @ kb.t())
            rel = ((2 * d + 32) * EPS * s * (qb.abs() @ kb.abs().t())).amax(-1, keepdim=True) + 32 * EPS
            sums = (2 * n + 64) * EPS  # the sums over the states
            p = torch.softmax(z, -1)
            bo[b, :, h] = 1.05 * (operand + rel + sums) * (p @ vb.abs() + o[b, :, h].abs()) + out * o[b, :, h].abs()
            bl[b, :, h] = (operand + rel + sums).squeeze(-1) * 1.05 + 4 * EPS * (z.abs().amax(-1) + 1)
    return bo, bl


def cross_attn_bwd(q, k, v, dy, kv_len=None, scale=None, y_err=None, operand=0.0, out=0.0):
    """The gradients dq, dk, dv, and the bounds of their errors (dict of pairs).  `y_err` [B, Tq, H, d] bounds the
    error of the kept output that <dy, y> is formed from."""
    B, Tq, H, d = q.shape
    L, Hkv, s = k.shape[1], k.shape[2], scale or 1 / math.sqrt(d)
    G = H // Hkv
    f64 = dict(dtype=torch.float64, device=q.device)
    r = {"dq": torch.zeros(q.shape, **f64), "dk": torch.zeros((B, L, Hkv, d), **f64), "dv": torch.zeros((B, L, Hkv, d), **f64)}
    e = {key: torch.zeros_like(t) for key, t in r.items()}
    for b in range(B):
        n = L if kv_len is None else min(max(int(kv_len[b]), 0), L)
        for h in range(H if n else 0):
            qb, g = q[b, :, h].double(), dy[b, :, h].double()
            kb, vb = k[b, :n, h // G].double(), v[b, :n, h // G].double()
            p = torch.softmax(s * (qb @ kb.t()), -1)
            dp = g @ vb.t()
            o = p @ vb
            delta = (g * o).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            r["dq"][b, :, h] = s * (ds @ kb)
            r["dk"][b, :n, h // G] += s * (ds.t() @ qb)
            r["dv"][b, :n, h // G] += p.t() @ g
            # errors
            rel = ((2 * d + 32) * EPS * s * (qb.abs() @ kb.abs().t())).amax(-1, keepdim=True) + 32 * EPS
            kept = g.abs() * (y_err[b, :, h] if y_err is not None else 0)
            ddelta = kept.sum(-1, keepdim=True) + (2 * d) * EPS * (g * o).abs().sum(-1, keepdim=True)
            ddp = (2 * d) * EPS * (g.abs() @ vb.abs().t())
            ep = (operand + rel) * p
            es = (operand + 3 * rel) * ds.abs() + 1.05 * p * (ddelta + ddp) + 4 * EPS * p * (dp.abs() + delta.abs())
            sq, sk = (2 * n + 64) * EPS, (2 * G * Tq + 64) * EPS  # the sums over the states, and over the rows
            e["dq"][b, :, h] = 1.05 * s * ((es + sq * ds.abs()) @ kb.abs())
            e["dk"][b, :n, h // G] += 1.05 * s * ((es + sk * ds.abs()).t() @ qb.abs())
            e["dv"][b, :n, h // G] += 1.05 * ((ep + sk * p).t() @ g.abs())
    return {key: (r[key], e[key] + out * r[key].abs()) for key in r}


# ------------------------------------------------------------ 8-bit layer
def quantize_int8(x):
    """Codes (int8) and scales (float32, the quotient rounded once) of every row."""
    x = x.double()
    bad = ~torch.isfinite(x).all(1, keepdim=True)
    amax = torch.where(bad, torch.zeros_like(x[:, :1]), x.abs().amax(1, keepdim=True))
    small = amax < 2.0 ** -119
    s = torch.where(small, torch.ones_like(amax), amax / 127).float()
    q = torch.where(small | bad, torch.zeros_like(x), torch.round(x / s.double()))
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    return q.to(torch.int8), s.squeeze(1)


def linear_int8(codes, x_scale, w, w_scale, bias):
    out = codes.double() @ w.double().t() * x_scale.double().unsqueeze(1) * w_scale.double()
    return out if bias is None else out + bias.double()
