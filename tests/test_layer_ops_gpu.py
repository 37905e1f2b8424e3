"""The layer's operators around the core against the fp64 oracle, within bounds
worked out from their roundings (oracle/layer_oracle.py)."""
import math

import pytest
import torch

from oracle import layer_oracle as R
from video_diffusion_hybrid_b200 import _lib as L
from video_diffusion_hybrid_b200.api import CrossAttention, Int8Linear, QKNormRope, quantize_int8, rope_table
from video_diffusion_hybrid_b200.build import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    if torch.cuda.is_available():
        build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def within(got, want, bound, what):
    """|got - want| <= bound everywhere (and no NaN)."""
    d = (got.double() - want).abs()
    worst = float((d / bound.clamp_min(1e-300)).nan_to_num(nan=math.inf).max()) if d.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound"


# ------------------------------------------------------- norm and rotation
QK = [  # tokens, Hq, Hk, d, rot, sections, pairing, dtype, per_head, packed
    (1, 24, 24, 128, 128, (64,), "split", "bf16", False, True),
    (1, 1, 0, 8, 0, (0,), "split", "f32", True, False),
    (1237, 24, 24, 128, 128, (16, 24, 24), "interleaved", "bf16", True, True),
    (333, 8, 2, 64, 32, (16,), "split", "f32", False, False),
    (5000, 1, 1, 32, 32, (16,), "interleaved", "bf16", False, False),
    (2049, 5, 1, 96, 48, (3, 12, 9), "split", "bf16", True, True),
    (700, 3, 3, 256, 256, (48, 40, 40), "interleaved", "f32", True, True),
    (97, 40, 7, 16, 16, (5, 3), "interleaved", "bf16", False, True),
    (64, 2, 2, 40, 16, (8,), "split", "bf16", True, False),
    (3001, 24, 8, 128, 64, (32,), "split", "f32", True, False),
]


def qk_case(case, seed=0, skip=True):
    tokens, Hq, Hk, d, rot, sections, pairing, dtype, per_head, packed = case
    g, dt = gen(seed), DT[dtype]
    if packed:
        x = rnd(g, tokens, Hq + 2 * Hk + 1, d, dtype=dt, scale=1.5)
        q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    else:
        q, k = rnd(g, tokens, Hq, d, dtype=dt, scale=1.5), rnd(g, tokens, Hk, d, dtype=dt, scale=1.5)
    wshape = (lambda h: (h, d)) if per_head else (lambda h: (d,))
    wq, wk = 1 + rnd(g, *wshape(Hq), scale=0.2), 1 + rnd(g, *wshape(Hk), scale=0.2)
    rows = 300
    table = rope_table(rows, sections) if rot else None
    pos = torch.randint(0, rows, (tokens, len(sections)), device="cuda", generator=g, dtype=torch.int32)
    on = torch.ones(tokens, dtype=torch.bool, device="cuda")
    if skip and tokens > 8:
        pos[3, 0], pos[5, -1], pos[tokens - 1, 0] = -1, rows if rot else -(2 ** 31), 2 ** 31 - 1
        on[torch.tensor([3, 5] + ([tokens - 1] if rot else []), device="cuda")] = False
    op = QKNormRope(Hq, Hk, d, rot=rot, pairing=pairing, sections=sections, per_head=per_head)
    return op, dict(q=q, k=k if Hk else None, wq=wq, wk=wk if Hk else None, table=table, pos=pos), on, dt


def qk_forward_check(op, a, on, dt, out):
    for key, got in zip(("q", "k"), out):
        if a[key] is None:
            assert got is None
            continue
        if a["pos"] is None:
            p = torch.arange(a[key].shape[0], device="cuda", dtype=torch.int32).unsqueeze(1)
        else:
            p = torch.where(on.unsqueeze(1), a["pos"], 0)
        pair = "interleaved" if op.pairing == L.PAIR_INTERLEAVED else "split"
        want = R.qk_norm_rope(a[key], a["w" + key], a["table"], p, op.rot, pair, op.sections, 1e-6)
        # an element is two products of values with a few roundings each; a pair's size bounds both
        size = want.abs().amax(-1, keepdim=True) * 2
        within(got[on], want[on], R.step(dt) * want[on].abs() + 24 * R.EPS * size[on], key)


@pytest.mark.parametrize("case", QK, ids=str)
def test_qk_norm_rope(cuda_ok, case):
    op, a, on, dt = qk_case(case)
    out = tuple(None if a[k] is None else torch.full(a[k].shape, 7.0, device="cuda", dtype=dt) for k in "qk")
    got = op(a["q"], a["k"], a["wq"], a["wk"], a["table"], a["pos"], out=out)
    qk_forward_check(op, a, on, dt, got)
    for t in got:  # skipped tokens' rows are left as they were
        assert t is None or bool((t[~on] == 7.0).all())


@pytest.mark.parametrize("case", QK, ids=str)
@pytest.mark.parametrize("gdtype", ["f32", "bf16"])
def test_qk_norm_rope_backward(cuda_ok, case, gdtype):
    if case[7] == "f32" and gdtype == "bf16":
        pytest.skip("refused: float32 tensors have float32 gradients")
    op, a, on, dt = qk_case(case, 1)
    g = gen(2)
    up = {k: None if a[k] is None else rnd(g, *a[k].shape, dtype=DT[gdtype]) for k in "qk"}
    # whatever stands in a skipped token's rows, nothing of it reaches a gradient
    for k in "qk":
        if a[k] is not None:
            a[k][~on] = math.nan
            up[k][~on] = math.inf
    got = op.backward(a["q"], a["k"], a["wq"], a["wk"], a["table"], up["q"], up["k"], a["pos"])
    p = torch.where(on.unsqueeze(1), a["pos"], 0)[on]
    pair = "interleaved" if op.pairing == L.PAIR_INTERLEAVED else "split"
    for k in "qk":
        if a[k] is None:
            assert "d" + k not in got and "dw" + k not in got
            continue
        dx, dw, scale, terms = R.qk_norm_rope_bwd(a[k][on], a["w" + k], a["table"], p, op.rot, pair, op.sections, 1e-6, up[k][on])
        assert bool((got["d" + k][~on] == 0).all())
        # sums over the row of at most 8 + log2(32) steps, and about twenty roundings of each term
        within(got["d" + k][on], dx, R.step(dt) * dx.abs() + 64 * R.EPS * scale, "d" + k)
        if not op.per_head:
            dw, terms = dw.sum(0), terms.sum(0)
        n = int(on.sum()) * (1 if op.per_head else a[k].shape[1])
        within(got["dw" + k], dw, (n + 64) * R.EPS * terms + 1e-30, "dw" + k)


def test_qk_index_positions_and_unit_weights(cuda_ok):
    op, a, on, dt = qk_case(QK[3], 3, skip=False)
    a.update(pos=None, wq=None, wk=None, table=rope_table(400, (16,)))
    qk_forward_check(op, a, on, dt, op(a["q"], a["k"], None, None, a["table"]))
    g = op.backward(a["q"], a["k"], None, None, a["table"], a["q"].contiguous(), a["k"].contiguous())
    assert g["dwq"].shape == (64,) and bool(torch.isfinite(g["dwq"]).all())


def test_qk_leading_axes_are_tokens(cuda_ok):
    """[B, T, H, d] slices of one projection [B, T, 3, H, d] give what their tokens in a row give."""
    g = gen(4)
    x = rnd(g, 2, 37, 3, 4, 64, dtype=torch.bfloat16)
    op = QKNormRope(4, 4, 64)
    table = rope_table(80, (32,))
    pos = torch.arange(74, device="cuda", dtype=torch.int32).view(2, 37)
    q, k = op(x[:, :, 0], x[:, :, 1], None, None, table, pos)
    q2, k2 = op(x[:, :, 0].reshape(74, 4, 64), x[:, :, 1].reshape(74, 4, 64), None, None, table)
    assert torch.equal(q.view(74, 4, 64), q2) and torch.equal(k.view(74, 4, 64), k2)


def test_qk_gradients_are_the_same_on_every_run(cuda_ok):
    op, a, _, _ = qk_case(QK[2], 5)
    g = gen(6)
    up = [rnd(g, *a[k].shape) for k in "qk"]
    one = op.backward(a["q"], a["k"], a["wq"], a["wk"], a["table"], *up, a["pos"])
    for _ in range(3):
        two = op.backward(a["q"], a["k"], a["wq"], a["wk"], a["table"], *up, a["pos"])
        assert all(torch.equal(one[k], two[k]) for k in one)


def test_qk_refusals(cuda_ok):
    op, a, _, _ = qk_case(QK[3], 7)
    call = lambda **kw: op(*({**a, **kw}[k] for k in ("q", "k", "wq", "wk", "table", "pos")))  # noqa: E731
    for bad in (dict(q=a["q"].half()), dict(q=a["q"][..., ::2]), dict(q=a["q"].transpose(0, 1)), dict(k=a["q"]), dict(k=a["k"][:-1]),
                dict(wq=a["wq"].double()), dict(wq=a["wq"][:8]), dict(table=a["table"][:, :8]), dict(pos=a["pos"].long()),
                dict(pos=a["pos"][:-1]), dict(q=a["q"].cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    for missing in ("q", "k", "table"):
        with pytest.raises((ValueError, TypeError)):
            call(**{missing: None})
    up = [torch.zeros_like(a[key]) for key in "qk"]
    for bad in ((None, up[1]), (up[0], None), (up[0].double(), up[1]), (up[0][:-1], up[1]), (up[0], up[1].bfloat16())):
        with pytest.raises((ValueError, TypeError)):
            op.backward(a["q"], a["k"], a["wq"], a["wk"], a["table"], *bad, a["pos"])
    with pytest.raises(L.VdnError):
        QKNormRope(8, 2, 64, pairing="other")
    with pytest.raises(L.VdnError):
        call(pos=None, table=a["table"][:100])  # fewer rows than tokens


# --------------------------------------------------------- cross-attention
X = [  # B, Tq, L, H, Hkv, d, dtype, lens, strided
    (1, 1, 1, 1, 1, 64, "bf16", None, False),
    (2, 1, 4096, 24, 8, 128, "bf16", [4096, 1023], True),
    (8, 1, 777, 4, 1, 64, "bf16", [0, 1, 63, 64, 65, 128, 129, 777], True),
    (3, 5, 300, 6, 2, 128, "bf16", [300, 0, 129], True),
    (1, 17, 4001, 5, 1, 64, "bf16", None, False),
    (1, 100, 77, 2, 2, 64, "bf16", [50], False),
    (2, 129, 128, 2, 2, 128, "bf16", [128, 127], False),
    (1, 256, 512, 4, 4, 128, "bf16", None, True),
    (2, 700, 300, 4, 2, 64, "bf16", [300, 0], True),
    (3, 1025, 515, 6, 2, 128, "bf16", [515, 385, -4], True),
    (1, 64, 8192, 3, 1, 128, "bf16", [8191], False),
    (1, 333, 1500, 24, 1, 64, "bf16", None, False),
    (5, 40, 20, 9, 3, 128, "bf16", [20, 1, 7, 0, 100], True),
    (2, 33, 40, 2, 1, 32, "bf16", [40, 11], False),
    (1, 1, 8192, 1, 1, 128, "bf16", None, False),
    (2, 1, 33, 8, 1, 128, "bf16", [33, 32], True),
    (3, 2, 1000, 4, 1, 64, "bf16", [1000, 999, 0], True),
    (70, 1, 130, 4, 2, 64, "bf16", [130 - i for i in range(70)], True),
    (1, 7, 517, 2, 2, 128, "bf16", [511], True),
    (300, 2, 24, 2, 1, 128, "bf16", [i % 25 for i in range(300)], False),
    (1, 1, 1, 1, 1, 32, "f32", None, False),
    (3, 97, 77, 4, 4, 64, "f32", [77, 0, 13], True),
    (2, 64, 65, 6, 2, 128, "f32", [65, 64], False),
    (4, 1, 200, 8, 2, 32, "f32", [200, 0, 1, 65], True),
]


def x_case(case, seed=0, poison=True, scale=0.0):
    B, Tq, Lk, H, Hkv, d, dtype, lens, strided = case
    g, dt = gen(seed), DT[dtype]
    q = rnd(g, B, Tq, H, d, dtype=dt, scale=1.5)
    if strided:
        kv = rnd(g, B, Lk, 2, Hkv, d, dtype=dt)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = rnd(g, B, Lk, Hkv, d, dtype=dt), rnd(g, B, Lk, Hkv, d, dtype=dt)
    n = None if lens is None else torch.tensor(lens, device="cuda", dtype=torch.int32)
    clean = (k.clone(), v.clone())
    if lens is not None and poison:  # states past the length may hold anything
        for b, m in enumerate(lens):
            m = max(m, 0)
            k[b, m:], v[b, m:] = math.nan, math.inf
            if m + 2 < Lk:
                k[b, m + 1::2], v[b, m + 1::2] = -math.inf, math.nan
    op = CrossAttention(B, Tq, Lk, H, Hkv, d, dtype=dtype, scale=scale, keep_lse=True)
    return op, q, k, v, n, clean, dt


def x_status(op, backward=False):
    assert op.status(backward)[0] == L.VDN_OK


def x_forward_check(op, q, k, v, n, dt, y, scale=None):
    want, lse = R.cross_attn(q, k, v, n, scale)
    operand = R.step(dt) if dt == torch.bfloat16 else 0.0
    bo, bl = R.cross_attn_bound(q, k, v, want, n, scale, operand, R.step(dt))
    within(y, want, bo, "y")
    dead = lse == -math.inf
    assert torch.equal(op.lse == -math.inf, dead)
    within(op.lse[~dead], lse[~dead], bl[~dead], "lse")
    return want, lse, bo


@pytest.mark.parametrize("case", X, ids=str)
def test_cross_attn(cuda_ok, case):
    op, q, k, v, n, (kc, vc), dt = x_case(case)
    room = torch.full((q.numel() + 512,), 7.0, device="cuda", dtype=dt)  # what lies behind the last row stays
    out = room[:q.numel()].view(q.shape)
    y = op(q, k, v, n, out=out)
    x_status(op)
    assert y is out and bool((room[q.numel():] == 7.0).all())
    x_forward_check(op, q, kc, vc, n, dt, y)


def x_grads(op, q, k, v, n, clean, dt, seed, scale=None):
    kc, vc = clean
    want, lse = R.cross_attn(q, kc, vc, n, scale)
    dy = rnd(gen(seed), *q.shape, dtype=dt)
    y = want.to(dt)
    got = op.backward(q, k, v, y, lse.float(), dy, n)
    x_status(op, True)
    operand = R.step(dt) if dt == torch.bfloat16 else 0.0
    ref = R.cross_attn_bwd(q, kc, vc, dy, n, scale, R.step(dt) * want.abs(), operand, R.step(dt))
    # the log-sum-exp comes in 32 bits: another relative error of P, and of every term
    more = 4 * R.EPS * (1 + float(lse[lse > -math.inf].abs().max()) if bool((lse > -math.inf).any()) else 1)
    for key, (r, e) in ref.items():
        within(got[key], r, e * (1 + 1e-3) + more * r.abs().max() + 1e-30, key)
    return got


@pytest.mark.parametrize("case", X, ids=str)
def test_cross_attn_backward(cuda_ok, case):
    op, q, k, v, n, clean, dt = x_case(case, 1)
    got = x_grads(op, q, k, v, n, clean, dt, 2)
    for b, m in enumerate(case[7] or []):  # no gradient past the length
        m = max(m, 0)
        assert bool((got["dk"][b, m:] == 0).all()) and bool((got["dv"][b, m:] == 0).all())
        assert m > 0 or bool((got["dq"][b] == 0).all())


@pytest.mark.parametrize("case", [X[1], X[9], X[-3]], ids=str)
def test_cross_attn_tiny_scale(cuda_ok, case):
    """Scores of zero in effect: every weight alike, the log-sum-exp that of the number of states."""
    op, q, k, v, n, clean, dt = x_case(case, 70, scale=1e-38)
    x_forward_check(op, q, *clean, n, dt, op(q, k, v, n), 1e-38)


@pytest.mark.parametrize("case", [X[2], X[9], X[-3]], ids=str)
def test_cross_attn_scale_and_large_scores(cuda_ok, case):
    """A scale of one: scores of tens, weights near one-hot."""
    op, q, k, v, n, clean, dt = x_case(case, 3, scale=1.0)
    y = op(q, k, v, n)
    x_forward_check(op, q, *clean, n, dt, y, 1.0)
    x_grads(op, q, k, v, n, clean, dt, 4, 1.0)


@pytest.mark.parametrize("case", [X[1], X[9], X[-3]], ids=str)
def test_cross_attn_rising_scores(cuda_ok, case):
    """Scores that rise along the states: the running maximum moves in every tile."""
    op, q, k, v, n, _, dt = x_case(case, 5, poison=False)
    q.fill_(1.0)
    ramp = torch.linspace(-2, 2, k.shape[1], device="cuda").view(1, -1, 1, 1)
    k.copy_(k * 0.1 + ramp)
    x_forward_check(op, q, k, v, n, dt, op(q, k, v, n))


FEW = [  # few rows of a key head: one and two blocks of 8, full and not; lengths that end inside a stage of 16 states
    (2, 4, 1100, 8, 2, 64, "bf16", [1100, 1089], True),
    (1, 1, 2000, 16, 1, 128, "bf16", None, False),
    (3, 3, 257, 6, 2, 128, "bf16", [257, 16, 0], True),
    (2, 1, 4096, 9, 1, 64, "bf16", [4001, 15], True),
    (40, 1, 65, 8, 8, 128, "bf16", [65 - i for i in range(40)], True),
]


@pytest.mark.parametrize("case", FEW, ids=str)
def test_cross_attn_few_rows(cuda_ok, case):
    op, q, k, v, n, clean, dt = x_case(case, 80)
    x_forward_check(op, q, *clean, n, dt, op(q, k, v, n))


@pytest.mark.parametrize("case", FEW, ids=str)
@pytest.mark.parametrize("rise", [0.2, 0.7, 3.0, -3.0])
def test_cross_attn_few_rows_rising_scores(cuda_ok, case, rise):
    """The reference of the running sum follows only scores that leave it far behind: a rise that stays below that, one
    that passes it now and then, one in nearly every stage, and a fall (weights that fade to zero)."""
    op, q, k, v, n, _, dt = x_case(case, 81, poison=False)
    q.fill_(1.0)
    k.copy_(k * 0.1 + torch.linspace(-rise, rise, k.shape[1], device="cuda").view(1, -1, 1, 1))
    x_forward_check(op, q, k, v, n, dt, op(q, k, v, n))


@pytest.mark.parametrize("case", [X[1], X[9], X[-3]], ids=str)
def test_cross_attn_states_that_weigh_nothing(cuda_ok, case):
    """States with a key of the type's lowest values: scores of -inf or close to it, a weight of zero."""
    op, q, k, v, n, _, dt = x_case(case, 6, poison=False)
    q.abs_().add_(0.5)
    low = torch.finfo(dt).min
    k[:, : k.shape[1] // 2] = low  # the first half: whole tiles of it
    y = op(q, k, v, n)
    x_status(op)
    half = k.shape[1] // 2
    nn = torch.full((q.shape[0],), k.shape[1], device="cuda", dtype=torch.int32) if n is None else n.clamp(0, k.shape[1])
    live = nn > half  # a batch element that has nothing else is undefined: its scores are all -inf
    assert bool(torch.isfinite(y[live]).all())
    want, _ = R.cross_attn(q, k[:, half:], v[:, half:], (nn - half).clamp_min(0))
    bo, _ = R.cross_attn_bound(q, k[:, half:], v[:, half:], want, (nn - half).clamp_min(0), None,
                               R.step(dt) if dt == torch.bfloat16 else 0.0, R.step(dt))
    within(y[live], want[live], bo[live], "y")


def test_cross_attn_a_bad_row_stays_alone(cuda_ok):
    """A query row of infinities or NaN gives NaN in its own row only."""
    for case in (X[9], X[-3], X[1]):
        op, q, k, v, n, clean, dt = x_case(case, 7)
        q[0, 0, 1] = math.nan
        q[0, -1, 0, 3] = math.inf
        y = op(q, k, v, n)
        ok = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
        ok[0, 0, 1] = ok[0, -1, 0] = False
        want, _ = R.cross_attn(q, *clean, n)
        bo, _ = R.cross_attn_bound(q, *clean, want, n, None, R.step(dt) if dt == torch.bfloat16 else 0.0, R.step(dt))
        assert bool(torch.isnan(y[0, 0, 1]).all()) and bool(torch.isnan(y[0, -1, 0]).any())
        within(y[ok], want[ok], bo[ok], "y")


def test_cross_attn_forward_feeds_backward(cuda_ok):
    """The kept output and log-sum-exp of the kernel's own forward, as a training step uses them."""
    for case in (X[9], X[3], X[-3], X[-9]):
        op, q, k, v, n, (kc, vc), dt = x_case(case, 8)
        y = op(q, k, v, n)
        want, lse, bo = x_forward_check(op, q, kc, vc, n, dt, y)
        dy = rnd(gen(9), *q.shape, dtype=dt)
        got = op.backward(q, k, v, y, op.lse, dy, n)
        operand = R.step(dt) if dt == torch.bfloat16 else 0.0
        _, bl = R.cross_attn_bound(q, kc, vc, want, n, None, operand, R.step(dt))
        # P off by the log-sum-exp's error more
        ref = R.cross_attn_bwd(q, kc, vc, dy, n, None, bo, operand + 1.05 * float(bl.max()), R.step(dt))
        for key, (r, e) in ref.items():
            within(got[key], r, e + 1e-30, key)


def test_cross_attn_gradient_against_differences(cuda_ok):
    """float32: the forward's own central difference along a direction.  With step h the difference has curvature
    terms of h^2 / 6 of the third derivative: h moves a score by at most 0.01 sum_c |k_c| / 8, about 0.06, so they stay
    below 0.06^2 of the gradient times a small number; the forward's errors of 1e-6 over 2 h add less than 1e-3 of it."""
    op, q, k, v, n, _, dt = x_case(X[-3], 10, poison=False)
    dy = rnd(gen(11), *q.shape)
    y = op(q, k, v, n)
    got = op.backward(q, k, v, y, op.lse.clone(), dy, n)
    h = 1e-2
    f = lambda q_, k_, v_: float((CrossAttention(*op.shape[:2], k.shape[1], op.shape[2], k.shape[2], op.shape[3], dtype="f32")  # noqa: E731
                                  (q_, k_, v_, n).double() * dy.double()).sum())
    for i, key in enumerate(("dq", "dk", "dv")):
        x = [q, k.contiguous(), v.contiguous()]
        d = got[key].sign()  # the steepest direction of this size: the difference is the gradient's sum of |.|
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + h * d, x[i] - h * d
        want = (f(*up) - f(*dn)) / (2 * h)
        assert abs(want - float(got[key].double().abs().sum())) <= 0.02 * abs(want), key


def test_cross_attn_is_the_same_on_every_run(cuda_ok):
    for case in (X[1], X[9], X[10]):
        op, q, k, v, n, _, dt = x_case(case, 12)
        dy = rnd(gen(13), *q.shape, dtype=dt)
        y = op(q, k, v, n)
        lse = op.lse.clone()
        g = op.backward(q, k, v, y, lse, dy, n)
        for _ in range(3):
            assert torch.equal(y, op(q, k, v, n))
            h = op.backward(q, k, v, y, lse, dy, n)
            assert all(torch.equal(g[key], h[key]) for key in g)


def test_cross_attn_matches_the_text_cross_attention(cuda_ok):
    """Same numbers as the framework's uniform text cross-attention, within both kernels' bounds."""
    g = gen(14)
    B, T, N, H, d, Lt = 2, 3, 50, 4, 64, 77
    q, k, v = (rnd(g, B, t, H, d, dtype=torch.bfloat16) for t in (T * N, Lt, Lt))
    op = CrossAttention(B, T * N, Lt, H, H, d, keep_lse=True)
    y = op(q, k, v)
    cfg = L.HybridCfg(B=B, T=T, N=N, H=H, d_k=d, d_v=d, L=Lt, dtype=L.VDN_BF16)
    y2 = torch.empty(B, T, N, H, d, device="cuda")
    args = L.make_args(q, None, None, None, None, None, None, y2, torch.zeros(256, dtype=torch.uint8, device="cuda"), text_k=k, text_v=v)
    L.vdn_text_cross_attn(cfg, args)
    want, _ = R.cross_attn(q, k, v)
    bo, _ = R.cross_attn_bound(q, k, v, want, None, None, R.step(torch.bfloat16), R.step(torch.bfloat16))
    within(y, want, bo, "y")
    within(y2.view(y.shape), want, bo, "text")


def test_cross_attn_refusals(cuda_ok):
    op, q, k, v, n, _, _ = x_case(X[8], 15)
    dy, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    for bad in ((q.float(), k, v, n), (q[:, :-1], k, v, n), (q.transpose(1, 2), k, v, n), (q, k[:, :, :1], v, n), (q, k, v[:, ::2], n),
                (q, k, v.transpose(1, 2), n), (q, k, v, n.long()), (q, k, v, n[:1]), (q, k, v, n.cpu()), (q.cpu(), k, v, n)):
        with pytest.raises((ValueError, TypeError)):
            op(*bad)
        with pytest.raises((ValueError, TypeError)):
            op.backward(bad[0], bad[1], bad[2], q, lse, dy, bad[3])
    with pytest.raises(ValueError):
        op(q, k, v, n, out=torch.empty_like(q).float())
    for bad in ((None, k, v), (q, None, v), (q, k, None)):
        with pytest.raises(TypeError):
            op(*bad)
    for kw in (dict(y=q.float()), dict(lse=lse.double()), dict(dy=dy[:1]), dict(y=None), dict(lse=None), dict(dy=None)):
        a = {**dict(y=q, lse=lse, dy=dy), **kw}
        with pytest.raises((ValueError, TypeError)):
            op.backward(q, k, v, a["y"], a["lse"], a["dy"], n)
    for shape in ((0, 1, 1, 1, 1, 64), (1, 1, 1, 3, 2, 64), (1, 1, 1, 1, 1, 48)):
        with pytest.raises(L.VdnError):
            CrossAttention(*shape)


# ------------------------------------------------------------ 8-bit layer
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (7, 48), (33, 1024), (5, 1040), (3, 6144), (2, 16384), (300, 784)])
def test_quantize_int8(cuda_ok, rows, cols, dtype):
    g = gen(20)
    x = rnd(g, rows, cols, dtype=DT[dtype]) * torch.exp2(torch.randint(-30, 30, (rows, 1), device="cuda", generator=g)).to(DT[dtype])
    x[0, : cols // 2] = x[0].abs().max() / 2  # quotients of 63.5 up to the scale's rounding
    q, s = quantize_int8(x)
    qr, sr = R.quantize_int8(x)
    assert torch.equal(s, sr) and torch.equal(q, qr)


def test_quantize_int8_edges(cuda_ok):
    big = torch.finfo(torch.float32).max
    x = torch.zeros(10, 32, device="cuda")
    x[1, 3] = 2.0 ** -120  # counts as zero
    x[2, 3], x[2, 4] = 2.0 ** -119, -(2.0 ** -126)
    x[3, 0], x[3, 1] = big, -big / 2
    x[4, 0], x[4, 1] = math.inf, 1
    x[5, 0], x[5, 1] = 1, math.nan
    x[6] = -3.0
    x[7, 0], x[7, 1:] = 127, torch.arange(1, 32, device="cuda") + 0.5  # ties: half to even
    x[8, 0], x[8, 1] = -127, 0.5
    x[9, 5] = 1e-45
    q, s = quantize_int8(x)
    qr, sr = R.quantize_int8(x)
    assert torch.equal(q, qr) and torch.equal(torch.nan_to_num(s, 9.0), torch.nan_to_num(sr, 9.0))


I8 = [(1, 16, 16), (1, 6144, 4096), (2, 64, 48), (3, 8192, 80), (8, 1280, 784), (9, 1280, 784), (8, 32768, 32), (64, 16, 16), (127, 112, 272),
      (128, 128, 128), (237, 1280, 784), (257, 4096, 256), (300, 144, 1040), (1000, 6144, 400), (5, 131056, 16), (40, 131056, 32)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("M,K,N", I8, ids=str)
def test_linear_int8(cuda_ok, M, K, N, dtype, out):
    g = gen(21)
    w, ws = quantize_int8(rnd(g, N, K, scale=K ** -0.5))
    bias = rnd(g, N) if (M + N) % 2 else None
    op = Int8Linear(w, ws, bias, out_dtype=out)
    room = torch.full((M * N + 256,), 7.0, device="cuda", dtype=DT[out])
    y = room[:M * N].view(M, N)
    if dtype == "i8":
        codes = torch.randint(-128, 128, (M, K), device="cuda", generator=g, dtype=torch.int8)
        xs = torch.rand(M, device="cuda", generator=g) + 0.1
        op(codes, xs, out=y)
    else:
        x = rnd(g, M, K, dtype=DT[dtype])
        codes, xs = R.quantize_int8(x)
        op(x, out=y)
    assert L.vdn_proj_device_status()[0] == L.VDN_OK
    want = R.linear_int8(codes, xs, w, ws, bias)
    # one rounding of the exact sum to 32 bits and of each product with a scale, one of the bias's sum
    size = want.abs() + (0 if bias is None else 2 * bias.abs())
    within(y, want, (R.step(DT[out]) + 8 * R.EPS) * size, "out")
    assert bool((room[M * N:] == 7.0).all())


def test_linear_int8_extreme_codes(cuda_ok):
    """The largest sums the layer allows: -128 x -128 x 131056 stays inside 32 bits."""
    for M in (2, 64):
        K, N = 131056, 16
        codes = torch.full((M, K), -128, device="cuda", dtype=torch.int8)
        one = torch.ones(N, device="cuda")
        y = Int8Linear(codes[:1].expand(N, K).contiguous(), one, None, out_dtype="f32")(codes, torch.ones(M, device="cuda"))
        assert bool((y == float(128 * 128 * K)).all())


def test_linear_int8_leading_axes_bad_rows(cuda_ok):
    g = gen(22)
    w, ws = quantize_int8(rnd(g, 48, 64))
    op = Int8Linear(w, ws, None, out_dtype="f32")
    for shape in ((2, 3), (10, 7)):
        x = rnd(g, *shape, 64)
        x[1, 2, 5] = math.nan
        x[0, 1] = 0
        y = op(x)
        assert y.shape == (*shape, 48) and bool(torch.isnan(y[1, 2]).all()) and bool((y[0, 1] == 0).all())
        y[1, 2] = 0
        assert bool(torch.isfinite(y).all())


def test_linear_int8_refusals(cuda_ok):
    g = gen(23)
    w, ws = quantize_int8(rnd(g, 48, 64))
    op = Int8Linear(w, ws)
    x = rnd(g, 4, 64)
    for bad in (x[:, :48], x.t(), x.cpu(), x.half()):
        with pytest.raises((ValueError, TypeError)):
            op(bad)
    with pytest.raises(L.VdnError):
        op(x, torch.ones(4, device="cuda"))  # scales without codes
    with pytest.raises(L.VdnError):
        op(torch.zeros(4, 64, device="cuda", dtype=torch.int8))  # codes without scales
    with pytest.raises(ValueError):
        Int8Linear(w, ws.double())
    with pytest.raises(ValueError):
        Int8Linear(w.float(), ws)
    with pytest.raises(ValueError):
        quantize_int8(x.t())
    with pytest.raises(TypeError):
        quantize_int8(x.half())


# ---------------------------------------------------------- 16-byte alignment
def shifted(t):
    """A copy of t that starts 16 bytes behind a 256-byte boundary."""
    off = 16 // t.element_size()
    room = torch.zeros(t.numel() + off, device="cuda", dtype=t.dtype)
    out = room[off:].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


@pytest.mark.parametrize("case", [X[1], X[3], X[9], X[-3], X[10]], ids=str)
def test_cross_attn_sixteen_byte_alignment(cuda_ok, case):
    """Every tensor at an address of 16 mod 32: the same bits as aligned ones, forward and backward."""
    op, q, k, v, n, _, dt = x_case(case, 60)
    k, v, dy = k.contiguous(), v.contiguous(), rnd(gen(61), *q.shape, dtype=dt)
    y = op(q, k, v, n).clone()
    lse = op.lse.clone()
    y2 = op(shifted(q), shifted(k), shifted(v), n, out=shifted(y))
    assert torch.equal(y, y2) and torch.equal(lse, op.lse)
    g = op.backward(q, k, v, y, lse, dy, n)
    h = op.backward(shifted(q), shifted(k), shifted(v), shifted(y), lse, shifted(dy), n)
    assert all(torch.equal(g[key], h[key]) for key in g)


def test_others_sixteen_byte_alignment(cuda_ok):
    op, a, _, _ = qk_case(QK[5], 62, skip=False)
    q, k = a["q"].contiguous(), a["k"].contiguous()
    rest = (a["wq"], a["wk"], a["table"], a["pos"])
    want = op(q, k, *rest)
    got = op(shifted(q), shifted(k), a["wq"], a["wk"], shifted(a["table"]), a["pos"], out=(shifted(q), shifted(k)))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    g = gen(63)
    w, ws = quantize_int8(rnd(g, 272, 1040))
    b = rnd(g, 272)
    for M in (1, 5, 200):
        x = rnd(g, M, 1040, dtype=torch.bfloat16)
        y = Int8Linear(w, ws, b)(x)
        assert torch.equal(y, Int8Linear(shifted(w), shifted(ws), shifted(b))(shifted(x), out=shifted(y)))


# ------------------------------------------------- together, streams, graphs
class Layer:
    """Projection -> norm and rotation -> cross-attention -> 8-bit output layer."""

    def __init__(self, B, T, Lk, H, Hkv, d, N, seed):
        g = gen(seed)
        self.x = rnd(g, B, T, H + 2, d, dtype=torch.bfloat16)  # packed: queries and something else
        self.kv = rnd(g, B, Lk, 2, Hkv, d, dtype=torch.bfloat16)
        self.n = torch.tensor([Lk, Lk // 3][:B], device="cuda", dtype=torch.int32)
        self.wq, self.wk = 1 + rnd(g, d, scale=0.2), 1 + rnd(g, d, scale=0.2)
        self.table = rope_table(max(T, Lk), (d // 2,))
        self.pos_q = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)
        self.pos_k = torch.arange(Lk, device="cuda", dtype=torch.int32).repeat(B, 1)
        self.nq, self.nk = QKNormRope(H, 0, d), QKNormRope(Hkv, 0, d)
        self.attn = CrossAttention(B, T, Lk, H, Hkv, d, keep_lse=True)
        self.w = rnd(g, N, H * d, scale=(H * d) ** -0.5)
        self.out = Int8Linear(*quantize_int8(self.w), None, out_dtype="f32")
        self.B, self.T, self.H, self.d, self.Hkv = B, T, H, d, Hkv

    def forward(self, stream=None):
        q, _ = self.nq(self.x[:, :, :self.H], None, self.wq, None, self.table, self.pos_q, stream=stream)
        k, _ = self.nk(self.kv[:, :, 0], None, self.wk, None, self.table, self.pos_k, stream=stream)
        y = self.attn(q, k, self.kv[:, :, 1], self.n, stream=stream)
        return q, k, y, self.out(y.view(self.B, self.T, self.H * self.d), stream=stream)

    def backward(self, q, k, y, dy, stream=None):
        g = self.attn.backward(q, k, self.kv[:, :, 1], y, self.attn.lse, dy, self.n, stream=stream)
        a = self.nq.backward(self.x[:, :, :self.H], None, self.wq, None, self.table, g["dq"], None, self.pos_q, stream=stream)
        b = self.nk.backward(self.kv[:, :, 0], None, self.wk, None, self.table, g["dk"], None, self.pos_k, stream=stream)
        return {"dx": a["dq"], "dwq": a["dwq"], "dk": b["dq"], "dwk": b["dwq"], "dv": g["dv"]}


def layer_reference(m, dy):
    """The layer in float64 through autograd, up to the attention's output."""
    x = m.x[:, :, :m.H].double().requires_grad_()
    kx, v = m.kv[:, :, 0].double().requires_grad_(), m.kv[:, :, 1].double().requires_grad_()
    wq, wk = m.wq.double().requires_grad_(), m.wk.double().requires_grad_()

    def turn(z, w, pos):
        z = z / (z.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        c = m.table.double()[pos.long()].unsqueeze(2)
        a, b = z[..., 0::2], z[..., 1::2]
        return torch.stack([a * c[..., 0] - b * c[..., 1], a * c[..., 1] + b * c[..., 0]], -1).flatten(-2)

    q, k = turn(x, wq, m.pos_q), turn(kx, wk, m.pos_k)
    G = m.H // m.Hkv
    z = torch.einsum("bthd,blhd->bhtl", q, k.repeat_interleave(G, 2)) / math.sqrt(m.d)
    z = z.masked_fill(torch.arange(k.shape[1], device="cuda").view(1, 1, 1, -1) >= m.n.view(-1, 1, 1, 1), -math.inf)
    y = torch.einsum("bhtl,blhd->bthd", torch.softmax(z, -1), v.repeat_interleave(G, 2))
    grads = torch.autograd.grad((y * dy.double()).sum(), [x, wq, kx, wk, v])
    return y.detach(), dict(zip(("dx", "dwq", "dk", "dwk", "dv"), grads))


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_layer_run_together(cuda_ok):
    """Forward and backward through the chain.  Every stage rounds its tensors to bf16 (relative 2^-8 at most, about
    2^-9.8 in the 2-norm): four such roundings in the forward, six on the way back, amplified by scores of a few
    units: 2^-5 holds them with room."""
    m = Layer(2, 300, 200, 4, 2, 64, 80, 30)
    q, k, y, out = m.forward()
    dy = rnd(gen(31), *y.shape, dtype=torch.bfloat16)
    got = m.backward(q, k, y, dy)
    yr, want = layer_reference(m, dy)
    assert rel(y, yr) < 2 ** -5
    for key, r in want.items():
        assert rel(got[key], r) < 2 ** -5, key
    # the 8-bit layer: a code is off by half a step of amax / 127, about 2^-7 of a row's 2-norm, in x and in w
    assert rel(out, yr.reshape(2, 300, -1) @ m.w.double().t()) < 2 ** -4


def test_layer_on_streams_of_their_own(cuda_ok):
    """Two layers at once on two streams that are not the current one give what each gives alone."""
    ms = [Layer(2, 260, 150, 4, 2, 64, 80, 32), Layer(1, 1, 2000, 8, 2, 128, 48, 33)]
    want = [[t.clone() for t in m.forward()] for m in ms]
    dys = [rnd(gen(34 + i), *w[2].shape, dtype=torch.bfloat16) for i, w in enumerate(want)]
    grads = [m.backward(*w[:3], dy) for m, w, dy in zip(ms, want, dys)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in ms]
    for _ in range(3):
        got, back = [], []
        for m, s, dy in zip(ms, ss, dys):
            got.append(m.forward(stream=s))
            back.append(m.backward(*got[-1][:3], dy, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, z) for x, z in zip(a, b))
        for a, b in zip(grads, back):
            assert all(torch.equal(a[key], b[key]) for key in a)


def test_layer_captured_into_graphs(cuda_ok):
    """Two captured layers, replayed by turns and with new inputs, and an eager call between."""
    ms = [Layer(2, 140, 100, 4, 2, 64, 80, 36), Layer(1, 3, 900, 4, 1, 128, 48, 37)]
    dys = [rnd(gen(38 + i), m.B, m.T, m.H, m.d, dtype=torch.bfloat16) for i, m in enumerate(ms)]
    graphs, outs = [], []
    s = torch.cuda.Stream()
    for m, dy in zip(ms, dys):
        with torch.cuda.stream(s):
            r = m.forward()
            m.backward(*r[:3], dy)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            r = m.forward()
            b = m.backward(*r[:3], dy)
        graphs.append(gr)
        outs.append((r, b))
    for turn in range(3):
        for i, m in enumerate(ms):
            m.x.copy_(rnd(gen(40 + turn), *m.x.shape, dtype=torch.bfloat16))
            m.n.clamp_(max=m.kv.shape[1] - 7 * turn)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        kept = [([t.clone() for t in r], {k: t.clone() for k, t in b.items()}) for r, b in outs]
        for i, m in enumerate(ms):
            r = m.forward()
            b = m.backward(*r[:3], dys[i])
            assert all(torch.equal(x, z) for x, z in zip(kept[i][0], r))
            assert all(torch.equal(kept[i][1][k], b[k]) for k in b)


def test_offsets_past_31_bits(cuda_ok):
    """Tensors of more than 2^31 elements: the last rows are computed like the first."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    g = gen(50)
    T = (2 ** 31 + 2 ** 20) // (24 * 128)
    last = 700
    x = torch.zeros(T, 24, 128, device="cuda", dtype=torch.bfloat16)
    x[-last:] = rnd(g, last, 24, 128, dtype=torch.bfloat16)
    table = rope_table(T, (64,))
    op = QKNormRope(24, 0, 128)
    y, _ = op(x, None, None, None, table)
    pos = torch.arange(last, device="cuda", dtype=torch.int32)
    y2, _ = op(x[-last:], None, None, None, table[-last:].contiguous(), pos)
    assert torch.equal(y[-last:], y2)
    k = rnd(g, 1, 200, 24, 128, dtype=torch.bfloat16)
    a = CrossAttention(1, T, 200, 24, 24, 128)(y.unsqueeze(0), k, k)
    b = CrossAttention(1, last, 200, 24, 24, 128)(y2.unsqueeze(0), k, k)
    assert torch.equal(a[0, -last:], b[0])
