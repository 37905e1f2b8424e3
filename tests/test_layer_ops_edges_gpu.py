"""The layer's operators where their kernels change regime: several items of a
persistent kernel on one SM, every tile shape of the 8-bit product, rows past
2^31 elements, sizes next to 2^31, and what a call leaves in rows that it has
nothing to compute for."""
import gc
import math

import pytest
import torch

from oracle import layer_oracle as R
from test_layer_ops_gpu import DT, QK, X, gen, qk_case, rnd, within, x_case, x_forward_check, x_grads, x_status
from video_diffusion_hybrid_b200 import _lib as L
from video_diffusion_hybrid_b200.api import CrossAttention, Int8Linear, QKNormRope, quantize_int8, rope_table
from video_diffusion_hybrid_b200.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if torch.cuda.is_available():
        build()


@pytest.fixture
def room_for(cuda_ok):
    """room_for(n) skips below n GB of free memory; what the test had goes back at its end, before anything small that
    stays (a library's workspace) comes to lie in it."""
    def free():
        gc.collect()  # what a refused call's traceback holds
        torch.cuda.empty_cache()

    def need(gigabytes):
        free()
        if torch.cuda.mem_get_info()[0] < gigabytes << 30:
            pytest.skip(f"needs {gigabytes} GB")

    yield need
    free()


# ------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("case", [c for c in QK if c[0] > 8], ids=str)
def test_qk_skipped_rows_of_new_outputs_are_zero(cuda_ok, case):
    """Without `out` there is nothing to leave a skipped token's rows as: they are zeros, whatever the memory held."""
    op, a, on, dt = qk_case(case, 3)
    want = tuple(None if a[k] is None else torch.zeros(a[k].shape, device="cuda", dtype=dt) for k in "qk")
    op(a["q"], a["k"], a["wq"], a["wk"], a["table"], a["pos"], out=want)
    torch.cuda.synchronize()
    stale = [torch.full(a[k].shape, math.nan, device="cuda", dtype=dt) for k in "qk" if a[k] is not None for _ in range(3)]
    del stale  # the blocks that the call's outputs come from
    got = op(a["q"], a["k"], a["wq"], a["wk"], a["table"], a["pos"])
    for g, w in zip(got, want):
        assert (g is None and w is None) or (torch.equal(g, w) and bool((g[~on] == 0).all()))


@pytest.mark.parametrize("case", [(468, 24, 8, 24, 0, (0, 0, 0), "interleaved", "f32", False, False),
                                  (36, 5, 3, 128, 0, (0,), "split", "bf16", True, True)], ids=str)
def test_qk_norm_alone_takes_every_position(cuda_ok, case):
    """Without a rotation there is no table: a negative position skips a token, 2^31 - 1 does not."""
    op, a, on, dt = qk_case(case, 4)
    assert bool((a["pos"][-1] == 2 ** 31 - 1).any()) and bool(on[-1]) and not bool(on[3])
    out = tuple(torch.full(a[k].shape, 7.0, device="cuda", dtype=dt) for k in "qk")
    op(a["q"], a["k"], a["wq"], a["wk"], None, a["pos"], out=out)
    for key, t in zip("qk", out):
        want = R.qk_norm_rope(a[key], a["w" + key], None, None, 0, case[6], op.sections, 1e-6)
        within(t[on], want[on], R.step(dt) * want[on].abs() + 24 * R.EPS * want[on].abs().amax(-1, keepdim=True) * 2, key)
        assert bool((t[~on] == 7.0).all())


@pytest.mark.parametrize("gdtype", ["f32", "bf16"])
def test_qk_backward_of_index_positions_and_unit_weights(cuda_ok, gdtype):
    for case in (QK[3], QK[2]):
        if case[7] == "f32" and gdtype == "bf16":
            continue
        op, a, _, dt = qk_case((case[0], *case[1:5], (case[4] // 2,), *case[6:]), 8, skip=False)
        table = rope_table(case[0] + 3, (case[4] // 2,))
        g = gen(9)
        up = {k: rnd(g, *a[k].shape, dtype=DT[gdtype]) for k in "qk"}
        got = op.backward(a["q"], a["k"], None, None, table, up["q"], up["k"])
        p = torch.arange(case[0], device="cuda", dtype=torch.int32).unsqueeze(1)
        for k in "qk":
            dx, dw, scale, terms = R.qk_norm_rope_bwd(a[k], None, table, p, op.rot, case[6], op.sections, 1e-6, up[k])
            within(got["d" + k], dx, R.step(dt) * dx.abs() + 64 * R.EPS * scale, "d" + k)
            if not op.per_head:
                dw, terms = dw.sum(0), terms.sum(0)
            n = case[0] * (1 if op.per_head else a[k].shape[1])
            within(got["dw" + k], dw, (n + 64) * R.EPS * terms + 1e-30, "dw" + k)


def test_qk_tokens_next_to_31_bits(room_for):
    """2^31 - 1 tokens, the largest number: the last ones are computed like a few on their own."""
    room_for(130)
    T, last, g = 2 ** 31 - 1, 1000, gen(51)
    op = QKNormRope(1, 0, 8, rot=0, sections=(0,))
    x = torch.zeros(T, 1, 8, device="cuda", dtype=torch.bfloat16)
    x[-last:] = rnd(g, last, 1, 8, dtype=torch.bfloat16)
    y, _ = op(x, None)
    assert torch.equal(y[-last:], op(x[-last:], None)[0])
    y.zero_()
    y[-last:] = rnd(g, last, 1, 8, dtype=torch.bfloat16)
    a = op.backward(x, None, None, None, None, y, None)
    b = op.backward(x[-last:], None, None, None, None, y[-last:], None)
    assert torch.equal(a["dq"][-last:], b["dq"])


def test_qk_more_tokens_than_32_bits_are_refused(room_for):
    """2^32 + 5 tokens would be 5 of them in a 32-bit count."""
    room_for(75)
    with pytest.raises(ValueError):
        QKNormRope(1, 0, 8, rot=0, sections=(0,))(torch.empty(2 ** 32 + 5, 1, 8, device="cuda", dtype=torch.bfloat16), None)


# --------------------------------------------------------- cross-attention
WIDE = [  # more items than SMs, so that a CTA goes on from one to the next: in the forward and dq, and mostly in dk and dv
    (3, 1500, 700, 24, 24, 64, "bf16", [700, 0, 300], True),
    (3, 1500, 700, 24, 8, 128, "bf16", [300, 700, 0], True),
    (4, 1700, 515, 30, 10, 64, "bf16", [515, 0, 129, 1], False),   # heads of a group share tiles of 126 rows
    (5, 1100, 260, 24, 24, 128, "bf16", [0, 260, 0, 128, 7], True),  # empty batch elements between
    (2, 100, 8192, 40, 40, 64, "bf16", [8192, 3001], False),       # states split, more than one item a CTA
    (2, 256, 8192, 40, 20, 128, "bf16", [3000, 8191], True),
    (2, 6000, 600, 20, 10, 64, "bf16", [600, 385], False),         # query rows split in dk and dv
    (2, 6000, 600, 20, 10, 128, "bf16", [511, 600], True),
]


@pytest.mark.parametrize("case", WIDE, ids=str)
def test_cross_attn_many_items(cuda_ok, case):
    op, q, k, v, n, clean, dt = x_case(case, 90)
    assert L.vdn_cross_attn_impl(op.cfg) == 1
    y = op(q, k, v, n)
    x_status(op)
    x_forward_check(op, q, *clean, n, dt, y)
    assert all(torch.equal(y, op(q, k, v, n)) for _ in range(3))


@pytest.mark.parametrize("case", WIDE, ids=str)
def test_cross_attn_backward_many_items(cuda_ok, case):
    op, q, k, v, n, clean, dt = x_case(case, 91)
    assert L.vdn_cross_attn_impl(op.cfg, True) == 1
    got = x_grads(op, q, k, v, n, clean, dt, 92)
    for b, m in enumerate(case[7]):
        assert bool((got["dk"][b, m:] == 0).all()) and bool((got["dv"][b, m:] == 0).all())
        assert m > 0 or bool((got["dq"][b] == 0).all())


@pytest.mark.parametrize("case", [X[9], X[3], X[-3], X[-1], X[13]], ids=str)
def test_cross_attn_no_gradient_past_the_length_of_a_bad_row(cuda_ok, case):
    """A NaN or an infinity in the incoming gradient reaches the states of its batch element, not those past the length."""
    op, q, k, v, n, _, dt = x_case(case, 93)
    dy = rnd(gen(94), *q.shape, dtype=dt)
    dy[:, 0, 0, 3], dy[:, -1, -1, 1] = math.nan, math.inf
    y = op(q, k, v, n)
    got = op.backward(q, k, v, y, op.lse, dy, n)
    for b, m in enumerate(case[7]):
        m = min(max(m, 0), k.shape[1])
        for key in ("dk", "dv"):
            assert bool((got[key][b, m:] == 0).all()), (key, b)
            assert m == 0 or not bool(torch.isfinite(got[key][b, :m]).all())


def test_cross_attn_log_sum_exp_of_each_forward(cuda_ok):
    """Two forwards before the first backward (micro-batches): each call's log-sum-exp stays its own."""
    op, q, k, v, n, _, dt = x_case(X[9], 95)
    q2, dy = rnd(gen(96), *q.shape, dtype=dt, scale=3.0), rnd(gen(97), *q.shape, dtype=dt)
    y = op(q, k, v, n)
    lse = op.lse
    kept = lse.clone()
    want = op.backward(q, k, v, y, lse, dy, n)
    op(q2, k, v, n)
    assert torch.equal(lse, kept) and not torch.equal(op.lse, kept)
    got = op.backward(q, k, v, y, lse, dy, n)
    assert all(torch.equal(want[key], got[key]) for key in want)


def test_cross_attn_backward_offsets_past_31_bits(room_for):
    """More than 2^31 elements of q: the last rows' dq like that of the rows alone; the other rows have no gradient, so dk
    and dv are the last rows' too, up to the order of their sums (a step of bf16 in the 2-norm)."""
    room_for(60)
    g, T, last = gen(52), (2 ** 31 + 2 ** 20) // (24 * 128), 700
    q, dy = (torch.zeros(1, T, 24, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q[:, -last:], dy[:, -last:] = (rnd(g, 1, last, 24, 128, dtype=torch.bfloat16) for _ in range(2))
    k, v = (rnd(g, 1, 200, 24, 128, dtype=torch.bfloat16) for _ in range(2))
    big, few = CrossAttention(1, T, 200, 24, 24, 128, keep_lse=True), CrossAttention(1, last, 200, 24, 24, 128, keep_lse=True)
    y = big(q, k, v)
    a = big.backward(q, k, v, y, big.lse, dy)
    qt, yt, dt = (t[:, -last:].contiguous() for t in (q, y, dy))
    assert torch.equal(few(qt, k, v), yt)
    b = few.backward(qt, k, v, yt, few.lse, dt)
    assert torch.equal(a["dq"][:, -last:], b["dq"]) and bool((a["dq"][:, :1000] == 0).all())
    for key in ("dk", "dv"):
        x, z = a[key].double(), b[key].double()
        assert float((x - z).norm()) <= 2 ** -8 * float(z.norm()), key


@pytest.mark.parametrize("Tq,d,Hkv,dtype", [(1, 128, 8, "bf16"), (40, 128, 8, "bf16"), (3, 64, 16, "f32")], ids=str)
def test_cross_attn_states_past_31_bits(room_for, Tq, d, Hkv, dtype):
    """Packed states of more than 2^32 elements, gradients of more than 2^31.  All states but the last 700 are zeros: they
    weigh 1 each and add nothing, so that the last 700 give the output and the gradients.  Tolerance in the 2-norm: y, P and
    dS rounded to bf16 (a step of 2^-8 each at most, and Delta of a y rounded so), or a million fp32 sums."""
    room_for(60)
    g, dt, L_, last = gen(55), DT[dtype], 2 ** 20 + 77, 700
    kv = torch.zeros(2, L_, 2, Hkv, d, device="cuda", dtype=dt)
    kv[:, -last:] = rnd(g, 2, last, 2, Hkv, d, dtype=dt)
    q, dy = (rnd(g, 2, Tq, Hkv, d, dtype=dt) for _ in range(2))
    scale = 0.5
    op = CrossAttention(2, Tq, L_, Hkv, Hkv, d, dtype=dtype, scale=scale, keep_lse=True)
    k, v = kv[:, :, 0], kv[:, :, 1]
    y = op(q, k, v)
    assert op.status() == (L.VDN_OK, 0)
    kd, vd, qd, gd = (t.double() for t in (k[:, -last:], v[:, -last:], q, dy))
    s = scale * torch.einsum("bthd,blhd->bhtl", qd, kd)
    top = s.amax(-1, keepdim=True).clamp_min(0)
    z = torch.exp(s - top).sum(-1, keepdim=True) + (L_ - last) * torch.exp(-top)
    p = torch.exp(s - top) / z
    want = torch.einsum("bhtl,blhd->bthd", p, vd)
    tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -14
    near = lambda a, b, what: float((a.double() - b).norm()) <= tol * float(b.norm()) or pytest.fail(what)  # noqa: E731
    near(y, want, "y")
    near(op.lse, (top + z.log()).squeeze(-1).transpose(1, 2), "lse")
    got = op.backward(q, k, v, y, op.lse, dy)
    assert op.status(backward=True) == (L.VDN_OK, 0)
    ds = p * (torch.einsum("bthd,blhd->bhtl", gd, vd) - (gd * want).sum(-1).transpose(1, 2).unsqueeze(-1))
    near(got["dq"], scale * torch.einsum("bhtl,blhd->bthd", ds, kd), "dq")
    near(got["dk"][:, -last:], scale * torch.einsum("bhtl,bthd->blhd", ds, qd), "dk")
    near(got["dv"][:, -last:], torch.einsum("bhtl,bthd->blhd", p, gd), "dv")
    # a zero state's weight is exp(-lse)
    w = torch.exp(-(top + z.log())).squeeze(-1)
    near(got["dv"][:, 5], torch.einsum("bht,bthd->bhd", w, gd), "dv of a zero state")


# ------------------------------------------------------------ 8-bit layer
TILES = [  # M, K, N, columns of a tile: the CTA pairs with more tiles than pairs, and with fewer; one-CTA tiles, several
    (5000, 208, 1040, 256), (4999, 6160, 1040, 256), (20000, 48, 272, 256), (1500, 400, 2032, 256), (1000, 1296, 784, 64),
    (700, 272, 2000, 64), (1008, 6144, 1024, 64), (300, 144, 1040, 32), (513, 400, 512, 32),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("M,K,N,columns", TILES, ids=str)
def test_linear_int8_tiles(cuda_ok, M, K, N, columns, dtype, out):
    assert L.vdn_linear_int8_impl(L.Int8Cfg(M, K, N, L.VDN_I8, L.VDN_F32)) == columns
    g = gen(24)
    w, ws = quantize_int8(rnd(g, N, K, scale=K ** -0.5))
    bias = rnd(g, N) if M % 2 else None
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
    size = want.abs() + (0 if bias is None else 2 * bias.abs())
    within(y, want, (R.step(DT[out]) + 8 * R.EPS) * size, "out")
    assert bool((room[M * N:] == 7.0).all())


@pytest.mark.parametrize("M", [1, 4, 8, 200, 1000, 5000])
def test_linear_int8_large_scales(cuda_ok, M):
    """Rows of values near the type's largest against a weight that brings them back: no product on the way passes what
    the output can hold.  And small rows against large weights."""
    g = gen(25)
    K, N = 256, 1040
    for up, down in ((2.0 ** 124, 2.0 ** -40), (2.0 ** -100, 2.0 ** 110)):
        w, ws = quantize_int8(rnd(g, N, K, scale=down))
        x = rnd(g, M, K, scale=up)
        codes, xs = R.quantize_int8(x)
        y = Int8Linear(w, ws, None, out_dtype="f32")(x)
        want = R.linear_int8(codes, xs, w, ws, None)
        within(y, want, 8 * R.EPS * want.abs(), "out")


def test_linear_int8_offsets_past_31_bits(room_for):
    """More than 2^31 elements of x and of the output: the last rows like those rows alone."""
    room_for(40)
    g, M, K, last = gen(53), 360000, 6144, 300
    w, ws = quantize_int8(rnd(g, K, K, scale=K ** -0.5))
    op = Int8Linear(w, ws)
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    x[-last:] = rnd(g, last, K, dtype=torch.bfloat16)
    y = op(x)
    assert torch.equal(y[-last:], op(x[-last:])) and bool((y[:1000] == 0).all())
    q, s = quantize_int8(x)
    qt, st = quantize_int8(x[-last:])
    assert torch.equal(q[-last:], qt) and torch.equal(s[-last:], st)


def test_int8_rows_next_to_31_bits(room_for):
    """2^31 - 1 rows, the largest number, of 16 columns: codes and scales of the last ones, and their outputs."""
    room_for(130)
    g, M, last = gen(54), 2 ** 31 - 1, 1000
    x = torch.zeros(M, 16, device="cuda", dtype=torch.bfloat16)
    x[-last:] = rnd(g, last, 16, dtype=torch.bfloat16)
    tail = x[-last:].clone()
    q, s = quantize_int8(x)
    del x
    qt, st = quantize_int8(tail)
    assert torch.equal(q[-last:], qt) and torch.equal(s[-last:], st)
    w, ws = quantize_int8(rnd(g, 16, 16))
    torch.cuda.empty_cache()
    op = Int8Linear(w, ws)
    assert torch.equal(op(q, s)[-last:], op(qt, st))


def test_many_sizes_leave_no_trace(cuda_ok):
    """A user with another number of rows on every call: the objects do not grow with the numbers seen."""
    g = gen(26)
    w, ws = quantize_int8(rnd(g, 32, 32))
    lin, norm = Int8Linear(w, ws), QKNormRope(1, 0, 16, rot=0, sections=(0,))
    kv = rnd(g, 1, 1, 64 * 2000, dtype=torch.bfloat16)
    attn = CrossAttention(1, 1, 2, 1, 1, 64)
    q = rnd(g, 1, 1, 1, 64, dtype=torch.bfloat16)
    for i in range(1, 700):
        lin(torch.zeros(i, 32, device="cuda"))
        norm(torch.zeros(i, 1, 16, device="cuda"), None)
        k = torch.as_strided(kv, (1, 2, 1, 64), (64 * 2000, 64 + 8 * i, 64, 1))
        attn(q, k, k)
    assert max(len(op._cfgs) for op in (lin, norm, attn)) <= 256
