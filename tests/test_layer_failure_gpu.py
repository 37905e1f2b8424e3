"""The failure path of the layer's operators, made to happen without a fault:
their bounded waits get a limit far below what a load or a product takes, so
that some role of every CTA gives up.  The call's status words say so, the
CTAs drain what they issued and end, and the next call of the same process,
with the default limit, gives the same bits as before.  The limits put the
give-up at different places: at the first loads, between two loads of an item,
in the middle of the walk over the items.
"""
import pytest
import torch

from video_diffusion_hybrid_b200 import _lib as L
from video_diffusion_hybrid_b200.api import CrossAttention, Int8Linear, quantize_int8
from video_diffusion_hybrid_b200.build import build

pytestmark = pytest.mark.gpu
LIMITS = [1, 300, 1000, 3000, 10000]


@pytest.fixture(scope="module", autouse=True)
def built():
    if torch.cuda.is_available():
        build()


def attention(d):
    """More items than SMs in every kernel, an empty batch element between full ones, a tile that ends early."""
    g = torch.Generator(device="cuda").manual_seed(d)
    B, Tq, Lk, H, Hkv = 3, 1500, 700, 12, 12
    q, dy = (torch.randn(B, Tq, H, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    k, v = (torch.randn(B, Lk, Hkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    n = torch.tensor([700, 0, 300], device="cuda", dtype=torch.int32)
    op = CrossAttention(B, Tq, Lk, H, Hkv, d, keep_lse=True)
    assert (L.vdn_cross_attn_impl(op.cfg), L.vdn_cross_attn_impl(op.cfg, True)) == (1, 1)
    return op, q, k, v, n, dy


def gave_up(call, status, limits, tag):
    """Runs `call` with each limit; the timeout is reported, under the kernel's tag, at the shortest at least."""
    seen = []
    torch.cuda.synchronize()
    for cycles in limits:
        L.vdn_debug_set_layer_wait_limit(cycles)
        try:
            call()
            seen.append(status())
            torch.cuda.synchronize()
        finally:
            L.vdn_debug_set_layer_wait_limit(0)
        assert seen[-1] in ((L.VDN_OK, 0), (L.VDN_ERR_TIMEOUT, tag)), (cycles, seen)
    assert seen[0][0] == L.VDN_ERR_TIMEOUT, seen


@pytest.mark.parametrize("d", [64, 128])
def test_cross_attn_backward_wait_runs_out(cuda_ok, d):
    op, q, k, v, n, dy = attention(d)
    y = op(q, k, v, n)
    lse = op.lse.clone()
    back = lambda: op.backward(q, k, v, y, lse, dy, n)  # noqa: E731
    want = back()
    assert op.status(backward=True) == (L.VDN_OK, 0)
    for _ in range(3):
        gave_up(back, lambda: op.status(backward=True), LIMITS, L.TAG_XATTN_BWD)
        got = back()
        assert op.status(backward=True) == (L.VDN_OK, 0)
        assert all(torch.equal(want[key], got[key]) for key in want)


@pytest.mark.parametrize("d", [64, 128])
def test_cross_attn_wait_runs_out(cuda_ok, d):
    op, q, k, v, n, _ = attention(d)
    want = op(q, k, v, n)
    lse = op.lse.clone()
    assert op.status() == (L.VDN_OK, 0)
    for _ in range(3):
        gave_up(lambda: op(q, k, v, n), op.status, LIMITS, L.TAG_XATTN)
        assert torch.equal(want, op(q, k, v, n)) and torch.equal(lse, op.lse)
        assert op.status() == (L.VDN_OK, 0)


@pytest.mark.parametrize("codes", [False, True])
def test_linear_int8_wait_runs_out_and_stays_on_record(cuda_ok, codes):
    """The timeout of one call is still there after calls on another stream, of many rows and of few."""
    g = torch.Generator(device="cuda").manual_seed(7)
    w, ws = quantize_int8(torch.randn(272, 1296, device="cuda", generator=g))
    x = torch.randn(300, 1296, device="cuda", generator=g)
    given = quantize_int8(x) if codes else (x,)
    one, two = Int8Linear(w, ws), Int8Linear(w, ws)
    others = [x.repeat(70, 1)[:rows] for rows in (300, 5, 20000)]  # each of the layer's kernels
    want = one(*given)
    torch.cuda.synchronize()
    assert one.status() == (L.VDN_OK, 0)
    for _ in range(3):
        gave_up(lambda: one(*given), one.status, LIMITS[:1], L.TAG_PROJ)
        s = torch.cuda.Stream()
        for other in others:
            two(other, stream=s)
            assert two.status(s) == (L.VDN_OK, 0)
        assert one.status() == (L.VDN_ERR_TIMEOUT, L.TAG_PROJ)
        assert torch.equal(want, one(*given)) and one.status() == (L.VDN_OK, 0)
        gave_up(lambda: one(*given), one.status, LIMITS, L.TAG_PROJ)
        assert torch.equal(want, one(*given)) and one.status() == (L.VDN_OK, 0)


def test_status_of_a_call_on_another_stream(cuda_ok):
    """status() without a stream waits for the call that it tells about: the words are not read before they are written
    (here the call starts a tenth of a second late, and the memory of its words holds something else)."""
    op, q, k, v, n, dy = attention(64)
    g = torch.Generator(device="cuda").manual_seed(8)
    w, ws = quantize_int8(torch.randn(272, 1296, device="cuda", generator=g))
    x = torch.randn(300, 1296, device="cuda", generator=g)
    y = op(q, k, v, n)
    lse = op.lse
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lin = Int8Linear(w, ws)
    for call, status in ((lambda: op(q, k, v, n, stream=s), op.status),
                         (lambda: op.backward(q, k, v, y, lse, dy, n, stream=s), lambda: op.status(backward=True)),
                         (lambda: lin(x, stream=s), lin.status)):
        call()  # the stream's allocations of these sizes exist now
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
                    for size in (op.need, op.bwd_need, 300 * 1296 + 4096) for _ in range(2)]
            del held
            torch.cuda._sleep(200_000_000)
        call()
        assert status() == (L.VDN_OK, 0)
        assert s.query()  # the call was waited for
