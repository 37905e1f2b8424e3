"""The gradient formulas of the layer oracle against differences (float64, CPU)."""
import pytest
import torch

from oracle import layer_oracle as R

D64 = torch.float64


def diff(f, x, v, h=1e-6):
    """Central difference of the scalar f along v."""
    return float((f(x + h * v) - f(x - h * v)) / (2 * h))


@pytest.mark.parametrize("pairing", ["interleaved", "split"])
@pytest.mark.parametrize("rot,sections", [(0, (0,)), (16, (8,)), (16, (3, 0, 5)), (32, (10, 6))])
def test_qk_norm_rope_gradients_match_differences(pairing, rot, sections):
    g = torch.Generator().manual_seed(1)
    t, H, d = 5, 3, 32
    rnd = lambda *s: torch.randn(s, generator=g, dtype=D64)  # noqa: E731
    x, w, up = rnd(t, H, d), rnd(H, d), rnd(t, H, d)
    pos = torch.randint(0, 9, (t, len(sections)), generator=g, dtype=torch.int32)
    ang = 6 * torch.rand((9, max(rot // 2, 1)), generator=g, dtype=D64)
    table = torch.stack([ang.cos(), ang.sin()], -1)
    f = lambda x_, w_: (up * R.qk_norm_rope(x_, w_, table, pos, rot, pairing, sections, 1e-6)).sum()  # noqa: E731
    dx, dw, _, _ = R.qk_norm_rope_bwd(x, w, table, pos, rot, pairing, sections, 1e-6, up)
    for _ in range(3):
        vx, vw = rnd(t, H, d), rnd(H, d)
        # a difference of step 1e-6: 1e-16 / 1e-6 of the sum's size in rounding, 1e-12 in curvature
        assert abs(diff(lambda z: f(z, w), x, vx) - float((dx * vx).sum())) < 1e-6
        assert abs(diff(lambda z: f(x, z), w, vw) - float((dw * vw).sum())) < 1e-6


@pytest.mark.parametrize("lens", [None, [5, 0], [1, 3]])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 2), (3, 1)])
def test_cross_attn_gradients_match_differences(H, Hkv, lens):
    g = torch.Generator().manual_seed(2)
    B, Tq, L, d = 2, 4, 5, 8
    rnd = lambda *s: torch.randn(s, generator=g, dtype=D64)  # noqa: E731
    x = {"q": rnd(B, Tq, H, d), "k": rnd(B, L, Hkv, d), "v": rnd(B, L, Hkv, d)}
    up = rnd(B, Tq, H, d)
    n = None if lens is None else torch.tensor(lens)
    f = lambda y: (up * R.cross_attn(y["q"], y["k"], y["v"], n)[0]).sum()  # noqa: E731
    r = R.cross_attn_bwd(x["q"], x["k"], x["v"], up, n)
    for key in x:
        v = rnd(*x[key].shape)
        want = diff(lambda z: f({**x, key: z}), x[key], v)
        assert abs(want - float((r["d" + key][0] * v).sum())) < 1e-6, key


def test_int8_codes_by_hand():
    x = torch.tensor([[127.0, 63.5, -0.5, 1.5], [0, 0, 0, 0], [2.0, 1.0, -2.0, 0.1], [float("inf"), 1, 2, 3]])
    q, s = R.quantize_int8(x)
    assert q.tolist() == [[127, 64, 0, 2], [0, 0, 0, 0], [127, 64 if 1.0 / float(s[2]) >= 63.5 else 63, -127, 6], [0, 0, 0, 0]]
    assert s[0] == 1 and s[1] == 1 and s[3].isnan()
