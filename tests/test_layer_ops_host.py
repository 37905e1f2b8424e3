"""Host-side checks of the layer's operators around the core: arguments are
refused before anything is launched (no device needed), sizes and the
implementation that a configuration selects."""
import ctypes as C

import pytest

from video_diffusion_hybrid_b200 import _lib as L
from video_diffusion_hybrid_b200.build import build

P = 1 << 20  # aligned, never dereferenced: every call here fails validation


@pytest.fixture(scope="module", autouse=True)
def built():
    build()
    return L.lib()


def qk_cfg(**kw):
    c = dict(tokens=10, Hq=4, Hk=2, d=64, rot=64, pairing=0, axes=1, table_rows=16, per_head=0, dtype=L.VDN_BF16,
             grad_dtype=L.VDN_BF16, eps=1e-6, q_stride=0, k_stride=0)
    sections = kw.pop("sections", None)
    c.update(kw)
    cfg = L.QkCfg(**c)
    for i, s in enumerate(sections if sections is not None else [c["rot"] // 2]):
        cfg.sections[i] = s
    return cfg


def qk_args(**kw):
    a = dict(q=P, k=P, wq=P, wk=P, table=P, pos=P, q_out=P, k_out=P)
    a.update(kw)
    return L.QkArgs(**a)


def qk_grads(cfg, **kw):
    g = dict(dq_out=P, dk_out=P, dq=P, dk=P, dwq=P, dwk=P, workspace=P,
             workspace_bytes=L.vdn_qk_norm_rope_bwd_workspace_size(cfg))
    g.update(kw)
    return L.QkGrads(**g)


BAD_QK = [dict(tokens=0), dict(Hq=0), dict(Hk=-1), dict(d=0), dict(d=60), dict(d=264), dict(rot=80), dict(rot=8),
          dict(rot=-16), dict(pairing=2), dict(axes=0), dict(axes=4), dict(table_rows=0), dict(per_head=2), dict(dtype=2),
          dict(grad_dtype=3), dict(eps=float("nan")), dict(q_stride=255), dict(q_stride=260), dict(k_stride=-8),
          dict(sections=[31]), dict(axes=2, sections=[40, -8]), dict(axes=2, sections=[2**31 - 1, 2**31 - 1])]


@pytest.mark.parametrize("kw", BAD_QK, ids=str)
def test_qk_bad_config(kw):
    cfg = qk_cfg(**kw)
    assert L.vdn_qk_norm_rope(cfg, qk_args(), stream=0, check=False) == L.VDN_ERR_INVALID_ARG
    assert L.vdn_qk_norm_rope_bwd_workspace_size(cfg) == 0
    assert L.vdn_qk_norm_rope_bwd(cfg, qk_args(), qk_grads(cfg), stream=0, check=False) == L.VDN_ERR_INVALID_ARG


def test_qk_too_many_heads():
    assert L.vdn_qk_norm_rope(qk_cfg(Hq=65535, Hk=1), qk_args(), stream=0, check=False) == L.VDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(q=P + 8), dict(k=P + 2), dict(table=None),
                                dict(table=P + 8), dict(q_out=None), dict(k_out=P + 4), dict(wq=P + 2), dict(pos=P + 1)], ids=str)
def test_qk_bad_arguments(kw):
    assert L.vdn_qk_norm_rope(qk_cfg(), qk_args(**kw), stream=0, check=False) == L.VDN_ERR_INVALID_ARG


def test_qk_index_positions_need_the_table_rows():
    """Without positions a token's index is its position: the table has to hold them all, and there is one axis."""
    a = qk_args(pos=None)
    assert L.vdn_qk_norm_rope(qk_cfg(tokens=17), a, stream=0, check=False) == L.VDN_ERR_INVALID_ARG
    assert L.vdn_qk_norm_rope(qk_cfg(axes=2, sections=[16, 16]), a, stream=0, check=False) == L.VDN_ERR_INVALID_ARG
    # a table without a rotation is refused too
    assert L.vdn_qk_norm_rope(qk_cfg(rot=0), qk_args(), stream=0, check=False) == L.VDN_ERR_INVALID_ARG


def test_qk_backward_arguments():
    cfg = qk_cfg()
    bad = lambda c=cfg, a=None, **kw: L.vdn_qk_norm_rope_bwd(c, a or qk_args(), qk_grads(c, **kw), stream=0, check=False)  # noqa: E731
    for kw in (dict(dq_out=None), dict(dk_out=None), dict(dq=None), dict(dk=P + 8), dict(dwq=P + 2)):
        assert bad(**kw) == L.VDN_ERR_INVALID_ARG, kw
    for kw in (dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=64)):
        assert bad(**kw) == L.VDN_ERR_WORKSPACE, kw
    assert bad(qk_cfg(dtype=L.VDN_F32, grad_dtype=L.VDN_BF16)) == L.VDN_ERR_INVALID_ARG
    assert L.vdn_qk_norm_rope_bwd(cfg, qk_args(), None, stream=0, check=False) == L.VDN_ERR_INVALID_ARG


def x_cfg(**kw):
    c = dict(B=2, Tq=100, L=77, H=8, Hkv=4, d=64, dtype=L.VDN_BF16, scale=0.0, k_stride=0, v_stride=0)
    c.update(kw)
    return L.XattnCfg(**c)


def x_args(cfg, **kw):
    n = max(L.vdn_cross_attn_workspace_size(cfg), L.vdn_cross_attn_bwd_workspace_size(cfg))
    a = dict(q=P, k=P, v=P, kv_len=P, y=P, lse=P, workspace=P, workspace_bytes=n)
    a.update(kw)
    return L.XattnArgs(**a)


GRADS = dict(dy=P, dq=P, dk=P, dv=P)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), L.VDN_ERR_INVALID_ARG), (dict(Tq=0), L.VDN_ERR_INVALID_ARG), (dict(L=0), L.VDN_ERR_INVALID_ARG),
    (dict(H=0), L.VDN_ERR_INVALID_ARG), (dict(Hkv=0), L.VDN_ERR_INVALID_ARG), (dict(Hkv=3), L.VDN_ERR_INVALID_ARG),
    (dict(dtype=2), L.VDN_ERR_INVALID_ARG), (dict(scale=float("nan")), L.VDN_ERR_INVALID_ARG),
    (dict(k_stride=255), L.VDN_ERR_INVALID_ARG), (dict(v_stride=260), L.VDN_ERR_INVALID_ARG),
    (dict(k_stride=-256), L.VDN_ERR_INVALID_ARG), (dict(d=256), L.VDN_ERR_UNSUPPORTED), (dict(d=96), L.VDN_ERR_UNSUPPORTED),
    (dict(B=1 << 16, Tq=1 << 16), L.VDN_ERR_UNSUPPORTED), (dict(B=1 << 16, L=1 << 16), L.VDN_ERR_UNSUPPORTED),
    (dict(B=1 << 14, Tq=1 << 15, H=1 << 14, Hkv=1), L.VDN_ERR_UNSUPPORTED),
], ids=str)
def test_xattn_bad_config(kw, status):
    cfg = x_cfg(**kw)
    assert L.vdn_cross_attn_workspace_size(cfg) == 0 and L.vdn_cross_attn_bwd_workspace_size(cfg) == 0
    assert L.vdn_cross_attn_impl(cfg) == -1 and L.vdn_cross_attn_impl(cfg, True) == -1
    assert L.vdn_cross_attn(cfg, x_args(cfg), stream=0, check=False) == status
    assert L.vdn_cross_attn_bwd(cfg, x_args(cfg), L.XattnGrads(**GRADS), stream=0, check=False) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), L.VDN_ERR_INVALID_ARG), (dict(k=None), L.VDN_ERR_INVALID_ARG), (dict(v=P + 8), L.VDN_ERR_INVALID_ARG),
    (dict(y=None), L.VDN_ERR_INVALID_ARG), (dict(kv_len=P + 2), L.VDN_ERR_INVALID_ARG), (dict(lse=P + 1), L.VDN_ERR_INVALID_ARG),
    (dict(workspace=None), L.VDN_ERR_WORKSPACE), (dict(workspace=P + 128), L.VDN_ERR_WORKSPACE),
    (dict(workspace_bytes=0), L.VDN_ERR_WORKSPACE),
], ids=str)
def test_xattn_bad_arguments(kw, status):
    cfg = x_cfg()
    assert L.vdn_cross_attn(cfg, x_args(cfg, **kw), stream=0, check=False) == status
    assert L.vdn_cross_attn_bwd(cfg, x_args(cfg, **kw), L.XattnGrads(**GRADS), stream=0, check=False) == status


def test_xattn_backward_arguments():
    cfg = x_cfg()
    for k in GRADS:
        for v in (None, P + 8):
            assert L.vdn_cross_attn_bwd(cfg, x_args(cfg), L.XattnGrads(**{**GRADS, k: v}), stream=0, check=False) == \
                L.VDN_ERR_INVALID_ARG
    assert L.vdn_cross_attn_bwd(cfg, x_args(cfg, lse=None), L.XattnGrads(**GRADS), stream=0, check=False) == L.VDN_ERR_INVALID_ARG
    assert L.vdn_cross_attn_bwd(cfg, x_args(cfg), None, stream=0, check=False) == L.VDN_ERR_INVALID_ARG


def i8_cfg(**kw):
    c = dict(M=100, K=64, N=48, x_dtype=L.VDN_BF16, out_dtype=L.VDN_BF16)
    c.update(kw)
    return L.Int8Cfg(**c)


def i8_args(cfg, **kw):
    a = dict(x=P, x_scale=None, w=P, w_scale=P, bias=P, out=P, workspace=P,
             workspace_bytes=L.vdn_linear_int8_workspace_size(cfg))
    a.update(kw)
    return L.Int8Args(**a)


@pytest.mark.parametrize("kw", [dict(M=0), dict(K=0), dict(K=24), dict(K=131072), dict(N=0), dict(N=24), dict(x_dtype=3),
                                dict(out_dtype=2)], ids=str)
def test_int8_bad_config(kw):
    cfg = i8_cfg(**kw)
    assert L.vdn_linear_int8_workspace_size(cfg) == 0
    assert L.vdn_linear_int8(cfg, i8_args(cfg), stream=0, check=False) == L.VDN_ERR_INVALID_ARG


def test_int8_bad_arguments():
    cfg = i8_cfg()
    for kw in (dict(x=None), dict(w=P + 8), dict(w_scale=P + 4), dict(bias=P + 4), dict(out=None), dict(x_scale=P)):
        assert L.vdn_linear_int8(cfg, i8_args(cfg, **kw), stream=0, check=False) == L.VDN_ERR_INVALID_ARG, kw
    for kw in (dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=100 * 64)):
        assert L.vdn_linear_int8(cfg, i8_args(cfg, **kw), stream=0, check=False) == L.VDN_ERR_WORKSPACE, kw
    codes = i8_cfg(x_dtype=L.VDN_I8)
    assert L.vdn_linear_int8_workspace_size(codes) == 0
    assert L.vdn_linear_int8(codes, i8_args(codes), stream=0, check=False) == L.VDN_ERR_INVALID_ARG  # no x_scale
    assert L.vdn_linear_int8(codes, i8_args(codes, x_scale=P + 2), stream=0, check=False) == L.VDN_ERR_INVALID_ARG


def test_int8_quantize_arguments():
    q = lambda **kw: L.vdn_quantize_int8(**{**dict(x=P, x_dtype=L.VDN_F32, rows=3, cols=32, q=P, scale=P, stream=0, check=False), **kw})  # noqa: E731
    for kw in (dict(x=None), dict(x=P + 8), dict(q=None), dict(scale=P + 2), dict(x_dtype=2), dict(rows=0), dict(cols=24), dict(cols=0)):
        assert q(**kw) == L.VDN_ERR_INVALID_ARG, kw


def test_null_structs():
    lib, c, a = L.lib(), C.byref, None
    assert lib.vdn_qk_norm_rope(None, None, None) == L.VDN_ERR_INVALID_ARG
    assert lib.vdn_qk_norm_rope(c(qk_cfg()), a, None) == L.VDN_ERR_INVALID_ARG
    assert lib.vdn_cross_attn(None, None, None) == L.VDN_ERR_INVALID_ARG
    assert lib.vdn_cross_attn(c(x_cfg()), a, None) == L.VDN_ERR_INVALID_ARG
    assert lib.vdn_linear_int8(None, None, None) == L.VDN_ERR_INVALID_ARG
    assert lib.vdn_linear_int8(c(i8_cfg()), a, None) == L.VDN_ERR_INVALID_ARG
    assert lib.vdn_cross_attn_device_status(None, None, None) == L.VDN_ERR_INVALID_ARG
    for fn in ("vdn_qk_norm_rope_bwd_workspace_size", "vdn_cross_attn_workspace_size", "vdn_cross_attn_bwd_workspace_size",
               "vdn_linear_int8_workspace_size"):
        assert getattr(lib, fn)(None) == 0


@pytest.mark.parametrize("kw,fwd,bwd", [
    (dict(), 1, 1), (dict(Tq=8), 2, 1), (dict(Tq=9), 1, 1), (dict(Tq=1, H=16, Hkv=1), 2, 1), (dict(Tq=1, H=17, Hkv=1), 1, 1),
    (dict(d=32), 0, 0), (dict(dtype=L.VDN_F32), 0, 0), (dict(Tq=1, d=32), 0, 0), (dict(Tq=1, dtype=L.VDN_F32), 0, 0),
], ids=str)
def test_xattn_implementation(kw, fwd, bwd):
    """bf16 of d = 64 or 128: up to 16 query rows a key head take the kernel for few rows, more the tensor cores."""
    cfg = x_cfg(**kw)
    assert (L.vdn_cross_attn_impl(cfg), L.vdn_cross_attn_impl(cfg, True)) == (fwd, bwd)


def test_xattn_workspace_sizes():
    """Status words alone where nothing is split; few rows need no more however long the states are."""
    assert L.vdn_cross_attn_workspace_size(x_cfg(Tq=1, L=1 << 20)) == 256
    assert L.vdn_cross_attn_workspace_size(x_cfg(B=40, Tq=4000)) == 256
    assert L.vdn_cross_attn_workspace_size(x_cfg(B=1, Tq=64, L=8192)) > 256
    rows = 2 * 100 * 8
    assert L.vdn_cross_attn_bwd_workspace_size(x_cfg()) >= 256 + 4 * rows


def test_int8_workspace_is_for_codes_and_scales():
    assert L.vdn_linear_int8_workspace_size(i8_cfg(M=8)) == 0
    assert L.vdn_linear_int8_workspace_size(i8_cfg(M=9)) >= 9 * 64 + 9 * 4
    assert L.vdn_linear_int8_workspace_size(i8_cfg(M=1 << 20, K=131056)) >= (1 << 20) * (131056 + 4)


def test_layer_wait_limit_is_bounded():
    """The failure tests' hook: up to the default limit of about a second, and no further."""
    assert L.vdn_debug_set_layer_wait_limit(2_000_000_001, check=False) == L.VDN_ERR_INVALID_ARG
    assert L.vdn_debug_set_layer_wait_limit(300) == L.VDN_OK
    assert L.vdn_debug_set_layer_wait_limit(0) == L.VDN_OK


def test_qk_zero_skipped_is_a_flag():
    """The output rows of skipped tokens: left, or zeros; nothing else is taken."""
    for v in (2, -1):
        assert L.vdn_qk_norm_rope(qk_cfg(zero_skipped=v), qk_args(), stream=0, check=False) == L.VDN_ERR_INVALID_ARG
    assert L.vdn_qk_norm_rope_bwd_workspace_size(qk_cfg(zero_skipped=1)) == L.vdn_qk_norm_rope_bwd_workspace_size(qk_cfg()) > 0


def test_int8_status_words():
    """A call's own status words: four-byte aligned, or none."""
    cfg = i8_cfg()
    assert L.vdn_linear_int8(cfg, i8_args(cfg, status=P + 2), stream=0, check=False) == L.VDN_ERR_INVALID_ARG
    assert L.vdn_linear_int8_device_status(None, stream=0) == (L.VDN_ERR_INVALID_ARG, 0)


@pytest.mark.parametrize("M,K,N,impl", [
    (1, 6144, 4096, 0), (8, 6144, 4096, 0), (9, 6144, 4096, 32), (5, 131056, 16, 32), (128, 6144, 4096, 32), (237, 1280, 784, 32),
    (237, 6144, 4096, 64), (512, 6144, 4096, 64), (1008, 6144, 2048, 64), (1008, 6144, 4096, 256), (1500, 6144, 2048, 256),
    (2016, 6144, 784, 64), (2016, 6144, 4096, 256), (90720, 6144, 4096, 256), (2**31 - 1, 16, 16, 256), (9, 16, 2**31 - 16, 256),
])
def test_int8_implementation(M, K, N, impl):
    """The kernel of few rows, one-CTA tiles up to two turns of the SMs, CTA pairs."""
    assert L.vdn_linear_int8_impl(i8_cfg(M=M, K=K, N=N)) == impl
    assert L.vdn_linear_int8_impl(i8_cfg(M=M, K=24, N=N)) == -1
