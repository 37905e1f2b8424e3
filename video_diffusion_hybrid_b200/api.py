"""Torch-facing helpers over the C ABI: device placement of the inputs and a
small callable that owns nothing but a workspace and an output buffer.

Every byte of compute runs in ``libvdn_hybrid.so``; torch provides device
memory and the current stream.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import torch

from . import _lib as L
from .synth import Shape

TENSOR_NAMES = ("q", "k", "v", "beta", "alpha", "gate_sm", "gate_lin", "text_k", "text_v", "text_beta",
                "init_state", "rms_weight", "fwd_init")


def cfg_for(shape: Shape, dtype: str, **kw) -> L.HybridCfg:
    return L.HybridCfg(B=shape.B, T=shape.T, N=shape.N, H=shape.H, d_k=shape.d_k, d_v=shape.d_v, L=shape.L,
                       dtype=L.VDN_BF16 if dtype == "bf16" else L.VDN_F32, **kw)


def to_torch(inp: dict, dtype: str, device="cuda", pin: bool = False) -> dict:
    """Move the synthetic inputs to `device` in their storage types (bf16
    tensors from their exact bit patterns).  With device="cpu" and pin=True
    the result lives in pinned host memory."""
    out = {}
    for name in TENSOR_NAMES:
        if name not in inp:
            continue
        if dtype == "bf16" and name + "_bits" in inp:
            t = torch.from_numpy(np.ascontiguousarray(inp[name + "_bits"]).view(np.int16)).view(torch.bfloat16)
        else:
            t = torch.from_numpy(np.ascontiguousarray(inp[name], dtype=np.float32))
        if pin:
            t = t.pin_memory()
        out[name] = t.to(device) if device != "cpu" else t
    return out


def output_shape(cfg: L.HybridCfg) -> tuple:
    base = (cfg.B, cfg.T, cfg.N, cfg.H)
    return base + ((2, cfg.d_v) if cfg.out_mode == 0 else (cfg.d_v,))


class HybridAttention:
    """Calls ``vdn_hybrid_attn_fwd`` on torch tensors.  Workspace and output
    are allocated once (by torch) and reused."""

    def __init__(self, cfg: L.HybridCfg, device="cuda", keep_lse: bool = False):
        self.cfg = cfg
        self.ws_bytes = L.vdn_hybrid_attn_workspace_size(cfg)
        if self.ws_bytes == 0:
            raise L.VdnError(L.VDN_ERR_INVALID_ARG, "vdn_hybrid_attn_workspace_size")
        self.device = torch.device(device)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        tdt = torch.bfloat16 if cfg.y_dtype == L.VDN_BF16 else torch.float32
        self.y = torch.empty(output_shape(cfg), dtype=tdt, device=self.device)
        # the forward's softmax log-sum-exp per query row, which the softmax
        # backward then takes in place of recomputing the row statistics
        self.sm_lse = (torch.empty((cfg.B, cfg.T, cfg.N, cfg.H), dtype=torch.float32, device=self.device)
                       if keep_lse else None)

    def args(self, t: dict) -> L.VdnArgs:
        return L.make_args(t["q"], t["k"], t["v"], t["beta"], t["alpha"], t["gate_sm"], t["gate_lin"], self.y,
                           self.workspace, self.ws_bytes, text_k=t.get("text_k"), text_v=t.get("text_v"),
                           text_beta=t.get("text_beta"), init_state=t.get("init_state"),
                           rms_weight=t.get("rms_weight"), fwd_init=t.get("fwd_init"), sm_lse=self.sm_lse)

    def __call__(self, t: dict, stages: int = L.STAGE_ALL, stream=None) -> torch.Tensor:
        a = self.args(t)
        if stages == L.STAGE_ALL:
            L.vdn_hybrid_attn_fwd(self.cfg, a, stream)
        else:
            L.vdn_hybrid_attn_fwd_stages(self.cfg, a, stages, stream)
        return self.y

    def linear_backward(self, t: dict, dy: torch.Tensor, want_rms: bool = False, want_fwd_init: bool = False,
                        stream=None) -> dict:
        """Gradients through the linear branch after a forward call on the same
        inputs `t` (the forward's workspace is read): dy has y's shape and
        dtype.  Returns float32 tensors dq, dk, dv, dbeta, dalpha, dgate_lin
        (and drms_weight, dfwd_init when asked)."""
        c = self.cfg
        if getattr(self, "bwd_workspace", None) is None:
            nb = L.vdn_hybrid_lin_bwd_workspace_size(c)
            if nb == 0:
                raise L.VdnError(L.VDN_ERR_UNSUPPORTED, "vdn_hybrid_lin_bwd_workspace_size")
            self.bwd_workspace = torch.empty(nb, dtype=torch.uint8, device=self.device)
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=self.device)
        tok = (c.B, c.T, c.N, c.H)
        g = {"dq": f(*tok, c.d_k), "dk": f(*tok, c.d_k), "dv": f(*tok, c.d_v), "dbeta": f(*tok),
             "dalpha": f(c.B, c.T, c.H), "dgate_lin": f(*tok, c.d_v)}
        if want_rms:
            g["drms_weight"] = f(c.H, c.d_v)
        if want_fwd_init:
            g["dfwd_init"] = f(c.B, c.H, c.d_v, c.d_k)
        lg = L.make_lin_grads(dy, g["dq"], g["dk"], g["dv"], g["dbeta"], g["dalpha"], g["dgate_lin"],
                              self.bwd_workspace, drms_weight=g.get("drms_weight"), dfwd_init=g.get("dfwd_init"))
        L.vdn_hybrid_lin_bwd(c, self.args(t), lg, stream)
        return g

    def softmax_backward(self, t: dict, dy: torch.Tensor, stream=None) -> dict:
        """Gradients through the windowed softmax branch: float32 tensors dq,
        dk, dv, dgate_sm.  With keep_lse, the forward's log-sum-exp (kept by
        the last forward call on the same inputs) replaces the recomputed row
        statistics."""
        c = self.cfg
        if getattr(self, "sm_workspace", None) is None:
            nb = L.vdn_hybrid_sm_bwd_workspace_size(c)
            if nb == 0:
                raise L.VdnError(L.VDN_ERR_UNSUPPORTED, "vdn_hybrid_sm_bwd_workspace_size")
            self.sm_workspace = torch.empty(nb, dtype=torch.uint8, device=self.device)
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=self.device)
        tok = (c.B, c.T, c.N, c.H)
        g = {"dq": f(*tok, c.d_k), "dk": f(*tok, c.d_k), "dv": f(*tok, c.d_v), "dgate_sm": f(*tok, c.d_v)}
        sg = L.make_sm_grads(dy, g["dq"], g["dk"], g["dv"], g["dgate_sm"], self.sm_workspace, sm_lse=self.sm_lse)
        L.vdn_hybrid_sm_bwd(c, self.args(t), sg, stream)
        return g

    def softmax_backward_status(self, stream=None) -> tuple:
        """(status, kernel tag) of the last softmax backward's bounded waits,
        from the status words at the head of its scratch."""
        a = L.VdnArgs()
        a.workspace = self.sm_workspace.data_ptr()
        a.workspace_bytes = self.sm_workspace.numel()
        return L.vdn_hybrid_device_status(self.cfg, a, stream)

    def backward(self, t: dict, dy: torch.Tensor, stream=None) -> dict:
        """The whole core's gradients after a forward call on the same inputs,
        in one library call (``vdn_hybrid_bwd``): dq, dk, dv with both
        branches' shares summed on the device, and the branch-specific
        gradients (drms_weight / dfwd_init when those inputs are given)."""
        c = self.cfg
        if getattr(self, "whole_bwd_workspace", None) is None:
            nb = L.vdn_hybrid_bwd_workspace_size(c)
            if nb == 0:
                raise L.VdnError(L.VDN_ERR_UNSUPPORTED, "vdn_hybrid_bwd_workspace_size")
            self.whole_bwd_workspace = torch.empty(nb, dtype=torch.uint8, device=self.device)
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=self.device)
        tok = (c.B, c.T, c.N, c.H)
        g = {"dq": f(*tok, c.d_k), "dk": f(*tok, c.d_k), "dv": f(*tok, c.d_v), "dbeta": f(*tok),
             "dalpha": f(c.B, c.T, c.H), "dgate_lin": f(*tok, c.d_v), "dgate_sm": f(*tok, c.d_v)}
        if t.get("rms_weight") is not None:
            g["drms_weight"] = f(c.H, c.d_v)
        if t.get("fwd_init") is not None:
            g["dfwd_init"] = f(c.B, c.H, c.d_v, c.d_k)
        gr = L.make_grads(dy, g["dq"], g["dk"], g["dv"], g["dbeta"], g["dalpha"], g["dgate_lin"], g["dgate_sm"],
                          self.whole_bwd_workspace, drms_weight=g.get("drms_weight"), dfwd_init=g.get("dfwd_init"),
                          sm_lse=self.sm_lse)
        L.vdn_hybrid_bwd(c, self.args(t), gr, stream)
        return g

    def backward_status(self, stream=None) -> tuple:
        """(status, kernel tag) of the last whole-core backward: the softmax
        branch's status words (head of the shared scratch), else the linear
        branch's (head of the forward's workspace)."""
        a = L.VdnArgs()
        a.workspace = self.whole_bwd_workspace.data_ptr()
        a.workspace_bytes = self.whole_bwd_workspace.numel()
        st = L.vdn_hybrid_device_status(self.cfg, a, stream)
        if st[0] != L.VDN_OK:
            return st
        a.workspace = self.workspace.data_ptr()
        a.workspace_bytes = self.ws_bytes
        return L.vdn_hybrid_device_status(self.cfg, a, stream)

    def intermediates(self) -> dict:
        """Views of the workspace's intermediate values (float32)."""
        lay = L.vdn_hybrid_workspace_layout(self.cfg)
        c = self.cfg
        C = c.C
        f = lambda off, shape: self.workspace[off:off + 4 * int(np.prod(shape))].view(torch.float32).view(*shape)
        return {
            "half_text": f(lay["half_text"], (c.B, c.H, c.d_v, c.d_k)),
            "M": f(lay["frame_M"], (c.B, c.T, c.H, c.d_k, c.d_k)),
            "C": f(lay["frame_C"], (c.B, c.T, c.H, c.d_v, c.d_k)),
            "fwd_snap": f(lay["fwd_snap"], (c.B, c.H, C + 1, c.d_v, c.d_k)),
            "bwd_snap": f(lay["bwd_snap"], (c.B, c.H, C + 1, c.d_v, c.d_k)),
            "R": f(lay["read_table"], (c.B, c.H, C + 1, c.d_v, c.d_k)),
        }

    def forward_end_state(self) -> torch.Tensor:
        """A copy of the forward state after the last frame (fwd_snap slot C),
        [B, H, d_v, d_k] float32: the next appended segment's ``fwd_init``."""
        return self.intermediates()["fwd_snap"][:, :, self.cfg.C].clone()

    def chunk_maps(self) -> dict:
        """The chunk maps of the chunk-stepped tensor-core scan (bf16 mode,
        d = 128, C >= 4): P_c as hi + lo (float32), Cf_c, Cb_c, Lam_c."""
        lay = L.vdn_hybrid_workspace_layout(self.cfg)
        c = self.cfg
        C, d = c.C, c.d_k
        n = c.B * C * c.H
        if lay["chunk_C"] == lay["chunk_P16"]:
            raise ValueError("no chunk maps for this configuration")
        p16 = self.workspace[lay["chunk_P16"]:lay["chunk_P16"] + 2 * n * 2 * d * d].view(torch.bfloat16)
        p16 = p16.view(c.B, C, c.H, 2, d, d).float()
        cc = self.workspace[lay["chunk_C"]:lay["chunk_C"] + 4 * 2 * n * d * d].view(torch.float32)
        cc = cc.view(2, c.B, C, c.H, d, d)
        lam = self.workspace[lay["chunk_lam"]:lay["chunk_lam"] + 4 * n].view(torch.float32).view(c.B, C, c.H)
        return {"P": p16[:, :, :, 0] + p16[:, :, :, 1], "Cf": cc[0], "Cb": cc[1], "Lam": lam}


# ------------------------------------------ the layer's operators around the core
def _dtype_of(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return L.VDN_BF16
    if t.dtype == torch.float32:
        return L.VDN_F32
    raise TypeError(f"bfloat16 or float32 expected, got {t.dtype}")


def _given(t, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a tensor is needed, got {type(t).__name__}")


def _need(t, name: str, shape, dtype, device) -> None:
    """A dense tensor of this shape, type and device (None passes)."""
    if t is None:
        return
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _int32(n: int, name: str) -> int:
    """A count that the library takes as a 32-bit integer (ctypes would drop its upper bits in silence)."""
    if n > 2**31 - 1:
        raise ValueError(f"{name}: {n} is more than 2^31 - 1")
    return n


def _head_rows(t: torch.Tensor, name: str, lead: tuple, H: int, d: int, dtype, device) -> int:
    """Checks a [*lead, H, d] tensor whose head rows are dense and whose tokens
    lie one stride apart (a slice of a packed projection); returns that stride
    in elements."""
    _given(t, name)
    shape, strides = t.shape, t.stride()
    if shape != (*lead, H, d) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {(*lead, H, d)} on {device}, got {t.dtype} {tuple(shape)} on {t.device}")
    # the stride of an axis of size one says nothing
    if (d > 1 and strides[-1] != 1) or (H > 1 and strides[-2] != d):
        raise ValueError(f"{name}: the head rows have to be dense, got strides {strides}")
    stride, span = None, 0
    for i in range(len(shape) - 3, -1, -1):
        if shape[i] == 1:
            continue
        if strides[i] < H * d or (stride is not None and strides[i] != span):
            raise ValueError(f"{name}: the tokens have to lie one stride apart, got strides {strides}")
        stride = strides[i] if stride is None else stride
        span = strides[i] * shape[i]
    return H * d if stride is None else stride


class _Streamed:
    """What the layer's operators share: a device of their own, and calls that
    run with that device current.  Autograd does not record the calls: gradients
    come from ``backward``.  Every call has at least one token (row)."""

    def __init__(self, device):
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._like = torch.empty(0, device=self.device)
        self._cfgs = {}  # configurations by what changes from call to call (see _keep)

    def _call(self, name, stream, *args):
        """The library's function with the operator's device current, on `stream` or that device's current one; returns
        the stream's handle, where the call's status words can be read."""
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self._call(name, stream, *args)
        on = L._stream_handle(stream)
        st = getattr(L.lib(), name)(*args, on)
        if st != L.VDN_OK:
            raise L.VdnError(st, name)
        return on

    def _keep(self, key, value):
        """Keeps a configuration for the next call with this key.  Their number is bounded: a user with other sizes on
        every call forms a few again now and then."""
        if len(self._cfgs) >= 256:
            self._cfgs.clear()
        self._cfgs[key] = value
        return value

    def _new(self, shape, dtype, stream=None) -> torch.Tensor:
        """A tensor that belongs to the stream of the call: its memory is not
        handed out again before that stream's work is done.  Scratch is new on
        every call, so calls on several streams and captured graphs do not share it."""
        if stream is None:
            return self._like.new_empty(shape, dtype=dtype)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)


class QKNormRope(_Streamed):
    """RMSNorm of every query and key head and the rotation by position, in one
    pass (``vdn_qk_norm_rope``), and its gradients.  q [..., Hq, d] and
    k [..., Hk, d] may be slices of a packed projection; the outputs are dense
    and new on every call.

    wq, wk: float32 [d] (or [H, d] with per_head), None = ones.  table: float32
    [rows, rot / 2, 2] (cos, sin), see ``rope_table``.  pos: int32 [..., axes]
    (or [...] for one axis); None = the token's index (over all leading axes).
    A token with a position outside the table (without a rotation: a negative
    one) is skipped: its output rows are zeros, or with `out` left
    as they were."""

    def __init__(self, Hq: int, Hk: int, d: int, *, rot: int | None = None, pairing: str = "interleaved", sections=None,
                 per_head: bool = False, eps: float = 1e-6, device="cuda"):
        super().__init__(device)
        self.Hq, self.Hk, self.d, self.per_head = Hq, Hk, d, per_head
        self.rot = d if rot is None else rot
        self.sections = tuple(sections) if sections is not None else (self.rot // 2,)
        pair = {"interleaved": L.PAIR_INTERLEAVED, "split": L.PAIR_SPLIT}
        if pairing not in pair or not 1 <= len(self.sections) <= 3:
            raise L.VdnError(L.VDN_ERR_INVALID_ARG, "QKNormRope")
        self.axes, self.pairing, self.eps = len(self.sections), pair[pairing], eps
        self.c_sections = (ctypes.c_int * 3)(*self.sections)
        self.wq_shape, self.wk_shape = ((Hq, d), (Hk, d)) if per_head else ((d,), (d,))

    def _cfg_args(self, q, k, wq, wk, table, pos, grad=0, zero_skipped=False):
        _given(q, "q")
        lead, dt, dev = q.shape[:-2], q.dtype, self.device
        qs = _head_rows(q, "q", lead, self.Hq, self.d, dt, dev)
        ks = _head_rows(k, "k", lead, self.Hk, self.d, dt, dev) if self.Hk else 0
        _need(wq, "wq", self.wq_shape, torch.float32, dev)
        _need(wk, "wk", self.wk_shape, torch.float32, dev)
        rows = 0
        if self.rot:
            if table is None:
                raise ValueError("table: the rotation needs one")
            rows = _int32(table.shape[0], "table rows")
            _need(table, "table", (rows, self.rot // 2, 2), torch.float32, dev)
        if pos is not None:
            _need(pos, "pos", lead if self.axes == 1 and pos.dim() == len(lead) else (*lead, self.axes), torch.int32, dev)
        key = (lead, rows, dt, grad, zero_skipped, qs, ks)
        cfg = self._cfgs.get(key)
        if cfg is None:
            cfg = self._keep(key, L.QkCfg(_int32(math.prod(lead), "tokens"), self.Hq, self.Hk, self.d, self.rot, self.pairing, self.axes,
                                          self.c_sections, rows, int(self.per_head), _dtype_of(q), grad, self.eps,
                                          int(zero_skipped), qs, ks))
        return cfg, L.QkArgs(q.data_ptr(), k.data_ptr() if self.Hk else None, L._ptr(wq), L._ptr(wk),
                             table.data_ptr() if self.rot else None, L._ptr(pos))

    def __call__(self, q, k, wq=None, wk=None, table=None, pos=None, out=None, stream=None):
        """(q_out, k_out), dense, of q's type; `out`: a pair of tensors to write."""
        cfg, args = self._cfg_args(q, k, wq, wk, table, pos, zero_skipped=out is None)
        if out is None:
            out = (self._new(q.shape, q.dtype, stream), self._new(k.shape, q.dtype, stream) if self.Hk else None)
        else:
            _need(out[0], "q_out", q.shape, q.dtype, self.device)
            _need(out[1], "k_out", k.shape if self.Hk else (), q.dtype, self.device)
        args.q_out, args.k_out = out[0].data_ptr(), L._ptr(out[1])
        self._call("vdn_qk_norm_rope", stream, cfg, args)
        return out

    def backward(self, q, k, wq, wk, table, dq_out, dk_out, pos=None, stream=None) -> dict:
        """dq, dk (q's type) and dwq, dwk (float32) from the gradients of the
        outputs (float32, or q's type)."""
        _given(dq_out, "dq_out")
        cfg, args = self._cfg_args(q, k, wq, wk, table, pos, _dtype_of(dq_out))
        _need(dq_out, "dq_out", q.shape, dq_out.dtype, self.device)
        if self.Hk:
            _given(dk_out, "dk_out")
            _need(dk_out, "dk_out", k.shape, dq_out.dtype, self.device)
        ws = self._new(L.vdn_qk_norm_rope_bwd_workspace_size(cfg), torch.uint8, stream)
        new = lambda shape, dt: self._new(shape, dt, stream)  # noqa: E731
        g = {"dq": new(q.shape, q.dtype), "dwq": new(self.wq_shape, torch.float32)}
        if self.Hk:
            g["dk"], g["dwk"] = new(k.shape, q.dtype), new(self.wk_shape, torch.float32)
        gr = L.QkGrads(L._ptr(dq_out), L._ptr(dk_out) if self.Hk else None, L._ptr(g["dq"]), L._ptr(g.get("dk")),
                       L._ptr(g["dwq"]), L._ptr(g.get("dwk")), ws.data_ptr(), ws.numel())
        self._call("vdn_qk_norm_rope_bwd", stream, cfg, args, gr)
        return g


def rope_table(rows: int, sections, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """(cos, sin) of position * base^(-j / pairs) for the pairs j of every axis
    section, float32 [rows, sum(sections), 2]; the angles are formed in float64."""
    freq = np.concatenate([base ** (-np.arange(n, dtype=np.float64) / max(n, 1)) for n in sections])
    a = np.arange(rows, dtype=np.float64)[:, None] * freq
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)).to(device)


class CrossAttention(_Streamed):
    """Softmax cross-attention of Tq query tokens to L encoder states for each of
    B batch elements (``vdn_cross_attn``), and its gradients.  k and v
    [B, L, Hkv, d] may be slices of a packed projection; kv_len: int32 [B] in
    device memory, None = L everywhere.  Outputs and scratch are new on every
    call, and so is the log-sum-exp that keep_lse asks for: `lse` is the last
    forward's, and one that was taken from there stays that call's."""

    def __init__(self, B: int, Tq: int, L_: int, H: int, Hkv: int, d: int, *, dtype: str = "bf16", scale: float = 0.0,
                 keep_lse: bool = False, device="cuda"):
        super().__init__(device)
        self.shape, self.kv_shape = (B, Tq, H, d), (B, L_, Hkv, d)
        self.torch_dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.sizes = (B, Tq, L_, H, Hkv, d, L.VDN_BF16 if dtype == "bf16" else L.VDN_F32, scale)
        self.cfg = L.XattnCfg(*self.sizes)
        self.need, self.bwd_need = L.vdn_cross_attn_workspace_size(self.cfg), L.vdn_cross_attn_bwd_workspace_size(self.cfg)
        if self.need == 0:
            raise L.VdnError(L.VDN_ERR_INVALID_ARG, "vdn_cross_attn_workspace_size")
        self.workspace = self.bwd_workspace = None  # the last calls'
        self.ran_on = self.bwd_ran_on = None  # and their streams
        self.keep_lse, self.lse = keep_lse, None  # of every query row, which the backward takes

    def _inputs(self, q, k, v, kv_len):
        B, _, Hkv, d = self.kv_shape
        _given(q, "q")
        _need(q, "q", self.shape, self.torch_dtype, self.device)
        _need(kv_len, "kv_len", (B,), torch.int32, self.device)
        key = (_head_rows(k, "k", self.kv_shape[:2], Hkv, d, self.torch_dtype, self.device),
               _head_rows(v, "v", self.kv_shape[:2], Hkv, d, self.torch_dtype, self.device))
        cfg = self._cfgs.get(key)
        if cfg is None:
            cfg = self._keep(key, L.XattnCfg(*self.sizes, *key))
        return cfg, L.XattnArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), L._ptr(kv_len))

    def __call__(self, q, k, v, kv_len=None, out=None, stream=None) -> torch.Tensor:
        cfg, a = self._inputs(q, k, v, kv_len)
        if out is None:
            out = self._new(self.shape, self.torch_dtype, stream)
        else:
            _need(out, "out", self.shape, self.torch_dtype, self.device)
        self.workspace = ws = self._new(self.need, torch.uint8, stream)
        self.lse = self._new(self.shape[:3], torch.float32, stream) if self.keep_lse else None
        a.y, a.lse, a.workspace, a.workspace_bytes = out.data_ptr(), L._ptr(self.lse), ws.data_ptr(), self.need
        self.ran_on = self._call("vdn_cross_attn", stream, cfg, a)
        return out

    def backward(self, q, k, v, y, lse, dy, kv_len=None, stream=None) -> dict:
        """dq, dk, dv from the forward's output y and log-sum-exp."""
        cfg, a = self._inputs(q, k, v, kv_len)
        for t, name in ((y, "y"), (lse, "lse"), (dy, "dy")):
            _given(t, name)
        _need(y, "y", self.shape, self.torch_dtype, self.device)
        _need(dy, "dy", self.shape, self.torch_dtype, self.device)
        _need(lse, "lse", self.shape[:3], torch.float32, self.device)
        self.bwd_workspace = ws = self._new(self.bwd_need, torch.uint8, stream)
        a.y, a.lse, a.workspace, a.workspace_bytes = y.data_ptr(), lse.data_ptr(), ws.data_ptr(), self.bwd_need
        new = lambda shape: self._new(shape, self.torch_dtype, stream)  # noqa: E731
        g = {"dq": new(self.shape), "dk": new(self.kv_shape), "dv": new(self.kv_shape)}
        gr = L.XattnGrads(dy.data_ptr(), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr())
        self.bwd_ran_on = self._call("vdn_cross_attn_bwd", stream, cfg, a, gr)
        return g

    def status(self, backward: bool = False, stream=None) -> tuple:
        """(status, kernel tag) of the last forward (or backward) call's bounded waits, read behind that call on its
        stream (or on `stream`)."""
        ws, on = (self.bwd_workspace, self.bwd_ran_on) if backward else (self.workspace, self.ran_on)
        with torch.cuda.device(self.device):
            return L.vdn_cross_attn_device_status(ws, on if stream is None else stream)


def quantize_int8(x: torch.Tensor, stream=None) -> tuple:
    """Signed 8-bit codes of every row of x [rows, cols] and the rows' scales
    (``vdn_quantize_int8``); a weight [out, in] gets a scale per output channel."""
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("quantize_int8: expected a contiguous matrix")
    _int32(x.shape[0], "rows"), _int32(x.shape[1], "columns")
    on = _Streamed(x.device)
    q, scale = on._new(x.shape, torch.int8, stream), on._new(x.shape[:1], torch.float32, stream)
    on._call("vdn_quantize_int8", stream, x.data_ptr(), _dtype_of(x), x.shape[0], x.shape[1], q.data_ptr(), scale.data_ptr())
    return q, scale


class Int8Linear(_Streamed):
    """A linear layer on signed 8-bit codes (``vdn_linear_int8``): w int8
    [N, K] with w_scale float32 [N] (``quantize_int8`` of the weight), bias
    float32 [N] or None.  The call quantises x [..., K] (bfloat16 or float32) by
    rows, or takes codes (int8) with x_scale.  Outputs, scratch and status words
    are new on every call."""

    def __init__(self, w: torch.Tensor, w_scale: torch.Tensor, bias=None, *, out_dtype: str = "bf16"):
        super().__init__(w.device)
        self.N, self.K = w.shape
        _int32(self.N, "channels"), _int32(self.K, "inputs")
        _need(w, "w", (self.N, self.K), torch.int8, self.device)
        _need(w_scale, "w_scale", (self.N,), torch.float32, self.device)
        _need(bias, "bias", (self.N,), torch.float32, self.device)
        self.w, self.w_scale, self.bias = w, w_scale, bias
        self.words = self.ran_on = None  # the last call's status words (their tensor and offset; None: nothing waits) and stream
        self.out_torch = {"bf16": torch.bfloat16, "f32": torch.float32}[out_dtype]
        self.out_dtype = L.VDN_BF16 if out_dtype == "bf16" else L.VDN_F32

    def __call__(self, x: torch.Tensor, x_scale=None, out=None, stream=None) -> torch.Tensor:
        _given(x, "x")
        codes = x.dtype == torch.int8
        if x.shape[-1] != self.K or not x.is_contiguous() or x.device != self.device:
            raise ValueError(f"Int8Linear: expected a contiguous [..., {self.K}] tensor on {self.device}")
        M = x.numel() // self.K
        _need(x_scale, "x_scale", x.shape[:-1], torch.float32, self.device)
        found = self._cfgs.get((M, x.dtype))
        if found is None:
            cfg = L.Int8Cfg(_int32(M, "rows"), self.K, self.N, L.VDN_I8 if codes else _dtype_of(x), self.out_dtype)
            found = self._keep((M, x.dtype), (cfg, L.vdn_linear_int8_workspace_size(cfg)))
        cfg, need = found
        # the status words behind the scratch; a few rows of x need neither
        ws = self._new(need + 256, torch.uint8, stream) if need or codes else None
        self.words = (ws, need) if ws is not None else None
        shape = (*x.shape[:-1], self.N)
        if out is None:
            out = self._new(shape, self.out_torch, stream)
        else:
            _need(out, "out", shape, self.out_torch, self.device)
        a = L.Int8Args(x.data_ptr(), L._ptr(x_scale), self.w.data_ptr(), self.w_scale.data_ptr(), L._ptr(self.bias),
                       out.data_ptr(), L._ptr(ws), need, ws.data_ptr() + need if ws is not None else None)
        self.ran_on = self._call("vdn_linear_int8", stream, cfg, a)
        return out

    def status(self, stream=None) -> tuple:
        """(status, kernel tag) of the last call's bounded waits, read behind that call on its stream (or on `stream`)."""
        if self.words is None:
            return L.VDN_OK, 0
        with torch.cuda.device(self.device):
            return L.vdn_linear_int8_device_status(self.words[0].data_ptr() + self.words[1], self.ran_on if stream is None else stream)
