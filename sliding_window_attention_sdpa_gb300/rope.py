"""What goes into the attention: binding of ``include/sdpa_rope.h``.

``qk_rotate`` norms each head of queries and keys and rotates them by their
tokens' positions, in one pass; ``qk_rotate_backward`` takes the gradients that
``backward`` gives for them back to what came in. All work runs in the CUDA
library on torch's current stream; the calls can be captured into a CUDA graph.

    q, k = qk_rotate(q0, k0, positions, freq, q_weight=wq, k_weight=wk)
    o, lse = forward(q, k, v, scale=s, window_left=w)
    dq, dk, dv, _ = backward(q, k, v, o, do, lse, scale=s, window_left=w)
    dq0, dk0, dwq, dwk = qk_rotate_backward(dq, dk, q0, k0, positions, freq, q_weight=wq, k_weight=wk)
"""
from __future__ import annotations

import ctypes
import struct

from .cache import _apart, _flat, _given, _strides, _strides4

_i64x3 = ctypes.c_int64 * 3
_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class SdpaRopeParams(ctypes.Structure):
    """Mirror of ``sdpa_rope_params`` (field order and types as in the header)."""
    _fields_ = [
        ("dtype", _i32), ("layout", _i32), ("interleaved", _i32), ("weight_f32", _i32),
        ("b", _i64), ("s", _i64), ("total", _i64), ("h_q", _i64), ("h_kv", _i64), ("d", _i64),
        ("rot", _i64), ("n_axes", _i64),
        ("eps", _f32), ("weight_offset", _f32), ("rot_scale", _f32), ("reserved0", _i32),
        ("positions", _vp), ("axis", _vp), ("freq", _vp), ("seq_lens", _vp),
        ("q_weight", _vp), ("k_weight", _vp), ("q", _vp), ("k", _vp), ("gq", _vp), ("gk", _vp),
        ("oq", _vp), ("ok", _vp), ("dq_weight", _vp), ("dk_weight", _vp),
        ("q_stride", _i64x3), ("k_stride", _i64x3), ("gq_stride", _i64x3), ("gk_stride", _i64x3),
        ("oq_stride", _i64x3), ("ok_stride", _i64x3),
    ]


ENTRY_POINTS = ("sdpa_rope_params_bytes", "sdpa_rope_fwd", "sdpa_rope_bwd_workspace_bytes", "sdpa_rope_bwd")


def bind(lib) -> None:
    """Argument and result types of the rotation's entry points."""
    P, sz, st = ctypes.POINTER(SdpaRopeParams), ctypes.c_size_t, ctypes.c_int
    lib.sdpa_rope_params_bytes.argtypes, lib.sdpa_rope_params_bytes.restype = [], sz
    lib.sdpa_rope_fwd.argtypes, lib.sdpa_rope_fwd.restype = [P, _vp], st
    lib.sdpa_rope_bwd_workspace_bytes.argtypes, lib.sdpa_rope_bwd_workspace_bytes.restype = [P], sz
    lib.sdpa_rope_bwd.argtypes, lib.sdpa_rope_bwd.restype = [P, _vp, sz, _vp], st


def _lib():
    from . import load
    return load()


# ----------------------------------------------------- one-to-one C entry points

def sdpa_rope_fwd(params: SdpaRopeParams, stream: int) -> int:
    return _lib().sdpa_rope_fwd(params, stream)


def sdpa_rope_bwd_workspace_bytes(params: SdpaRopeParams) -> int:
    return int(_lib().sdpa_rope_bwd_workspace_bytes(params))


def sdpa_rope_bwd(params: SdpaRopeParams, workspace: int, workspace_bytes: int, stream: int) -> int:
    return _lib().sdpa_rope_bwd(params, workspace, workspace_bytes, stream)


# ------------------------------------------------------------- torch helpers

class _Calls:
    """The entry points with their parameter block as packed bytes (the layout of
    the struct above), and torch's current stream: see cache._Calls."""

    def __init__(self):
        import torch
        from . import SDPA_BF16, SDPA_F16
        lib = _lib()
        self.fwd, self.bwd = lib["sdpa_rope_fwd"], lib["sdpa_rope_bwd"]
        self.fwd.argtypes, self.fwd.restype = [ctypes.c_char_p, _vp], ctypes.c_int
        self.bwd.argtypes, self.bwd.restype = [ctypes.c_char_p, _vp, ctypes.c_size_t, _vp], ctypes.c_int
        self.dtypes = {torch.bfloat16: SDPA_BF16, torch.float16: SDPA_F16}
        self.empty, self.float32, self.int32, self.uint8 = torch.empty, torch.float32, torch.int32, torch.uint8
        self.stream = torch._C._cuda_getCurrentRawStream


_PARAMS = struct.Struct("4i8q3fi14Q18q")
assert _PARAMS.size == ctypes.sizeof(SdpaRopeParams)
_NONE = (0, 0, 0)
_calls = None


def _c() -> _Calls:
    global _calls
    if _calls is None:
        _calls = _Calls()
    return _calls


def _rows(name, t, shape, dev, dt):
    """Strides (batch, token, head) of a tensor of this shape."""
    if len(shape) == 4:
        return _strides4(name, t, shape, dev, dt)
    return 0, *_strides(name, t, shape, dev, dt)


def _weight(name, w, d, dev, dt, c):
    if w.dtype is not dt and w.dtype is not c.float32:
        raise ValueError(f"{name}: expected dtype {dt} or {c.float32}, got {w.dtype}")
    return _flat(name, w, (d,), dev, w.dtype)


class _Shape:
    """What the tensors' common shape and the arrays give of a call's parameters."""
    __slots__ = ("c", "dt", "dev", "qs", "ks", "head", "floats", "arrays", "norm")

    def __init__(self, q, k, positions, freq, q_weight, k_weight, eps, weight_offset, axis, interleaved, rot_scale, seq_lens):
        c = self.c = _calls or _c()
        dt, dev = self.dt, self.dev = q.dtype, q.device
        code = c.dtypes.get(dt)
        if code is None:
            raise ValueError(f"unsupported dtype {dt}")
        qs = self.qs = q.shape
        n = len(qs)
        if n not in (3, 4):
            raise ValueError(f"q: expected [b, s, h, d] or [total, h, d], got {tuple(qs)}")
        rows, d = qs[:-2], qs[-1]
        h_kv, self.ks = 0, None
        if k is not None:
            ks = self.ks = k.shape
            if len(ks) != n or ks[:-2] != rows or ks[-1] != d:
                raise ValueError(f"k: expected {tuple(rows)} rows of heads of {d} features like q's, got {tuple(ks)}")
            h_kv = ks[-2]
        if freq.dim() != 1:
            raise ValueError(f"freq: expected [rot / 2], got {tuple(freq.shape)}")
        half = freq.shape[0]
        n_axes, at = 1, positions.shape
        if len(at) == n - 1:
            n_axes = at[0]
            if axis is None and n_axes != 1:
                raise ValueError("axis: positions of several axes need each pair's axis")
            want = (n_axes, *rows)
        else:
            want = rows
        if seq_lens is not None and n == 3:
            raise ValueError("seq_lens: only with [b, s, h, d]")
        wq = wk = f32 = 0
        self.norm = q_weight is not None
        if k is None:
            if k_weight is not None:
                raise ValueError("k_weight: there is no k")
        elif self.norm != (k_weight is not None):
            raise ValueError("q_weight and k_weight: both or neither")
        if self.norm:
            wq = _weight("q_weight", q_weight, d, dev, dt, c)
            f32 = int(q_weight.dtype is c.float32)
            if k is not None:
                if k_weight.dtype is not q_weight.dtype:
                    raise ValueError(f"k_weight: expected dtype {q_weight.dtype}, got {k_weight.dtype}")
                wk = _weight("k_weight", k_weight, d, dev, dt, c)
        b, s, total = (0, 0, rows[0]) if n == 3 else (*rows, 0)
        self.head = (code, int(n == 3), int(bool(interleaved)), f32, b, s, total, qs[-2], h_kv, d, 2 * half, n_axes, eps, weight_offset,
                     rot_scale, 0)
        self.arrays = (_flat("positions", positions, want, dev, c.int32),
                       0 if axis is None else _flat("axis", axis, (half,), dev, c.int32), _flat("freq", freq, (half,), dev, c.float32),
                       0 if seq_lens is None else _flat("seq_lens", seq_lens, rows[:1], dev, c.int32), wq, wk)

    def outputs(self, out):
        """The tensors to write to, their addresses, their strides."""
        qs, ks, dt, dev = self.qs, self.ks, self.dt, self.dev
        if out is None:
            oq = self.c.empty(qs, dtype=dt, device=dev)
            ok = None if ks is None else self.c.empty(ks, dtype=dt, device=dev)
        else:
            oq, ok = out
            _apart("out q", oq)
            if ks is not None:
                _apart("out k", ok)
        sq = _rows("out q", oq, qs, dev, dt)
        if ks is None:
            return oq, None, oq.data_ptr(), 0, sq, _NONE
        return oq, ok, oq.data_ptr(), ok.data_ptr(), sq, _rows("out k", ok, ks, dev, dt)


def _check(code, where):
    if code:
        from . import SdpaError, last_error
        raise SdpaError(code, where, last_error())


def qk_rotate(q, k, positions, freq, *, q_weight=None, k_weight=None, eps: float = 1e-6, weight_offset: float = 0.0, axis=None,
              interleaved: bool = False, rot_scale: float = 1.0, seq_lens=None, out=None):
    """Each head's RMS norm (with weights) and position rotation; returns (q, k).

    q: [b, s, h_q, d], k: [b, s, h_kv, d] (or None), or packed [total, h, d];
    positions: int32 [b, s] ([total]), or [n_axes, b, s] with axis: int32
    [rot / 2], each pair's axis; freq: fp32 [rot / 2], radians per position;
    q_weight, k_weight: [d] in q's dtype or fp32, applied as w + weight_offset
    (without them there is no norm); interleaved: pairs are neighbours, else
    feature i and i + rot / 2; rot_scale multiplies what is rotated; seq_lens:
    int32 [b], rows behind it are not read and become zeros. out: (q, k) to
    write to, q and k themselves too. No gradient is recorded
    (qk_rotate_backward computes it).
    """
    x = _Shape(q, k, positions, freq, q_weight, k_weight, eps, weight_offset, axis, interleaved, rot_scale, seq_lens)
    sq = _rows("q", q, x.qs, x.dev, x.dt)
    kp, sk = (0, _NONE) if k is None else (k.data_ptr(), _rows("k", k, x.ks, x.dev, x.dt))
    oq, ok, oqp, okp, soq, sok = x.outputs(out)
    p = _PARAMS.pack(*x.head, *x.arrays, q.data_ptr(), kp, 0, 0, oqp, okp, 0, 0, *sq, *sk, 0, 0, 0, 0, 0, 0, *soq, *sok)
    code = x.c.fwd(p, x.c.stream(x.dev.index or 0))
    if code:
        _check(code, "sdpa_rope_fwd")
    return oq, ok


def qk_rotate_backward(dq, dk, q, k, positions, freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                       weight_offset: float = 0.0, axis=None, interleaved: bool = False, rot_scale: float = 1.0, seq_lens=None,
                       out=None, workspace=None):
    """Gradients of qk_rotate: (dq, dk, dq_weight, dk_weight) from those of its
    outputs, dq and dk, and its inputs q and k (not read, and may be None, without
    weights). The other arguments are qk_rotate's; the weights' gradients are fp32
    [d] (None without weights). out: (dq, dk) to write to, the given ones too.
    """
    x = _Shape(dq, dk, positions, freq, q_weight, k_weight, eps, weight_offset, axis, interleaved, rot_scale, seq_lens)
    c, dev, dt = x.c, x.dev, x.dt
    sgq = _rows("dq", dq, x.qs, dev, dt)
    gkp, sgk = (0, _NONE) if dk is None else (dk.data_ptr(), _rows("dk", dk, x.ks, dev, dt))
    wq = wk = None
    qp = kp = wqp = wkp = n = 0
    sq = sk = _NONE
    if x.norm:
        if q is None or dk is not None and k is None:
            raise ValueError(f"{'q' if q is None else 'k'}: needed with q_weight and k_weight")
        qp, sq = q.data_ptr(), _rows("q", q, x.qs, dev, dt)
        wq = c.empty(x.qs[-1], dtype=c.float32, device=dev)
        wqp = wq.data_ptr()
        if dk is not None:
            kp, sk = k.data_ptr(), _rows("k", k, x.ks, dev, dt)
            wk = c.empty(x.qs[-1], dtype=c.float32, device=dev)
            wkp = wk.data_ptr()
    oq, ok, oqp, okp, soq, sok = x.outputs(out)
    p = _PARAMS.pack(*x.head, *x.arrays, qp, kp, dq.data_ptr(), gkp, oqp, okp, wqp, wkp, *sq, *sk, *sgq, *sgk, *soq, *sok)
    if x.norm:
        if workspace is None:
            n = sdpa_rope_bwd_workspace_bytes(SdpaRopeParams.from_buffer_copy(p))
            if n == 0:
                from . import SDPA_ERR_INVALID_ARG
                _check(SDPA_ERR_INVALID_ARG, "sdpa_rope_bwd_workspace_bytes")
            workspace = c.empty(n, dtype=c.uint8, device=dev)
        else:
            n = _given(workspace, c)
    code = c.bwd(p, workspace.data_ptr() if n else 0, n, c.stream(dev.index or 0))
    if code:
        _check(code, "sdpa_rope_bwd")
    return oq, ok, wq, wk
