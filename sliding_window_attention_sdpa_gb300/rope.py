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

def _rows(name, t, shape, dev, dt, output=False):
    """Strides (batch, token, head) of a tensor of this shape; 0 where there is no second entry."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dt:
        raise ValueError(f"{name}: expected dtype {dt}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name}: the feature dimension must be contiguous (stride 1)")
    if output and any(s == 0 and n > 1 for s, n in zip(st, t.shape)):
        raise ValueError(f"{name}: rows share memory (an expanded tensor)")
    st = [s if n > 1 else 0 for s, n in zip(st[:-1], t.shape)]
    return _i64x3(*(st if len(st) == 3 else [0, *st]))


def _array(name, t, shape, dev, dtypes):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _params(like_q, like_k, positions, freq, q_weight, k_weight, eps, weight_offset, axis, interleaved, rot_scale, seq_lens):
    """The parameters that the tensors' common shape gives (like_k: None for queries alone)."""
    import torch
    from . import SDPA_BF16, SDPA_BSHD, SDPA_F16, SDPA_THD
    dt, dev = like_q.dtype, like_q.device
    if dt not in (torch.bfloat16, torch.float16):
        raise ValueError(f"unsupported dtype {dt}")
    if like_q.dim() not in (3, 4):
        raise ValueError(f"q: expected [b, s, h, d] or [total, h, d], got {tuple(like_q.shape)}")
    p = SdpaRopeParams()
    p.dtype = SDPA_BF16 if dt == torch.bfloat16 else SDPA_F16
    *rows, p.h_q, p.d = like_q.shape
    if like_k is not None:
        if like_k.dim() != like_q.dim() or list(like_k.shape[:-2]) != rows or like_k.shape[-1] != p.d:
            raise ValueError(f"k: expected {tuple(rows)} rows of heads of {p.d} features like q's, got {tuple(like_k.shape)}")
        p.h_kv = like_k.shape[-2]
    if len(rows) == 1:
        p.layout, p.total = SDPA_THD, rows[0]
    else:
        p.layout, p.b, p.s = SDPA_BSHD, *rows
    if freq.dim() != 1:
        raise ValueError(f"freq: expected [rot / 2], got {tuple(freq.shape)}")
    p.rot = 2 * freq.shape[0]
    p.freq = _array("freq", freq, freq.shape, dev, (torch.float32,))
    p.n_axes = 1
    if positions.dim() == len(rows) + 1:
        p.n_axes = positions.shape[0]
        if axis is None and p.n_axes != 1:
            raise ValueError("axis: positions of several axes need each pair's axis")
    shape = positions.shape[:1] if positions.dim() == len(rows) + 1 else ()
    p.positions = _array("positions", positions, (*shape, *rows), dev, (torch.int32,))
    if axis is not None:
        p.axis = _array("axis", axis, freq.shape, dev, (torch.int32,))
    if seq_lens is not None:
        if len(rows) == 1:
            raise ValueError("seq_lens: only with [b, s, h, d]")
        p.seq_lens = _array("seq_lens", seq_lens, rows[:1], dev, (torch.int32,))
    if like_k is None and k_weight is not None:
        raise ValueError("k_weight: there is no k")
    if like_k is not None and (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight: both or neither")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            setattr(p, name, _array(name, w, (p.d,), dev, (dt, torch.float32)))
            if name == "k_weight" and w.dtype != q_weight.dtype:
                raise ValueError(f"k_weight: expected dtype {q_weight.dtype}, got {w.dtype}")
            p.weight_f32 = int(w.dtype == torch.float32)
    p.eps, p.weight_offset, p.rot_scale, p.interleaved = eps, weight_offset, rot_scale, int(bool(interleaved))
    return p, dt, dev


def _stream(dev):
    import torch
    return torch._C._cuda_getCurrentRawStream(dev.index or 0)


def _check(code, where):
    if code:
        from . import SdpaError, last_error
        raise SdpaError(code, where, last_error())


def _outputs(p, q, k, out, dt, dev):
    import torch
    if out is None:
        out = torch.empty(q.shape, dtype=dt, device=dev), None if k is None else torch.empty(k.shape, dtype=dt, device=dev)
    oq, ok = out
    p.oq, p.oq_stride = oq.data_ptr(), _rows("out q", oq, q.shape, dev, dt, True)
    if k is not None:
        p.ok, p.ok_stride = ok.data_ptr(), _rows("out k", ok, k.shape, dev, dt, True)
    return oq, ok


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
    p, dt, dev = _params(q, k, positions, freq, q_weight, k_weight, eps, weight_offset, axis, interleaved, rot_scale, seq_lens)
    p.q, p.q_stride = q.data_ptr(), _rows("q", q, q.shape, dev, dt)
    if k is not None:
        p.k, p.k_stride = k.data_ptr(), _rows("k", k, k.shape, dev, dt)
    oq, ok = _outputs(p, q, k, out, dt, dev)
    _check(sdpa_rope_fwd(p, _stream(dev)), "sdpa_rope_fwd")
    return oq, ok


def qk_rotate_backward(dq, dk, q, k, positions, freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                       weight_offset: float = 0.0, axis=None, interleaved: bool = False, rot_scale: float = 1.0, seq_lens=None,
                       out=None, workspace=None):
    """Gradients of qk_rotate: (dq, dk, dq_weight, dk_weight) from those of its
    outputs, dq and dk, and its inputs q and k (not read, and may be None, without
    weights). The other arguments are qk_rotate's; the weights' gradients are fp32
    [d] (None without weights). out: (dq, dk) to write to, the given ones too.
    """
    import torch
    p, dt, dev = _params(dq, dk, positions, freq, q_weight, k_weight, eps, weight_offset, axis, interleaved, rot_scale, seq_lens)
    p.gq, p.gq_stride = dq.data_ptr(), _rows("dq", dq, dq.shape, dev, dt)
    if dk is not None:
        p.gk, p.gk_stride = dk.data_ptr(), _rows("dk", dk, dk.shape, dev, dt)
    wq = wk = None
    n = 0
    if q_weight is not None:
        p.q, p.q_stride = q.data_ptr(), _rows("q", q, dq.shape, dev, dt)
        wq = torch.empty(p.d, dtype=torch.float32, device=dev)
        p.dq_weight = wq.data_ptr()
        if dk is not None:
            p.k, p.k_stride = k.data_ptr(), _rows("k", k, dk.shape, dev, dt)
            wk = torch.empty(p.d, dtype=torch.float32, device=dev)
            p.dk_weight = wk.data_ptr()
    oq, ok = _outputs(p, dq, dk, out, dt, dev)
    if q_weight is not None:
        if workspace is None:
            n = sdpa_rope_bwd_workspace_bytes(p)
            if n == 0:
                from . import SDPA_ERR_INVALID_ARG, SdpaError, last_error
                raise SdpaError(SDPA_ERR_INVALID_ARG, "sdpa_rope_bwd_workspace_bytes", last_error())
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous uint8 tensor")
        n = workspace.numel()
    _check(sdpa_rope_bwd(p, workspace.data_ptr() if n else 0, n, _stream(dev)), "sdpa_rope_bwd")
    return oq, ok, wq, wk
