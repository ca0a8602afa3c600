"""CPU checks of the norm and rotation of queries and keys: struct size, every
refusal that needs no device, and the tests' own formula of the gradients against
differences of the forward formula."""
import ctypes

import pytest
import torch

import rope_ref as P
import sliding_window_attention_sdpa_gb300 as swa


@pytest.fixture(scope="module", autouse=True)
def lib():
    swa._build.build()
    return swa.load()


def test_struct_matches_binding(lib):
    assert lib.sdpa_rope_params_bytes() == ctypes.sizeof(swa.SdpaRopeParams)


def params(**kw):
    p = swa.SdpaRopeParams()
    p.dtype, p.layout = swa.SDPA_BF16, swa.SDPA_BSHD
    p.b, p.s, p.h_q, p.h_kv, p.d, p.rot, p.n_axes = 2, 5, 4, 2, 64, 64, 1
    p.eps, p.rot_scale = 1e-6, 1.0
    st = swa._i64x3(5 * 4 * 64, 4 * 64, 64)
    for n in ("q", "k", "gq", "gk", "oq", "ok"):
        setattr(p, n + "_stride", st)
        setattr(p, n, 4096)
    p.positions = p.freq = p.q_weight = p.k_weight = p.dq_weight = p.dk_weight = 4096
    for k, v in kw.items():
        setattr(p, k, v)
    return p


INVALID, UNSUP = swa.SDPA_ERR_INVALID_ARG, swa.SDPA_ERR_UNSUPPORTED
ODD, MINUS = swa._i64x3(1280, 260, 64), swa._i64x3(-8, 8, 8)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(dtype=3), INVALID, "dtype"), (dict(layout=2), INVALID, "layout"),
    (dict(b=-1), INVALID, "b=-1"), (dict(s=-1), INVALID, "s=-1"), (dict(layout=1, total=-2), INVALID, "total=-2"),
    (dict(b=2 ** 20, s=2 ** 20), UNSUP, "rows"), (dict(b=2 ** 40, s=2 ** 40), UNSUP, "rows"), (dict(layout=1, total=2 ** 31), UNSUP, "rows"),
    (dict(d=96), UNSUP, "d=96"), (dict(h_q=0), INVALID, "h_q=0"), (dict(h_kv=-1), INVALID, "h_kv=-1"),
    (dict(h_q=2 ** 40), INVALID, "heads"),
    (dict(rot=3), INVALID, "rot=3"), (dict(rot=66), INVALID, "rot=66"), (dict(rot=-2), INVALID, "rot=-2"),
    (dict(n_axes=0), INVALID, "n_axes=0"), (dict(n_axes=9), INVALID, "n_axes=9"),
    (dict(interleaved=2), INVALID, "interleaved=2"), (dict(weight_f32=5), INVALID, "weight_f32=5"),
    (dict(eps=0.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"), (dict(eps=float("inf")), INVALID, "eps"),
    (dict(rot_scale=float("nan")), INVALID, "rot_scale"), (dict(weight_offset=float("inf")), INVALID, "weight_offset"),
    (dict(k_weight=0), INVALID, "both"), (dict(q_weight=0), INVALID, "both"),
    (dict(layout=1, total=5, seq_lens=4096), INVALID, "seq_lens"),
    (dict(q_stride=ODD), INVALID, "q_stride[1]"), (dict(ok_stride=MINUS), INVALID, "ok_stride[0]"),
])
def test_refusals(kw, code, needle):
    p = params(**kw)
    assert swa.sdpa_rope_fwd(p, 0) == code and needle in swa.last_error(), swa.last_error()
    assert swa.sdpa_rope_bwd(p, 4096, 1 << 40, 0) == code and needle in swa.last_error(), swa.last_error()
    assert swa.sdpa_rope_bwd_workspace_bytes(p) == 0 and needle in swa.last_error()


def test_backward_workspace():
    p = params()
    n = swa.sdpa_rope_bwd_workspace_bytes(p)
    assert n >= 2 * 64 * 4
    for ws, have, needle in ((0, n, "non-NULL"), (4096 + 16, n, "aligned"), (4096, n - 1, "need")):
        assert swa.sdpa_rope_bwd(p, ws, have, 0) == swa.SDPA_ERR_WORKSPACE and needle in swa.last_error()
    assert swa.sdpa_rope_bwd(params(gk_stride=ODD), 4096, n, 0) == INVALID and "gk_stride[1]" in swa.last_error()
    assert swa.sdpa_rope_bwd_workspace_bytes(params(q_weight=0, k_weight=0)) == 0 and swa.last_error() == ""


def test_calls_refuse_wrong_tensors():
    q, k = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    pos, freq = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(32)
    w = torch.zeros(64)
    good = dict(q=q, k=k, positions=pos, freq=freq)
    for change, needle in [
            (dict(q=q.float()), "dtype"), (dict(q=q[0, 0]), "expected"), (dict(k=k[:, :4]), "k: expected"),
            (dict(k=k[..., :32]), "k: expected"), (dict(k=k.half()), "k: expected dtype"),
            (dict(positions=pos.long()), "positions: expected dtype"), (dict(positions=pos[:, :4]), "positions: expected shape"),
            (dict(positions=torch.zeros(3, 2, 5, dtype=torch.int32)), "axis"),
            (dict(positions=torch.zeros(3, 2, 5, dtype=torch.int32), axis=torch.zeros(31, dtype=torch.int32)), "axis: expected shape"),
            (dict(positions=pos.t().contiguous().t()), "positions: must be contiguous"),
            (dict(freq=freq.double()), "freq: expected dtype"), (dict(freq=freq[None]), "freq: expected"),
            (dict(q_weight=w), "both or neither"), (dict(q_weight=w, k_weight=w.bfloat16()), "k_weight: expected dtype"),
            (dict(q_weight=w[:32], k_weight=w), "q_weight: expected shape"), (dict(q_weight=w.half(), k_weight=w.half()), "q_weight: expected dtype"),
            (dict(k=None, q_weight=w, k_weight=w), "no k"),
            (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), "seq_lens: expected shape"),
            (dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), "feature dimension"),
            (dict(out=(q[:, :, :1].expand(2, 5, 4, 64), k)), "share memory"),
            (dict(out=(q, k[:, :, :1])), "out k: expected shape")]:
        kw = dict(good, **change)
        with pytest.raises(ValueError, match=needle):
            swa.qk_rotate(kw.pop("q"), kw.pop("k"), kw.pop("positions"), kw.pop("freq"), **kw)
    with pytest.raises(ValueError, match="q: expected shape"):
        swa.qk_rotate_backward(q, k, q[:, :4], k, pos, freq, q_weight=w, k_weight=w)
    with pytest.raises(ValueError, match="seq_lens"):
        swa.qk_rotate(q[0], k[0], pos[0], freq, seq_lens=torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("rot,interleaved,norm", [(64, False, True), (30, True, True), (16, False, False)])
def test_formula_of_the_gradients_against_differences(rot, interleaved, norm):
    g = torch.Generator().manual_seed(rot)
    x, dy = (torch.randn(3, 2, 64, generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(64, generator=g, dtype=torch.float64) if norm else None
    pos, freq = torch.tensor([0, 5, 900], dtype=torch.int32), torch.rand(rot // 2, generator=g)
    kw = dict(interleaved=interleaved, rot_scale=1.2, weight_offset=0.5, eps=1e-3)
    P.U[torch.float64], P.TINY[torch.float64] = 0.0, 0.0
    dx, _, dw, _ = P.backward(dy, x, w, pos, freq, **kw)
    f = lambda x, w: (P.forward(x, w, pos, freq, **kw)[0] * dy).sum()  # noqa: E731
    # differences at a step of 2^-17: an error of its square times the third derivative, and 2^-52 / 2^-17 of the sum
    step = 2.0 ** -17
    to = torch.randn(x.shape, generator=g, dtype=torch.float64)
    diff = (f(x + step * to, w) - f(x - step * to, w)) / (2 * step)
    assert abs(diff - (dx * to).sum()) <= 1e-7 * (dx * to).abs().sum()
    if norm:
        to = torch.randn(64, generator=g, dtype=torch.float64)
        diff = (f(x, w + step * to) - f(x, w - step * to)) / (2 * step)
        assert abs(diff - (dw * to).sum()) <= 1e-7 * (dw * to).abs().sum()
