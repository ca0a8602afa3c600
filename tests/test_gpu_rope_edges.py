"""Norm and rotation on the GPU at their edges."""
import math

import pytest
import torch

import rope_ref as P

pytestmark = pytest.mark.gpu

# 2^328 / (2 pi), whole
INV = 0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E4107F9458EAF7AEF1586DC91B8E909374B801


@pytest.mark.parametrize("d,interleaved,axes", [(64, 0, 1), (128, 0, 3), (128, 1, 1)])
@pytest.mark.parametrize("packed", [False, True])
def test_no_rows_and_no_arrays(packed, d, interleaved, axes):
    """A backward pass over no rows needs no positions and no frequencies (NULL through the C
    ABI): the weights' gradients are zeros."""
    import sliding_window_attention_sdpa_gb300 as swa
    p = swa.SdpaRopeParams()
    p.dtype, p.layout, p.interleaved = swa.SDPA_BF16, swa.SDPA_THD if packed else swa.SDPA_BSHD, interleaved
    p.b, p.s, p.total, p.h_q, p.h_kv, p.d, p.rot, p.n_axes = (0, 0, 0, 4, 2, d, d, axes) if packed else (2, 0, 0, 4, 2, d, d, axes)
    p.eps, p.rot_scale = 1e-6, 1.0
    for n, h in (("q", 4), ("k", 2), ("gq", 4), ("gk", 2), ("oq", 4), ("ok", 2)):
        setattr(p, n + "_stride", swa._i64x3(0, h * d, d))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((2, d), math.nan, device="cuda")
    p.q_weight = p.k_weight = w.data_ptr()
    p.dq_weight, p.dk_weight = dw[0].data_ptr(), dw[1].data_ptr()
    n = swa.sdpa_rope_bwd_workspace_bytes(p)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert not p.freq and not p.positions
    assert swa.sdpa_rope_bwd(p, ws.data_ptr(), n, stream) == swa.SDPA_OK, swa.last_error()
    assert swa.sdpa_rope_fwd(p, stream) == swa.SDPA_OK, swa.last_error()
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_turns_backwards_far_away():
    """Negative frequencies, slow ones too, at the last positions, where the angle comes near a whole number of turns: the
    sine there is small, and f16 shows its error. Against whole-number arithmetic."""
    import sliding_window_attention_sdpa_gb300 as swa
    one, near = 1 << 328, 1 << (328 - 16)
    rows = []
    g = torch.Generator().manual_seed(4)
    freqs = (-(10.0 ** (torch.rand(32, generator=g, dtype=torch.float64) * 7.5 - 5))).float()       # -1e-5 to -300
    for i, f in enumerate(freqs.tolist()):
        num, den = f.as_integer_ratio()
        step = (num * INV // den) % one
        for first in (2 ** 31 - 1, -2 ** 31 + 2 ** 15):
            for pos in range(first, first - 2 ** 15, -1):
                part = pos * step % one
                if part < near or one - part < near:
                    rows.append((i, pos, (part if part < near else part - one) / one))
                    break
    assert len(rows) >= 16
    x = torch.zeros(len(rows), 1, 64, dtype=torch.float16)
    x[..., :32] = 1
    pos = torch.tensor([r[1] for r in rows], dtype=torch.int32)
    y, _ = swa.qk_rotate(x.cuda(), None, pos.cuda(), freqs.cuda())
    y = y.double().cpu()
    for r, (i, _, turn) in enumerate(rows):
        want = math.sin(2 * math.pi * turn)
        # 2^-24 of a turn; the sine's and the products' roundings in fp32; f16
        tol = 2 * math.pi * 2.0 ** -24 + (2.0 ** -22 + 2.0 ** -11) * abs(want) + 2.0 ** -25
        assert abs(float(y[r, 0, 32 + i]) - want) <= tol, (float(freqs[i]), rows[r], float(y[r, 0, 32 + i]), want)


@pytest.mark.parametrize("d", [64, 128])
def test_heads_of_zeros_under_the_smallest_eps(d):
    """r = eps^(-1/2) is a number whatever eps is, r^2 need not be: dx = r u w has no part of it."""
    import sliding_window_attention_sdpa_gb300 as swa
    eps, rows = 2.0 ** -149, 5
    x = torch.zeros(rows, 2, d, dtype=torch.bfloat16)
    gen = torch.Generator().manual_seed(d)
    g = torch.randn(rows, 2, d, generator=gen).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(d, generator=gen)).to(torch.bfloat16)
    pos, freq = torch.arange(rows, dtype=torch.int32), (10.0 ** (-torch.arange(d // 2) / 16)).float()
    kw = dict(q_weight=w.cuda(), eps=eps)
    dx, _, dw, _ = swa.qk_rotate_backward(g.cuda(), None, x.cuda(), None, pos.cuda(), freq.cuda(), **kw)
    want, tol, _, _ = P.backward(g, x, w, pos, freq, eps=eps)
    assert torch.isfinite(dx).all() and (dw == 0).all()
    assert ((dx.double().cpu() - want).abs() <= tol).all()
    y, _ = swa.qk_rotate(x.cuda(), None, pos.cuda(), freq.cuda(), **kw)
    assert (y == 0).all()
