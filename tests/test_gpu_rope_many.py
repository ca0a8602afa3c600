"""Norm and rotation where each warp takes several units, one after the other: ragged
batches (padding between real rows), several axes, every kind of pair. The weights'
gradients are held to the depth of their sums, so that one head of one row that is left
out or counted twice shows."""
import pytest
import torch

import rope_ref as P
from test_gpu_rope import DT, cleared, close, call, freqs, randn

pytestmark = pytest.mark.gpu

LENS = [1000, 0, 1, 999, 513, 700, 37, 850, 1000]
# rows (b, s) or total, h_q, h_kv, d, rot, dtype, axes, interleaved, lens
CASES = {
    "ragged": ((9, 1000), 2, 1, 64, 64, "bf16", 1, False, LENS),
    "ragged_axes": ((9, 1000), 1, 2, 128, 128, "f16", 2, False, LENS),
    "ragged_odd_halves": ((9, 1000), 2, 1, 128, 92, "bf16", 1, False, LENS),
    "ragged_neighbours": ((9, 1000), 2, 2, 64, 26, "f16", 3, True, LENS),
    "axes": (7001, 2, 1, 64, 64, "bf16", 3, False, None),
    "odd_halves_axes": (7001, 1, 2, 64, 58, "f16", 2, False, None),
    "neighbours": (7001, 2, 1, 128, 128, "bf16", 1, True, None),
    "part": (7001, 1, 1, 128, 32, "f16", 1, False, None),
}
# a lane's terms (rows of a warp: at most 5 a tensor), those of the lanes, warps and CTAs that are added behind them
# (2, 8, 304 / 8 and 8): 61 sums in a row at most
DEPTH = 64


def case(name):
    rows, h_q, h_kv, d, rot, dtype, axes, interleaved, lens = CASES[name]
    seed, dt = 7000 + 17 * list(CASES).index(name), DT[dtype]
    shape = rows if isinstance(rows, tuple) else (rows,)
    t = {n: randn(seed + i, *shape, h, d, dtype=dt) for i, (n, h) in enumerate((("q", h_q), ("k", h_kv), ("gq", h_q), ("gk", h_kv)))}
    g = torch.Generator().manual_seed(seed + 4)
    pos = torch.randint(0, 5000, (axes, *shape), generator=g).to(torch.int32)
    t["pos"] = pos if axes > 1 else pos[0]
    t["axis"] = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.int32) if axes > 1 else None
    t["freq"] = freqs(rot)
    for i, n in enumerate("qk"):
        t["w" + n] = (1 + 0.3 * randn(seed + 5 + i, d)).to(dt)
    for i, n in enumerate(lens or []):
        for f in ("q", "k", "gq", "gk"):
            t[f][i, n:] = float("nan")
    return t, dict(interleaved=interleaved), lens


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    t, kw, lens = case(name)
    for n, y in zip("qk", call(t, kw, lens, False)):
        want, tol = P.forward(cleared(t[n], lens), t["w" + n], t["pos"], t["freq"], axis=t["axis"], **kw)
        close(n, y, cleared(want, lens), cleared(tol, lens))


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    t, kw, lens = case(name)
    got = call(t, kw, lens, True)
    for i, n in enumerate("qk"):
        g, x = cleared(t["g" + n], lens), cleared(t[n], lens)
        dx, tol, dw, _ = P.backward(g, x, t["w" + n], t["pos"], t["freq"], axis=t["axis"], **kw)
        close("d" + n, got[i], cleared(dx, lens), cleared(tol, lens))
        # dw = sum of u n: fp32's part in each term as in rope_ref, and the depth of the sums
        f, xx, d = g.double(), x.double(), x.shape[-1]
        at, _, _ = P.partner(2 * len(t["freq"]), d, kw["interleaved"])
        cs, sn = P.turns(t["pos"], t["freq"], t["axis"], d, kw["interleaved"], 1.0, True)
        u = f * cs + f[..., at] * sn
        norm = xx * torch.rsqrt((xx * xx).mean(-1, keepdim=True) + 1e-6)
        term = (u * norm).abs().reshape(-1, d)
        own = (P.E * (f.abs() + f[..., at].abs() + u.abs()) * norm.abs()).reshape(-1, d)
        bound = own.sum(0) + term.sum(0) * DEPTH * 2.0 ** -24
        # one head of one row is more than twice the bound in some feature
        assert ((term > 2 * bound).any(-1) | (term == 0).all(-1)).all()
        close(f"d{n}_weight", got[2 + i], dw, bound)
