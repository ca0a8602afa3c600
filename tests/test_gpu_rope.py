"""Norm and rotation of queries and keys on the GPU, and their gradients, against
plain 64-bit forms (rope_ref.py)."""
import math

import pytest
import torch

import rope_ref as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def close(name, got, want, tol):
    got = got.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{name}: {int((~torch.isfinite(got)).sum())} values not finite"
    over = (got - want).abs() - tol
    assert got.numel() == 0 or over.max() <= 0, f"{name}: over the bound by {float(over.max()):.3e}"


def freqs(rot):
    return (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float()


# rows (b, s) or total, h_q, h_kv, d, rot, dtype, extras
CASES = {
    "one_token": ((1, 1), 2, 1, 64, 64, "bf16", {}),
    "one_token_d128": (1, 48, 6, 128, 128, "f16", dict(norm=True)),
    "plain": ((2, 33), 4, 4, 64, 64, "bf16", dict(norm=True)),
    "gqa_packed": (77, 12, 3, 128, 128, "bf16", dict(norm=True, f32=True)),
    "neighbours": ((3, 17), 5, 1, 128, 128, "f16", dict(norm=True, interleaved=True)),
    "neighbours_part": (50, 3, 2, 64, 26, "bf16", dict(interleaved=True)),
    "half_of_the_features": (50, 7, 2, 128, 64, "bf16", dict(norm=True)),
    "halves_of_16": (50, 7, 2, 128, 16, "f16", dict(norm=True)),
    "odd_halves": (50, 7, 2, 128, 92, "bf16", dict(norm=True)),
    "odd_halves_d64": ((2, 9), 9, 3, 64, 2, "f16", dict(norm=True)),
    "odd_halves_d64_plain": ((2, 9), 9, 3, 64, 58, "bf16", {}),
    "no_rotation": (40, 3, 1, 64, 0, "bf16", dict(norm=True)),
    "nothing_at_all": (40, 3, 1, 128, 0, "bf16", {}),
    "three_axes": ((2, 40), 6, 2, 128, 128, "bf16", dict(norm=True, axes=3)),
    "two_axes_mixed": (61, 6, 2, 64, 44, "f16", dict(axes=2, interleaved=True)),
    "queries_alone": ((2, 21), 5, 0, 64, 64, "bf16", dict(norm=True)),
    "padded": ((4, 19), 3, 2, 64, 64, "bf16", dict(norm=True, lens=[19, 0, 1, 12])),
    "padded_plain": ((4, 19), 3, 2, 128, 60, "f16", dict(lens=[19, 0, 1, 12])),
    "far": ((2, 9), 2, 2, 128, 128, "f16", dict(far=2 ** 31 - 20, norm=True)),
    "before_zero": ((2, 9), 2, 2, 64, 64, "f16", dict(far=-(2 ** 31), norm=True)),
    "scaled": (30, 2, 2, 64, 32, "bf16", dict(norm=True, rot_scale=1.37, offset=1.0)),
    "many_tokens": (5000, 3, 1, 64, 64, "bf16", dict(norm=True)),
    "many_heads": (3, 200, 41, 128, 128, "bf16", dict(norm=True)),
    "no_rows": ((2, 0), 2, 2, 64, 64, "bf16", dict(norm=True)),
}


def case(name):
    rows, h_q, h_kv, d, rot, dtype, x = CASES[name]
    seed = 500 + 11 * list(CASES).index(name)
    shape = rows if isinstance(rows, tuple) else (rows,)
    dt = DT[dtype]
    t = dict(q=randn(seed, *shape, h_q, d, dtype=dt), k=randn(seed + 1, *shape, h_kv, d, dtype=dt) if h_kv else None,
             gq=randn(seed + 2, *shape, h_q, d, dtype=dt), gk=randn(seed + 3, *shape, h_kv, d, dtype=dt) if h_kv else None)
    axes = x.get("axes", 1)
    g = torch.Generator().manual_seed(seed + 4)
    pos = torch.randint(0, 5000, (axes, *shape), generator=g)
    if "far" in x:
        pos = pos % 20 + x["far"]
    pos = pos.to(torch.int32)
    t["pos"] = pos if axes > 1 else pos[0]
    t["axis"] = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.int32) if axes > 1 else None
    t["freq"] = freqs(rot)
    wt = torch.float32 if x.get("f32") else dt
    for i, n in enumerate("qk"):
        t["w" + n] = (1 + 0.3 * randn(seed + 5 + i, d)).to(wt) if x.get("norm") and t[n] is not None else None
    kw = dict(interleaved=x.get("interleaved", False), rot_scale=x.get("rot_scale", 1.0), weight_offset=x.get("offset", 0.0))
    lens = x.get("lens")
    if lens:
        for i, n in enumerate(lens):
            for f in ("q", "k", "gq", "gk"):
                t[f][i, n:] = math.nan
    return t, kw, lens


def dev(t):
    return None if t is None else t.cuda()


def call(t, kw, lens, back, **more):
    import sliding_window_attention_sdpa_gb300 as swa
    kw = dict(kw, q_weight=dev(t["wq"]), k_weight=dev(t["wk"]), axis=dev(t["axis"]),
              seq_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda(), **more)
    if back:
        return swa.qk_rotate_backward(dev(t["gq"]), dev(t["gk"]), dev(t["q"]), dev(t["k"]), dev(t["pos"]), dev(t["freq"]), **kw)
    return swa.qk_rotate(dev(t["q"]), dev(t["k"]), dev(t["pos"]), dev(t["freq"]), **kw)


def cleared(x, lens):
    """Padding rows as zeros."""
    x = x.clone()
    for i, n in enumerate(lens or []):
        x[i, n:] = 0
    return x


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    t, kw, lens = case(name)
    got = call(t, kw, lens, False)
    for n, y in zip("qk", got):
        if t[n] is None:
            assert y is None
            continue
        want, tol = P.forward(cleared(t[n], lens), t["w" + n], t["pos"], t["freq"], axis=t["axis"], **kw)
        close(n, y, cleared(want, lens), cleared(tol, lens))
    again = call(t, kw, lens, False)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    t, kw, lens = case(name)
    got = call(t, kw, lens, True)
    for i, n in enumerate("qk"):
        if t[n] is None:
            assert got[i] is None and got[2 + i] is None
            continue
        dx, tol, dw, tol_w = P.backward(cleared(t["g" + n], lens), cleared(t[n], lens), t["w" + n], t["pos"], t["freq"], axis=t["axis"], **kw)
        close("d" + n, got[i], cleared(dx, lens), cleared(tol, lens))
        if dw is None:
            assert got[2 + i] is None
        else:
            assert got[2 + i].dtype == torch.float32
            close(f"d{n}_weight", got[2 + i], dw, tol_w)
    # bitwise repeatable, in a dirty workspace too
    again = call(t, kw, lens, True, workspace=torch.full((1 << 21,), 255, dtype=torch.uint8, device="cuda"))
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("d,dtype,interleaved", [(64, "bf16", False), (128, "f16", True), (128, "bf16", False)])
def test_strides_and_in_place(d, dtype, interleaved):
    """Queries and keys cut from one projection, rotated where they are; their
    neighbours (the values) stay as they were. Broadcast gradients are taken."""
    import sliding_window_attention_sdpa_gb300 as swa
    b, s, h_q, h_kv = 2, 13, 6, 2
    qkv = randn(7, b, s, h_q + 2 * h_kv, d, dtype=DT[dtype])
    w = [(1 + 0.2 * randn(8 + i, d)).to(DT[dtype]) for i in range(2)]
    pos, freq = torch.arange(s, dtype=torch.int32).expand(b, s).contiguous(), freqs(d)
    g = qkv.cuda()
    q, k = g[:, :, :h_q], g[:, :, h_q:h_q + h_kv]
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), interleaved=interleaved)
    plain = swa.qk_rotate(q, k, pos.cuda(), freq.cuda(), **kw)
    out = swa.qk_rotate(q, k, pos.cuda(), freq.cuda(), out=(q, k), **kw)
    assert out[0] is q and torch.equal(q, plain[0]) and torch.equal(k, plain[1])
    assert torch.equal(g[:, :, h_q + h_kv:].cpu(), qkv[:, :, h_q + h_kv:])
    for n, y, x in (("q", q, qkv[:, :, :h_q]), ("k", k, qkv[:, :, h_q:h_q + h_kv])):
        close(n, y, *P.forward(x, w[n == "k"], pos, freq, interleaved=interleaved))
    one = randn(9, 1, 1, 1, d, dtype=DT[dtype]).cuda()
    x = qkv.cuda()
    q, k = x[:, :, :h_q], x[:, :, h_q:h_q + h_kv]
    got = swa.qk_rotate_backward(one.expand(b, s, h_q, d), one.expand(b, s, h_kv, d), q, k, pos.cuda(), freq.cuda(), **kw)
    full = [one.expand(b, s, h, d).contiguous() for h in (h_q, h_kv)]
    want = swa.qk_rotate_backward(*full, q, k, pos.cuda(), freq.cuda(), **kw)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    place = swa.qk_rotate_backward(*full, q, k, pos.cuda(), freq.cuda(), out=tuple(full), **kw)
    assert all(torch.equal(a, c) for a, c in zip(place, want)) and torch.equal(full[0], want[0])


def test_zero_rows_and_extremes():
    """A head of zeros stays zero (and its gradient finite); the largest and the
    smallest magnitudes of the types."""
    import sliding_window_attention_sdpa_gb300 as swa
    freq, pos = freqs(64).cuda(), torch.arange(4, dtype=torch.int32).cuda()
    for dt in (torch.bfloat16, torch.float16):
        x = randn(3, 4, 2, 64, dtype=dt)
        x[0] = 0
        x[1] = torch.finfo(dt).max if dt == torch.float16 else 1e18
        x[2] = 2.0 ** -24
        w = torch.ones(64, dtype=dt)
        y, _ = swa.qk_rotate(x.cuda(), None, pos, freq, q_weight=w.cuda())
        close("y", y, *P.forward(x, w, pos.cpu(), freq.cpu()))
        g = randn(4, 4, 2, 64, dtype=dt)
        dx, _, dw, _ = swa.qk_rotate_backward(g.cuda(), None, x.cuda(), None, pos, freq, q_weight=w.cuda(), eps=1e-2)
        want, tol, ww, tw = P.backward(g, x, w, pos.cpu(), freq.cpu(), eps=1e-2)
        close("dx", dx, want, tol)
        close("dw", dw, ww, tw)


def test_fast_turns_far_away():
    """Frequencies of many turns a position, at the last positions: against whole-number arithmetic (a 64-bit float
    loses 2^-14 of a turn there). f16 rows (1, 0) and (0, 1) of each pair show cosine and sine."""
    import sliding_window_attention_sdpa_gb300 as swa
    d, half = 64, 32
    freq = (torch.rand(half, generator=torch.Generator().manual_seed(9)) * 3000 - 1500).float()
    freq[:3] = torch.tensor([0.0, 1.0, -1e6])
    pos = torch.tensor([2 ** 31 - 1 - 977 * i for i in range(20)] + [-2 ** 31 + 31 * i for i in range(20)], dtype=torch.int32)
    inv = 0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E4107F9458EAF7AEF1586DC91B8E909374B801  # 2^328 / (2 pi), whole
    x = torch.zeros(len(pos), 1, d, dtype=torch.float16)
    x[..., :half] = 1
    y, _ = swa.qk_rotate(x.cuda(), None, pos.cuda(), freq.cuda())
    y = y.double().cpu()[:, 0]
    for i in range(half):
        num, den = float(freq[i]).as_integer_ratio()
        for r in range(len(pos)):
            part = (int(pos[r]) * num * inv // den) % (1 << 328)
            a = 2 * math.pi * (part / (1 << 328))
            for got, want in ((y[r, i], math.cos(a)), (y[r, half + i], math.sin(a))):
                assert abs(float(got) - want) <= 2.0 ** -11 * abs(want) + 2.0 ** -19 + 2.0 ** -25, (i, r, float(got), want)


def test_nan_and_infinity_stay_in_their_head():
    import sliding_window_attention_sdpa_gb300 as swa
    x = randn(3, 5, 3, 128, dtype=torch.bfloat16)
    clean = x.clone()
    x[1, 2, 7], x[3, 0, 100] = math.nan, math.inf
    w, pos, freq = torch.ones(128, dtype=torch.bfloat16).cuda(), torch.arange(5, dtype=torch.int32).cuda(), freqs(128).cuda()
    y, _ = swa.qk_rotate(x.cuda(), None, pos, freq, q_weight=w)
    z, _ = swa.qk_rotate(clean.cuda(), None, pos, freq, q_weight=w)
    assert torch.isnan(y[1, 2]).all() and not torch.isfinite(y[3, 0]).all()
    keep = torch.ones(5, 3, dtype=torch.bool)
    keep[1, 2] = keep[3, 0] = False
    assert torch.equal(y[keep.cuda()], z[keep.cuda()])
    # features that are not rotated do not see the others' NaN
    y, _ = swa.qk_rotate(x.cuda(), None, pos, freqs(64).cuda())
    assert torch.equal(y[..., 64:][1, 2], x[..., 64:][1, 2].cuda())


@pytest.mark.parametrize("back", [False, True])
def test_captured_and_on_another_stream(back):
    """A captured call, replayed on other values (positions too), gives what an
    eager one gives; so does a call on a stream of its own."""
    import sliding_window_attention_sdpa_gb300 as swa
    t, kw, _ = case("gqa_packed")
    c = {n: dev(x) for n, x in t.items()}
    kw = dict(kw, q_weight=c["wq"], k_weight=c["wk"])

    def step():
        if back:
            return swa.qk_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], c["pos"], c["freq"], **kw)
        return swa.qk_rotate(c["q"], c["k"], c["pos"], c["freq"], **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    c["q"].normal_()
    c["gk"].normal_()
    c["pos"].add_(1000)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_with_the_attention_it_feeds():
    """Forward and backward of the attention between the two calls: each stage's
    outputs go into the next, and the gradients come out as the formula has them."""
    import sliding_window_attention_sdpa_gb300 as swa
    b, s, h_q, h_kv, d = 2, 130, 4, 2, 64
    dt = torch.bfloat16
    q0, k0, v = randn(1, b, s, h_q, d, dtype=dt), randn(2, b, s, h_kv, d, dtype=dt), randn(3, b, s, h_kv, d, dtype=dt)
    do = randn(4, b, s, h_q, d, dtype=dt)
    w = [(1 + 0.2 * randn(5 + i, d)).to(dt) for i in range(2)]
    pos, freq = torch.arange(s, dtype=torch.int32).expand(b, s).contiguous(), freqs(d)
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda())
    q, k = swa.qk_rotate(q0.cuda(), k0.cuda(), pos.cuda(), freq.cuda(), **kw)
    o, lse = swa.forward(q, k, v.cuda(), scale=d ** -0.5, window_left=40)
    dq, dk, dv, _ = swa.backward(q, k, v.cuda(), o, do.cuda(), lse, scale=d ** -0.5, window_left=40, check_status=True)
    dq0, dk0, dwq, dwk = swa.qk_rotate_backward(dq, dk, q0.cuda(), k0.cuda(), pos.cuda(), freq.cuda(), **kw)
    for n, x, g, dx, dw, wt in (("q", q0, dq, dq0, dwq, w[0]), ("k", k0, dk, dk0, dwk, w[1])):
        want, tol, ww, tw = P.backward(g.cpu(), x, wt, pos, freq)
        close("d" + n, dx, want, tol)
        close(f"d{n}_weight", dw, ww, tw)
