"""The cache in 4 bits on the GPU against plain 64-bit forms (cache4_ref.py):
append, read, forward, and all three together as a decoding loop calls them.
Bytes that no key holds are 0xff, scales that are NaN, and table entries that are
not to be read are wild, so any use of them shows."""
import math

import numpy as np
import pytest
import torch

import cache4_ref as Q
import cache_ref as R
import test_gpu_cache as T

pytestmark = pytest.mark.gpu

dev, randn, close, same = T.dev, T.randn, T.close, T.same


def layout(seed, lens, h_kv, d, dtype, page, room=0, **kw):
    """R.make with pages of whole groups (one run: room rounded up)."""
    most = max([n + room for n in lens] + [1])
    lay = R.make(seed, lens, h_kv, d, dtype, page, room=room if page else -(-most // 16) * 16 - max(lens + [0]), **kw)
    assert lay.k.shape[1] % 16 == 0
    return lay


def read_all(c, lens, **kw):
    """Each sequence's rows, as read back."""
    import sliding_window_attention_sdpa_gb300 as swa
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    return swa.cache_read(c, offsets=off, total=int(sum(lens)), check_status=True, **kw)


def want_rows(lay, lens=None):
    lens = lay.lengths.tolist() if lens is None else lens
    out = []
    for x in (lay.k, lay.v):
        parts = [x[lay.where(i, np.arange(n))] for i, n in enumerate(lens)]
        out.append(torch.cat(parts))
    return out


# ------------------------------------------------------------- what rows are held as

def edge_rows(dtype, d):
    """Rows at the borders of the format: every size, ties of codes and of scales, the smallest and
    largest scales, blocks with NaN and infinities, zeros of both signs."""
    dt, g = R.DT[dtype], torch.Generator().manual_seed(3)
    x = torch.randn(600, d, generator=g)
    x[:100] *= 2.0 ** torch.randint(-24, 12, (100, 1), generator=g).float()
    whole = torch.randint(-15, 16, (100, d), generator=g).float() / 2            # x / s on borders where s is a power of two
    whole[:, ::16] = 7.0
    x[100:200] = whole * 2.0 ** torch.randint(-16, 7, (100, 1), generator=g).float()
    tie = torch.randint(-6, 7, (100, d), generator=g).float()
    tie[:, ::16] = 7 * (2 * torch.randint(8, 16, (100, d // 16), generator=g).float() + 1) / 16    # a / 7 between two scales
    x[200:300] = tie * 2.0 ** torch.randint(-12, 5, (100, 1), generator=g).float()
    x[300] = 0.0
    x[301] = -0.0
    x[302] = 65000.0
    x[303, ::3] = -30000.0
    x[304, 5], x[305, 17], x[306, 33] = math.nan, math.inf, -math.inf
    x[307] = 2.0 ** -18
    x[308] = 7 * 2.0 ** -18          # a / 7: half of the smallest scale
    x[309] = 1680.0
    x[310] = 1700.0
    x[311, ::16] = -1920.0
    return x.to(dt)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_held_values(dtype, d):
    import sliding_window_attention_sdpa_gb300 as swa
    x = edge_rows(dtype, d)
    rows = torch.stack([x, x.flip(0)], 1)                    # [600, 2 heads, d]
    k, v = rows, rows.flip(0)
    c = swa.KVCache.empty(1, 2, d, 640, dtype=R.DT[dtype], device="cuda", page_size=64, bits=4)
    swa.cache_append(c, dev(k)[None], dev(v)[None], check_status=True)
    gk, gv = read_all(c, [600])
    same("k", gk, Q.held(k))
    same("v", gv, Q.held(v))


# lens, room, counts (None: all), t, h_kv, d, dtype, page, picked
APPEND = {
    "one_token": ([0], 1, None, 1, 1, 64, "bf16", 16, False),
    "a_token_each": ([0, 1, 15, 16, 17, 31, 63, 64, 300], 1, None, 1, 3, 128, "bf16", 16, False),
    "pairs": ([0, 1, 14, 15, 16, 47, 48], 2, None, 2, 2, 64, "f16", 48, False),
    "picked": ([5, 0, 90, 31], 6, [3, 0, 6, 1], 7, 4, 64, "bf16", 64, True),
    "picked_d128": ([5, 0, 90, 31], 6, [3, 0, 6, 1], 7, 3, 128, "f16", 32, True),
    "one_run": ([5, 0, 90], 40, [40, 33, 7], 40, 2, 128, "bf16", 0, False),
    "many_rows": ([3, 500, 17], 700, [700, 1, 333], 700, 5, 128, "bf16", 64, False),
    "many_rows_d64": ([3, 500, 17], 700, [700, 1, 333], 700, 8, 64, "f16", 112, False),
}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name", APPEND)
def test_append_and_read(name, packed):
    import sliding_window_attention_sdpa_gb300 as swa
    lens, room, counts, t, h_kv, d, dtype, page, picked = APPEND[name]
    if packed and picked:
        packed = False
    seed = 900 + list(APPEND).index(name)
    b, n = len(lens), counts or [t] * len(lens)
    lay = layout(seed, lens, h_kv, d, dtype, page, room=room, tracked=True)
    c = Q.gpu_cache(lay)
    k, v = randn(seed + 1, b, t, h_kv, d, dtype=R.DT[dtype]), randn(seed + 2, b, t, h_kv, d, dtype=R.DT[dtype])
    before = (c.k.clone(), c.v.clone())
    index = None
    if picked:
        rs = np.random.RandomState(seed)
        index = torch.from_numpy(np.stack([rs.randint(0, t, room) for _ in range(b)]).astype(np.int32))   # twice the same too
        pk, pv = (torch.stack([x[i, index[i].long()] for i in range(b)]) for x in (k, v))
        swa.cache_append(c, dev(k), dev(v), index=dev(index), counts=torch.tensor(n, dtype=torch.int32).cuda(), check_status=True)
    elif packed:
        pk, pv = k, v
        off = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
        swa.cache_append(c, *(dev(torch.cat([x[i, :m] for i, m in enumerate(n)])) for x in (k, v)), offsets=off, max_seqlen=max(n),
                         check_status=True)
    else:
        pk, pv = k, v
        swa.cache_append(c, dev(k), dev(v), counts=None if counts is None else torch.tensor(n, dtype=torch.int32).cuda(),
                         check_status=True)
    want = R.append(Q.held_layout(lay), Q.held(pk), Q.held(pv), counts=torch.tensor(n))
    for f in ("lengths", "next_pos", "positions", "weights"):
        same(f, getattr(c, f), getattr(want, f))
    total = [x + m for x, m in zip(lens, n)]
    for got, ref, nm in zip(read_all(c, total), want_rows(want, total), "kv"):
        same(nm, got, ref)
    # pages that hold no new row are as they were
    new_pages = {p for i in range(b) for p in lay.where(i, np.arange(lens[i], total[i]))[0].tolist()}
    others = [p for p in range(lay.k.shape[0]) if p not in new_pages]
    assert torch.equal(c.k[others], before[0][others]) and torch.equal(c.v[others], before[1][others])
    # the same rows one by one are the same bytes
    if not picked and max(n) <= 40:
        one = Q.gpu_cache(lay)
        for r in range(max(n)):
            swa.cache_append(one, dev(k[:, r:r + 1].contiguous()), dev(v[:, r:r + 1].contiguous()),
                             counts=torch.tensor([int(r < m) for m in n], dtype=torch.int32).cuda(), check_status=True)
        assert torch.equal(one.k, c.k) and torch.equal(one.v, c.v) and torch.equal(one.lengths, c.lengths)


def test_append_that_cannot_be_done_leaves_the_cache_alone():
    import sliding_window_attention_sdpa_gb300 as swa
    lens = [20, 5, 30, 12]
    lay = layout(31, lens, 2, 64, "bf16", 16, room=4)
    table = lay.table.clone()
    table[2, 2] = 10 ** 6                         # sequence 2's rows 32 ff. (its new rows begin at 30)
    for what, kw, bad, code in [
            ("room", dict(counts=[4, 4, 1, 40]), [3], swa.SDPA_ERR_BAD_LENGTHS),
            ("count", dict(counts=[4, -1, 1, 4]), [1], swa.SDPA_ERR_BAD_LENGTHS),
            ("page", dict(counts=[4, 4, 4, 4]), [2], swa.SDPA_ERR_BOUNDS)]:
        c = Q.gpu_cache(R.Layout(lay.k, lay.v, table, lay.lengths, None, None, None, lay.real))
        was = (c.k.clone(), c.v.clone())
        k = randn(5, 4, 40, 2, 64, dtype=torch.bfloat16)
        swa.cache_append(c, dev(k), dev(k), counts=torch.tensor(kw["counts"], dtype=torch.int32).cuda())
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == code, what
        want = [n + (0 if i in bad else m) for i, (n, m) in enumerate(zip(lens, kw["counts"]))]
        assert c.lengths.tolist() == want, what
        for i in bad:
            pages = lay.real[i]
            assert torch.equal(c.k[pages], was[0][pages]) and torch.equal(c.v[pages], was[1][pages]), what


# --------------------------------------------------------------------------- read

@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("d,dtype,page", [(64, "bf16", 16), (128, "f16", 48), (128, "bf16", 0), (64, "f16", 64)])
def test_read(bits, d, dtype, page):
    import sliding_window_attention_sdpa_gb300 as swa
    lens = [0, 1, 33, 200, 17]
    lay = layout(41 + d, lens, 3, d, dtype, page, room=5)
    c = Q.gpu_cache(lay) if bits == 4 else T.gpu_cache(lay)
    ref = Q.held_layout(lay) if bits == 4 else lay
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    # padded, from a slot on, into wider tensors whose other columns stay
    start, counts, most = [0, 0, 5, 199, 3], [0, 1, 40, 1, 9], 40
    wide = [torch.full((5, most, 4, d + 8), 7.0, dtype=R.DT[dtype], device="cuda") for _ in range(2)]
    out = tuple(w[:, :, 1:, :d] for w in wide)
    swa.cache_read(c, start=i32(start), counts=i32(counts), max_rows=most, out=out, check_status=True)
    for got, x in zip(out, (ref.k, ref.v)):
        want = torch.zeros(5, most, 3, d, dtype=R.DT[dtype])
        for i in range(5):
            n = min(counts[i], lens[i] - start[i])
            want[i, :n] = x[lay.where(i, np.arange(start[i], start[i] + n))]
        same("padded", got, want)
    assert all((w[:, :, 0] == 7).all() and (w[..., d:] == 7).all() for w in wide)
    # the whole capacity without arguments
    k, v = swa.cache_read(c, check_status=True)
    assert k.shape == (5, c.capacity, 3, d)
    for i, n in enumerate(lens):
        same("all", k[i, :n], ref.k[lay.where(i, np.arange(n))])
        assert (k[i, n:] == 0).all() and (v[i, n:] == 0).all()
    # packed, slots longer and shorter than what there is
    slots = [2, 0, 20, 201, 17]
    off = np.concatenate([[0], np.cumsum(slots)])
    k, v = swa.cache_read(c, offsets=i32(off), total=int(off[-1]), check_status=True)
    for i, n in enumerate(slots):
        m = min(n, lens[i])
        same("packed", v[off[i]:off[i] + m], ref.v[lay.where(i, np.arange(m))])
        assert (k[off[i] + m:off[i] + n] == 0).all()
    # nothing
    k, v = swa.cache_read(c, max_rows=0, check_status=True)
    assert k.shape == (5, 0, 3, d)


@pytest.mark.parametrize("bits", [4, 16])
def test_read_reports(bits):
    import sliding_window_attention_sdpa_gb300 as swa
    lens = [20, 40]
    lay = layout(51, lens, 2, 64, "bf16", 16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    c = Q.gpu_cache(lay) if bits == 4 else T.gpu_cache(lay)
    for kw, code in [(dict(start=i32([21, 0])), swa.SDPA_ERR_BAD_LENGTHS), (dict(start=i32([0, -1])), swa.SDPA_ERR_BAD_LENGTHS),
                     (dict(counts=i32([49, 0])), swa.SDPA_ERR_BAD_LENGTHS), (dict(counts=i32([-1, 0])), swa.SDPA_ERR_BAD_LENGTHS)]:
        swa.cache_read(c, **kw)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == code
    for off in ([3, 4, 10], [0, 4, 8], [0, -5, 10]):
        swa.cache_read(c, offsets=i32(off), total=10)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
    c.page_table[1, 1] = -3
    k, v = swa.cache_read(c)
    with pytest.raises(swa.SdpaError) as e:
        c.check_status()
    assert e.value.code == swa.SDPA_ERR_BOUNDS
    assert (k[1, 16:32] == 0).all() and (v[1, 16:32] == 0).all() and not (k[1, :16] == 0).all()


# ------------------------------------------------------------------------- forward

CASES = [n for n, x in T.FORWARD.items() if x[6] % 16 == 0]


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    lens, t, h_q, h_kv, d, dtype, page, window, x = T.FORWARD[name]
    seed = 100 + 7 * list(T.FORWARD).index(name)
    lay = layout(seed, lens, h_kv, d, dtype, page, evicted=x.get("evicted", False))
    q_lens = x.get("q_lens")
    q, k, v = T.inputs(seed + 1, len(lens), t, h_q, h_kv, d, dtype, q_lens)
    tree = R.tree_masks(seed, len(lens), t, x.get("empty", 0.0)) if x.get("tree") else None
    kw = dict(scale=d ** -0.5, window=window, tree=tree, q_lens=q_lens, sink=randn(seed + 4, h_q) if x.get("sink") else None)
    c = Q.gpu_cache(lay)
    was = (c.k.clone(), c.v.clone())
    o, lse = T.call_forward(c, dev(q), dev(k), dev(v), kw, check_status=True)
    ref = Q.forward(Q.held_layout(lay), q, k, v, dtype=dtype, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)
    # bitwise repeatable, also into given outputs and a given (dirty) workspace
    out, ls = torch.full_like(o, math.nan), torch.full_like(lse, math.nan)
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")
    T.call_forward(c, dev(q), dev(k), dev(v), kw, out=out, lse=ls, workspace=ws, check_status=True)
    assert torch.equal(out, o) and torch.equal(ls, lse)
    assert torch.equal(c.k, was[0]) and torch.equal(c.v, was[1])
