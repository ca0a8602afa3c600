"""The key/value cache's operators on the GPU against plain 64-bit forms
(cache_ref.py): forward over a cache, append, weigh, evict, and all four
together as a decoding loop calls them. Places that no key holds are NaN and
table entries that are not to be read are wild, so any read of them shows."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu


def dev(t):
    return None if t is None else t.cuda()


def gpu_cache(lay, k=None, v=None):
    import sliding_window_attention_sdpa_gb300 as swa
    return swa.KVCache(dev(lay.k) if k is None else k, dev(lay.v) if v is None else v, dev(lay.lengths),
                       page_table=dev(lay.table), next_pos=dev(lay.next_pos), positions=dev(lay.positions),
                       weights=dev(lay.weights))


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def close(name, got, want, tol):
    got = got.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: infinite values differ"
    assert torch.isfinite(got[~inf]).all(), f"{name}: {int((~torch.isfinite(got[~inf])).sum())} values not finite"
    off = (got - want).abs()[~inf]
    over = max([0.0] + (off - tol[~inf]).tolist())
    assert over <= 0, f"{name}: off by up to {float(off.max()):.3e}, over the bound by {over:.3e}"


def same(name, got, want):
    """Equal bits, NaN in the same places."""
    got = got.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN places differ"
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want)), \
        f"{name}: {int((torch.nan_to_num(got) != torch.nan_to_num(want)).sum())} values differ"


def same_cache(c, lay):
    for f in ("k", "v", "lengths", "next_pos", "positions", "weights"):
        want = getattr(lay, f)
        if want is not None:
            same(f, getattr(c, f), want)


def inputs(seed, b, t, h_q, h_kv, d, dtype, q_lens=None):
    dt = R.DT[dtype]
    q, k, v = randn(seed, b, t, h_q, d, dtype=dt), randn(seed + 1, b, t, h_kv, d, dtype=dt), randn(seed + 2, b, t, h_kv, d, dtype=dt)
    if q_lens is not None:
        for i, n in enumerate(q_lens):
            q[i, n:], k[i, n:], v[i, n:] = math.nan, math.nan, math.nan
    return q, k, v


# ------------------------------------------------------------------------- forward

# lens, t, h_q, h_kv, d, dtype, page, window, extras
FORWARD = {
    "one_token_short": ([301], 1, 4, 4, 64, "bf16", 64, -1, {}),
    "one_key": ([1], 1, 2, 1, 128, "f16", 16, -1, {}),
    "no_keys_at_all": ([0, 0], 1, 2, 2, 64, "bf16", 16, -1, {}),
    "lengths_around_tiles": ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129], 1, 8, 2, 64, "bf16", 16, -1, {}),
    "d128_lengths_around_tiles": ([255, 256, 257, 0, 31, 33], 1, 4, 1, 128, "bf16", 64, -1, {}),
    "page_of_one": ([5, 40], 2, 2, 2, 64, "f16", 1, -1, {}),
    "odd_pages": ([100, 7, 213], 3, 6, 2, 128, "bf16", 7, -1, {}),
    "pages_of_24": ([100, 24, 213, 48], 1, 16, 2, 64, "bf16", 24, -1, {}),
    "pages_of_8": ([100, 8, 213, 47, 0, 130], 1, 8, 2, 64, "bf16", 8, -1, {}),
    "pages_of_8_d128": ([100, 8, 213, 47, 0, 130], 2, 4, 1, 128, "f16", 8, 77, dict(sink=True)),
    "pages_of_24_d128": ([100, 24, 213, 47], 1, 8, 2, 128, "bf16", 24, -1, dict(evicted=True)),
    "pages_of_40": ([1100, 24, 213, 47], 3, 10, 2, 64, "f16", 40, 500, {}),
    "one_run": ([100, 7, 213], 4, 6, 2, 64, "bf16", 0, -1, {}),
    "window": ([5, 130, 700, 129, 128], 1, 8, 2, 64, "bf16", 64, 128, {}),
    "window_zero": ([0, 130, 64], 3, 4, 2, 64, "bf16", 16, 0, {}),
    "window_cuts_the_tree": ([40, 300], 13, 4, 2, 64, "f16", 32, 3, dict(tree=True)),
    "window_sink": ([0, 130, 700], 1, 16, 2, 64, "bf16", 64, 100, dict(sink=True)),
    "sink_d128": ([0, 1, 300], 5, 6, 2, 128, "f16", 16, -1, dict(sink=True, tree=True)),
    "tree_9": ([50, 0, 201], 9, 8, 2, 64, "bf16", 64, -1, dict(tree=True)),
    "tree_37_gqa8": ([331, 64], 37, 16, 2, 128, "bf16", 64, -1, dict(tree=True)),
    "tree_64": ([200, 3], 64, 4, 2, 64, "bf16", 16, -1, dict(tree=True)),
    "tree_64_f16_mqa": ([130, 513], 64, 5, 1, 128, "f16", 128, 200, dict(tree=True)),
    "padding_rows": ([90, 10, 0], 11, 4, 1, 64, "bf16", 16, -1, dict(tree=True, empty=0.4)),
    "padding_rows_sink": ([90, 10, 0], 11, 4, 1, 64, "bf16", 16, 7, dict(tree=True, empty=0.4, sink=True)),
    "ragged_rows": ([90, 10, 0, 300], 7, 4, 2, 64, "bf16", 16, -1, dict(q_lens=[7, 0, 1, 5], sink=True)),
    "ragged_tree": ([90, 10, 0, 300], 40, 8, 2, 128, "f16", 64, 50, dict(q_lens=[40, 0, 1, 33], tree=True)),
    "evicted": ([90, 257, 0], 3, 4, 2, 64, "bf16", 32, -1, dict(evicted=True)),
    "evicted_window": ([90, 257, 0], 5, 4, 2, 64, "bf16", 32, 100, dict(evicted=True, sink=True)),
    "evicted_window_many_rows": ([90, 457, 0], 33, 8, 2, 128, "bf16", 64, 100, dict(evicted=True, tree=True)),
    "group_3": ([77, 300], 2, 9, 3, 64, "f16", 64, -1, {}),
    "group_16_mqa": ([300], 1, 16, 1, 128, "bf16", 64, -1, {}),
    "group_71": ([100, 20], 1, 71, 1, 64, "bf16", 64, -1, dict(sink=True)),
    "many_sequences": ([(37 * i) % 90 for i in range(70)], 1, 2, 1, 64, "bf16", 16, -1, {}),
    "long": ([9000, 11], 1, 4, 2, 64, "bf16", 64, -1, {}),
    "long_d128_rows": ([5000], 3, 8, 2, 128, "f16", 128, -1, {}),
    "long_tree": ([4100, 700], 20, 8, 1, 128, "bf16", 64, 4000, dict(tree=True, sink=True)),
    # units of one key tile and of many in one part: a slot of the tile kernel without work, segment after segment
    "short_units": ([(37 * i) % 90 for i in range(60)] + [1500], 5, 16, 2, 64, "bf16", 16, -1, dict(tree=True)),
    "short_units_d128": ([3, 60, 64, 65, 1, 0, 7, 130, 20, 5] * 6 + [900], 3, 8, 1, 128, "f16", 64, -1, {}),
    "short_units_two_tiles": ([3, 60, 64, 65, 1, 0, 7, 130, 20, 5] * 2 + [900], 20, 8, 1, 64, "bf16", 64, -1, dict(tree=True)),
    "short_units_three_tiles": ([3, 60, 1, 0, 130, 5, 700], 37, 8, 1, 128, "bf16", 16, -1, dict(tree=True)),
    "short_units_few_rows": ([3, 60, 64, 65, 1, 0, 7, 130, 20, 5] * 6 + [900], 1, 8, 2, 128, "bf16", 64, -1, {}),
    "mha_many_rows": ([333, 130], 48, 3, 3, 64, "bf16", 64, -1, dict(tree=True)),
    # more sequences than a CTA has threads
    "b_700": ([(37 * i) % 40 for i in range(700)] + [600], 1, 2, 1, 64, "bf16", 64, -1, {}),
    "b_700_many_rows": ([(37 * i) % 40 for i in range(700)] + [600], 3, 8, 1, 128, "bf16", 64, -1, {}),
}


def forward_case(name):
    lens, t, h_q, h_kv, d, dtype, page, window, x = FORWARD[name]
    seed = 100 + 7 * list(FORWARD).index(name)
    lay = R.make(seed, lens, h_kv, d, dtype, page, evicted=x.get("evicted", False))
    q_lens = x.get("q_lens")
    q, k, v = inputs(seed + 1, len(lens), t, h_q, h_kv, d, dtype, q_lens)
    tree = R.tree_masks(seed, len(lens), t, x.get("empty", 0.0)) if x.get("tree") else None
    kw = dict(scale=d ** -0.5, window=window, tree=tree, q_lens=q_lens, sink=randn(seed + 4, h_q) if x.get("sink") else None)
    return lay, q, k, v, kw, dtype


def call_forward(c, q, k, v, kw, **more):
    import sliding_window_attention_sdpa_gb300 as swa
    q_lens = kw["q_lens"]
    return swa.cache_forward(c, q, k, v, scale=kw["scale"], window_left=kw["window"], tree=dev(kw["tree"]),
                             seq_q_lens=None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda(),
                             sink=dev(kw["sink"]), **more)


@pytest.mark.parametrize("name", FORWARD)
def test_forward(name):
    lay, q, k, v, kw, dtype = forward_case(name)
    c = gpu_cache(lay)
    o, lse = call_forward(c, dev(q), dev(k), dev(v), kw, check_status=True)
    ref = R.forward(lay, q, k, v, dtype=dtype, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)
    # bitwise repeatable, also into given outputs and a given (dirty) workspace
    out, ls = torch.full_like(o, math.nan), torch.full_like(lse, math.nan)
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")
    call_forward(c, dev(q), dev(k), dev(v), kw, out=out, lse=ls, workspace=ws, check_status=True)
    assert torch.equal(out, o) and torch.equal(ls, lse)
    same_cache(c, lay)


def test_forward_equals_the_prompt_forward_of_this_package():
    """A chain over a cache is a bottom-right causal forward over all keys."""
    import sliding_window_attention_sdpa_gb300 as swa
    n, t, h_q, h_kv, d = 600, 40, 8, 2, 64
    lay = R.make(5, [n, n], h_kv, d, "bf16", 64)
    q, k, v = inputs(6, 2, t, h_q, h_kv, d, "bf16")
    o, lse = swa.cache_forward(gpu_cache(lay), dev(q), dev(k), dev(v), scale=0.125, window_left=200)
    full = [torch.stack([torch.cat([torch.stack([lay.rows(i, g, n)[x] for g in range(h_kv)], 1), new[i]])
                         for i in range(2)]).cuda() for x, new in ((0, k), (1, v))]
    o2, lse2 = swa.forward(dev(q), *full, scale=0.125, mask_mode=swa.SDPA_MASK_BOTTOM_RIGHT, window_left=200)
    # both round P to bf16 at most and O to bf16: two half steps of values within max |v|
    top = float(full[1].float().abs().max())
    assert (o.float() - o2.float()).abs().max() <= 4 * R.U["bf16"] * top
    assert (lse - lse2).abs().max() <= 1e-4


@pytest.mark.parametrize("t,d,dtype", [(1, 64, "bf16"), (3, 128, "f16"), (40, 128, "bf16"), (40, 64, "f16")])
def test_forward_strides(t, d, dtype):
    """Heads before rows in the pages, Q, K, V cut from one projection, O into
    a wider tensor whose other columns stay as they were."""
    import sliding_window_attention_sdpa_gb300 as swa
    h_q, h_kv, lens = 6, 2, [90, 300, 0]
    b = len(lens)
    lay = R.make(11, lens, h_kv, d, dtype, 16)
    kk, vv = (dev(x.transpose(1, 2).contiguous()).transpose(1, 2) for x in (lay.k, lay.v))
    qkv = randn(12, b, t, (h_q + 2 * h_kv) * d + 8, dtype=R.DT[dtype])
    q, k, v = (x.unflatten(2, (-1, d)) for x in qkv[..., :(h_q + 2 * h_kv) * d].split([h_q * d, h_kv * d, h_kv * d], 2))
    g = dev(qkv)
    gq, gk, gv = (x.unflatten(2, (-1, d)) for x in g[..., :(h_q + 2 * h_kv) * d].split([h_q * d, h_kv * d, h_kv * d], 2))
    wide = torch.full((b, t, h_q + 1, d + 8), 7.0, dtype=R.DT[dtype], device="cuda")
    o, lse = swa.cache_forward(gpu_cache(lay, kk, vv), gq, gk, gv, scale=0.1, out=wide[:, :, 1:, :d], check_status=True)
    ref = R.forward(lay, q, k, v, scale=0.1, dtype=dtype)
    close("o", o, ref.o, ref.tol_o)
    close("lse", lse, ref.lse, ref.tol_lse)
    assert (wide[:, :, 0] == 7).all() and (wide[..., d:] == 7).all()


def test_forward_broadcast_inputs():
    """Expanded inputs (stride 0): one query for all sequences, one key head."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(13, [50, 20, 130], 2, 64, "bf16", 16)
    q = randn(14, 1, 2, 1, 64, dtype=torch.bfloat16).expand(3, 2, 4, 64)
    k = randn(15, 1, 2, 1, 64, dtype=torch.bfloat16).expand(3, 2, 2, 64)
    gq, gk = dev(q[:1, :, :1]).expand(3, 2, 4, 64), dev(k[:1, :, :1]).expand(3, 2, 2, 64)
    o, lse = swa.cache_forward(gpu_cache(lay), gq, gk, gk, scale=0.125, check_status=True)
    ref = R.forward(lay, q, k, k, scale=0.125)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("t,d", [(1, 64), (2, 128), (40, 128), (40, 64)])
def test_forward_extreme_scores(t, d):
    """Scores far apart: one key outweighs the rest, and scores of -40000."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(17, [300, 129], 2, d, "bf16", 64)
    q, k, v = inputs(18, 2, t, 4, 2, d, "bf16")
    lay.k[lay.where(0, [77])] *= 60
    lay.k[lay.where(1, list(range(129)))] *= 200
    kw = dict(scale=1.0, window=-1, tree=None, q_lens=None, sink=None)
    o, lse = call_forward(gpu_cache(lay), dev(q), dev(k), dev(v), kw, check_status=True)
    ref = R.forward(lay, q, k, v, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("t,d,h_q", [(11, 64, 2), (7, 128, 2), (11, 128, 8), (40, 64, 4), (64, 128, 4)])
def test_forward_padding_tokens_hold_anything(t, d, h_q):
    """Tokens that no row admits (masks without their own bit): NaN in them
    reaches no output."""
    lens, h_kv = [90, 10, 0], 2
    lay = R.make(61, lens, h_kv, d, "bf16", 16)
    q, k, v = inputs(62, len(lens), t, h_q, h_kv, d, "bf16")
    tree = R.tree_masks(63, len(lens), t, 0.4)
    for i in range(len(lens)):
        pad = [r for r in range(t) if not int(tree[i, r]) >> r & 1]
        assert 0 < len(pad) < t
        q[i, pad], k[i, pad], v[i, pad] = math.nan, math.nan, math.inf
    kw = dict(scale=d ** -0.5, window=-1, tree=tree, q_lens=None, sink=None)
    o, lse = call_forward(gpu_cache(lay), dev(q), dev(k), dev(v), kw, check_status=True)
    ref = R.forward(lay, q, k, v, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("page", [4, 8, 16, 64, 0])
@pytest.mark.parametrize("t,d", [(1, 64), (2, 64), (2, 128), (40, 128), (40, 64)])
def test_forward_in_front_of_the_window(t, d, page):
    """Keys in front of every row's window may hold anything, pages in front of
    it may be on no page at all (freed ones)."""
    lens, h_q, h_kv, window = [301, 100, 77, 1000], 4, 2, 77
    lay = R.make(64, lens, h_kv, d, "bf16", page)
    for i, n in enumerate(lens):
        if n > window:
            pg, at = lay.where(i, list(range(n - window)))
            lay.k[pg, at], lay.v[pg, at] = math.nan, math.nan
            if page:
                lay.table[i, :(n - window) // page] = -1
    q, k, v = inputs(65, len(lens), t, h_q, h_kv, d, "bf16")
    kw = dict(scale=d ** -0.5, window=window, tree=None, q_lens=None, sink=None)
    o, lse = call_forward(gpu_cache(lay), dev(q), dev(k), dev(v), kw, check_status=True)
    ref = R.forward(lay, q, k, v, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("page", [7, 8, 64])
@pytest.mark.parametrize("t,d,tree", [(1, 64, False), (2, 128, False), (13, 64, True), (40, 128, False), (40, 64, True)])
def test_forward_out_of_the_window_by_position(t, d, tree, page):
    """The same where positions say which keys the windows have: keys in any
    slot that no row's window has may hold anything."""
    lens, h_q, h_kv, window = [301, 100, 77, 700], 4, 2, 60
    lay = R.make(68, lens, h_kv, d, "bf16", page, evicted=True)
    gone = 0
    for i, n in enumerate(lens):
        for h in range(h_kv):
            out = [j for j in range(n) if int(lay.positions[i, h, j]) < int(lay.next_pos[i]) - window]
            pg, at = lay.where(i, out)
            lay.k[pg, at, h], lay.v[pg, at, h] = math.nan, math.nan
            gone += len(out)
        # a page of which no head's windows have a key may be gone
        if page:
            for p in range(-(-n // page)):
                if int(lay.positions[i, :, p * page:min(n, (p + 1) * page)].max()) < int(lay.next_pos[i]) - window:
                    lay.table[i, p] = -1
    assert gone > 1000
    q, k, v = inputs(69, len(lens), t, h_q, h_kv, d, "bf16")
    masks = R.tree_masks(70, len(lens), t) if tree else None
    kw = dict(scale=d ** -0.5, window=window, tree=masks, q_lens=None, sink=None)
    o, lse = call_forward(gpu_cache(lay), dev(q), dev(k), dev(v), kw, check_status=True)
    ref = R.forward(lay, q, k, v, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("t,d", [(1, 64), (40, 128)])
def test_forward_pages_shared_by_sequences(t, d):
    """A common prefix on the same pages, read by all of its sequences; what is
    appended goes behind it."""
    import sliding_window_attention_sdpa_gb300 as swa
    lens, h_q, h_kv, page = [128, 150, 131], 4, 2, 64
    lay = R.make(66, lens, h_kv, d, "bf16", page, room=3 * t)
    for i in (1, 2):
        lay.real[i][:2] = lay.real[0][:2]
        lay.table[i, :2] = lay.table[0, :2]
    q, k, v = inputs(67, len(lens), t, h_q, h_kv, d, "bf16")
    kw = dict(scale=d ** -0.5, window=-1, tree=None, q_lens=None, sink=None)
    c = gpu_cache(lay)
    for _ in range(2):
        o, lse = call_forward(c, dev(q), dev(k), dev(v), kw, check_status=True)
        ref = R.forward(lay, q, k, v, **kw)
        close("lse", lse, ref.lse, ref.tol_lse)
        close("o", o, ref.o, ref.tol_o)
        swa.cache_append(c, dev(k), dev(v), check_status=True)
        lay = R.append(lay, k, v)
        same_cache(c, lay)


@pytest.mark.parametrize("t,d", [(1, 64), (4, 128), (40, 128), (40, 64)])
def test_forward_reports_bad_pages_and_lengths(t, d):
    """Found on the device, reported, nothing outside the buffers read; the
    other sequences' rows are right, keys on bad pages are left out."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(19, [200, 100, 64], 2, d, "bf16", 16)
    q, k, v = inputs(20, 3, t, 4, 2, d, "bf16")
    kw = dict(scale=0.125, window=-1, tree=None, q_lens=None, sink=None)
    for bad in (-1, lay.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        c = gpu_cache(lay)
        c.page_table[0, 12] = bad          # keys 192..199
        o, lse = call_forward(c, dev(q), dev(k), dev(v), kw)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BOUNDS
        c.check_status()                   # cleared
        cut = lay.clone()
        cut.lengths[0] = 192
        cut.next_pos = lay.lengths.clone()  # positions stay those of 200 keys
        cut.positions = torch.arange(cut.cap, dtype=torch.int32).expand(3, 2, -1)
        ref = R.forward(cut, q, k, v, **kw)
        close("lse", lse, ref.lse, ref.tol_lse)
        close("o", o, ref.o, ref.tol_o)
    for n in (-1, lay.cap + 1, 2 ** 31 - 1, -2 ** 31):
        full = R.make(21, [lay.cap, 100, 64], 2, d, "bf16", 16)
        c = gpu_cache(full)
        c.lengths[0] = n
        o, lse = call_forward(c, dev(q), dev(k), dev(v), kw)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
        ref = R.forward(full, q, k, v, **kw)
        close("lse", lse[1:], ref.lse[1:], ref.tol_lse[1:])
        close("o", o[1:], ref.o[1:], ref.tol_o[1:])
    c = gpu_cache(lay)
    o, lse = swa.cache_forward(c, dev(q), dev(k), dev(v), scale=0.125,
                               seq_q_lens=torch.tensor([t, t + 1, -1], dtype=torch.int32).cuda())
    with pytest.raises(swa.SdpaError) as e:
        c.check_status()
    assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
    ref = R.forward(lay, q, k, v, **kw)
    close("o", o[:2], ref.o[:2], ref.tol_o[:2])


def test_forward_no_sequences_and_no_room():
    import sliding_window_attention_sdpa_gb300 as swa
    bf = dict(dtype=torch.bfloat16, device="cuda")
    c = swa.KVCache(torch.zeros(1, 16, 2, 64, **bf), torch.zeros(1, 16, 2, 64, **bf),
                    torch.zeros(0, dtype=torch.int32, device="cuda"),
                    page_table=torch.zeros(0, 3, dtype=torch.int32, device="cuda"))
    o, lse = swa.cache_forward(c, torch.zeros(0, 1, 2, 64, **bf), torch.zeros(0, 1, 2, 64, **bf),
                               torch.zeros(0, 1, 2, 64, **bf), scale=1.0, check_status=True)
    assert o.shape == (0, 1, 2, 64) and lse.shape == (0, 2, 1)
    # no pages at all: a row sees itself only
    c = swa.KVCache(torch.zeros(0, 16, 2, 64, **bf), torch.zeros(0, 16, 2, 64, **bf),
                    torch.zeros(2, dtype=torch.int32, device="cuda"),
                    page_table=torch.zeros(2, 0, dtype=torch.int32, device="cuda"))
    q, k, v = (dev(x) for x in inputs(22, 2, 1, 2, 2, 64, "bf16"))
    o, lse = swa.cache_forward(c, q, k, v, scale=0.125, check_status=True)
    assert torch.equal(o, v)
    # the other calls on a cache without room, and calls without rows
    c = swa.KVCache.empty(2, 2, 64, 0, dtype=torch.bfloat16, device="cuda", track=True)
    swa.cache_append(c, k[:, :0], v[:, :0], check_status=True)
    swa.cache_append(c, k, v, index=torch.zeros(2, 0, dtype=torch.int32, device="cuda"), check_status=True)
    swa.cache_weigh(c, q, lse, scale=1.0, check_status=True)
    swa.cache_evict(c, 0, check_status=True)
    with pytest.raises(swa.SdpaError):
        swa.cache_append(c, k, v, check_status=True)
    assert c.lengths.tolist() == [0, 0] and c.next_pos.tolist() == [0, 0]


# ------------------------------------------------------------------------- append

@pytest.mark.parametrize("d,dtype,page,tracked", [(64, "bf16", 16, True), (128, "f16", 7, True), (128, "bf16", 0, False),
                                                  (64, "f16", 64, False)])
def test_append_forms(d, dtype, page, tracked):
    import sliding_window_attention_sdpa_gb300 as swa
    lens, h_kv, t = [0, 5, 16, 77], 3, 9
    b = len(lens)
    lay = R.make(31, lens, h_kv, d, dtype, page, room=t, tracked=tracked)
    k, v = (randn(s, b, t, h_kv, d, dtype=R.DT[dtype]) for s in (32, 33))
    counts = torch.tensor([0, 9, 1, 4], dtype=torch.int32)
    index = torch.tensor([[0, 8, 3, 3, 1, 2, 7, 5, 4]] * b, dtype=torch.int32)
    for kw in ({}, dict(counts=counts), dict(index=index), dict(index=index, counts=counts), dict(index=index[:, :3].contiguous())):
        c = gpu_cache(lay)
        swa.cache_append(c, dev(k), dev(v), check_status=True, **{n: dev(x) for n, x in kw.items()})
        same_cache(c, R.append(lay, k, v, **kw))
    # packed, strided, with gaps behind the counts
    off = torch.tensor([0, 2, 2, 8, 9], dtype=torch.int32)
    kp, vp = (randn(s, 9, h_kv + 1, d + 8, dtype=R.DT[dtype]) for s in (34, 35))
    for cnt in (None, torch.tensor([1, 0, 5, 1], dtype=torch.int32)):
        c = gpu_cache(lay)
        swa.cache_append(c, dev(kp)[:, 1:, :d], dev(vp)[:, 1:, :d], offsets=dev(off), max_seqlen=6, counts=dev(cnt),
                         check_status=True)
        same_cache(c, R.append(lay, kp[:, 1:, :d], vp[:, 1:, :d], offsets=off, counts=cnt))


def test_append_without_rows_looks_at_the_counts():
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(45, [3, 5], 2, 64, "bf16", 16, room=9, tracked=True)
    none = torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    some = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    no_index = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = gpu_cache(lay)
    for kw in ({}, dict(counts=i32(0, 0))):
        swa.cache_append(c, none, none, check_status=True, **kw)
        swa.cache_append(c, some, some, index=no_index, check_status=True, **kw)
        swa.cache_append(c, none[0], none[0], offsets=i32(0, 0, 0), max_seqlen=0, check_status=True, **kw)
    for args, kw in (((none, none), dict(counts=i32(0, 1))), ((some, some), dict(index=no_index, counts=i32(0, 1))),
                     ((none, none), dict(index=i32(0, 0).view(2, 1))),
                     ((some[0], some[0]), dict(offsets=i32(0, 1, 3), max_seqlen=0)),
                     ((none[0], none[0]), dict(offsets=i32(0, 0, 1), max_seqlen=2))):
        swa.cache_append(c, *args, **kw)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
    same_cache(c, lay)


@pytest.mark.parametrize("page", [64, 100])
def test_append_long_prompts(page):
    """More rows than one CTA takes: the lengths move on once, after all rows."""
    import sliding_window_attention_sdpa_gb300 as swa
    cnt = [1000, 0, 1, 4097]
    lay = R.make(36, [3, 60, 0, 100], 2, 64, "bf16", page, room=4097, tracked=True)
    off = torch.tensor([0, 1000, 1000, 1001, 5098], dtype=torch.int32)
    k, v = (randn(s, sum(cnt), 2, 64, dtype=torch.bfloat16) for s in (37, 38))
    c = gpu_cache(lay)
    swa.cache_append(c, dev(k), dev(v), offsets=dev(off), max_seqlen=4097, check_status=True)
    once = R.append(lay, k, v, offsets=off)
    same_cache(c, once)


def test_append_leaves_what_does_not_fit():
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(41, [3, 40, 8, 20], 2, 64, "bf16", 16, room=9, tracked=True)
    k, v = (randn(s, 4, 9, 2, 64, dtype=torch.bfloat16) for s in (42, 43))
    n = lay.cap
    i32 = torch.int32

    def bad(code, skip, change=None, ref_kw=None, **kw):
        c = gpu_cache(lay)
        want = lay.clone()
        if change:
            change(c)
            change(want)
        swa.cache_append(c, dev(k), dev(v), **{a: dev(x) for a, x in kw.items()})
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == code
        full = R.append(want, k, v, skip=skip, **kw)
        same_cache(c, full)

    B, P = swa.SDPA_ERR_BAD_LENGTHS, swa.SDPA_ERR_BOUNDS
    ok = [9, 9, 9, 9]
    for wrong in (-1, 10, 2 ** 31 - 1):
        bad(B, (1,), counts=torch.tensor([9, wrong, 9, 2], dtype=i32))
    for wrong in (-1, 9, 2 ** 31 - 1, -2 ** 31):
        idx = torch.arange(9, dtype=i32).repeat(4, 1)
        idx[2, 5] = wrong
        bad(B, (2,), index=idx, counts=torch.tensor(ok, dtype=i32))

    def length(x, i, n):
        x.lengths[i] = n
    for wrong in (-1, n - 8, n + 1, 2 ** 31 - 1):
        bad(B, (3,), change=lambda x: length(x, 3, wrong))

    def table(x, value):
        (x.page_table if hasattr(x, "page_table") else x.table)[1, 3] = value    # slots 48..
    for wrong in (-1, lay.k.shape[0], 2 ** 31 - 1):
        bad(P, (1,), change=lambda x: table(x, wrong))


# ------------------------------------------------------------------------- weigh

WEIGH = {
    "token": ([301], 1, 4, 4, 64, "bf16", 64, -1, {}),
    "edges": ([0, 1, 15, 16, 17, 127, 128, 129], 1, 8, 2, 64, "bf16", 16, -1, {}),
    "d128_f16": ([255, 256, 257, 0], 2, 6, 2, 128, "f16", 24, -1, {}),
    "window": ([5, 300, 129], 3, 4, 2, 64, "bf16", 64, 100, {}),
    "window_zero": ([5, 300], 2, 4, 2, 64, "bf16", 64, 0, {}),
    "rows_64": ([200, 30], 64, 4, 2, 128, "bf16", 16, -1, {}),
    "rows_300_window": ([500, 30], 300, 2, 1, 64, "f16", 128, 90, {}),
    "picked_rows": ([90, 100, 0], 12, 4, 2, 64, "bf16", 7, -1, dict(pos=True)),
    "picked_rows_window_gqa8": ([90, 600, 0], 33, 16, 2, 128, "bf16", 64, 40, dict(pos=True)),
    "evicted": ([90, 257, 0], 5, 4, 2, 64, "bf16", 32, -1, dict(evicted=True)),
    "evicted_window": ([90, 257, 0], 5, 40, 2, 128, "bf16", 32, 100, dict(evicted=True, pos=True)),
    "group_5_mqa": ([1100], 1, 5, 1, 128, "f16", 0, -1, {}),
    "long": ([9000, 11], 1, 4, 2, 64, "bf16", 64, -1, {}),
    # several rounds of 256 rows, some of which reach no key of a part
    "rounds": ([1500, 0, 40], 200, 8, 2, 64, "bf16", 64, -1, dict(pos=True)),
    "rounds_window": ([1500, 300, 40], 200, 8, 2, 64, "bf16", 24, 64, dict(pos=True)),
    "rounds_window_odd_pages": ([700, 300], 90, 8, 1, 128, "f16", 7, 30, dict(pos=True)),
    "rounds_evicted": ([300, 500], 70, 8, 1, 128, "bf16", 64, 100, dict(evicted=True, pos=True)),
    "short_units": ([(37 * i) % 90 for i in range(70)] + [1500], 2, 8, 4, 64, "bf16", 16, -1, {}),
    "short_units_window": ([(37 * i) % 90 for i in range(70)] + [1500], 3, 8, 4, 128, "bf16", 16, 5, dict(pos=True)),
    "b_700": ([(37 * i) % 40 for i in range(700)] + [600], 1, 2, 1, 64, "bf16", 64, -1, {}),
    "b_700_many_rows": ([(37 * i) % 40 for i in range(700)] + [600], 17, 4, 1, 64, "f16", 64, -1, dict(pos=True)),
}


@pytest.mark.parametrize("name", WEIGH)
def test_weigh(name):
    import sliding_window_attention_sdpa_gb300 as swa
    lens, t, h_q, h_kv, d, dtype, page, window, x = WEIGH[name]
    seed = 1000 + 7 * list(WEIGH).index(name)
    lay = R.make(seed, lens, h_kv, d, dtype, page, tracked=True, evicted=x.get("evicted", False))
    b = len(lens)
    q = randn(seed + 1, b, t, h_q, d, dtype=R.DT[dtype])
    lse = randn(seed + 2, b, h_q, t) + 4
    lse[0, 0, 0] = -math.inf
    if b > 1:
        lse[1, h_q - 1, t - 1] = math.nan
    q_pos = None
    if x.get("pos"):
        g = torch.Generator().manual_seed(seed)
        q_pos = (torch.rand(b, t, generator=g) * 1.3 * (lay.next_pos[:, None] + 1) - 10).to(torch.int32)
        q[q_pos < 0] = math.nan
    w, tol = R.weigh(lay, q, lse, scale=d ** -0.5, window=window, q_pos=q_pos)
    got = []
    for _ in range(2):
        c = gpu_cache(lay)
        swa.cache_weigh(c, dev(q), dev(lse), scale=d ** -0.5, window_left=window, q_pos=dev(q_pos), check_status=True)
        got.append(c.weights.cpu())
    same("repeat", got[0], got[1])
    assert torch.equal(torch.isnan(got[0]), torch.isnan(lay.weights))
    held = ~torch.isnan(lay.weights)
    close("weights", got[0][held], w[held], tol[held])
    c.weights.copy_(lay.weights)
    same_cache(c, lay)


def test_weigh_without_positions():
    """A cache with weights but no positions: slots count as positions."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(51, [300, 40], 2, 64, "bf16", 64, tracked=True)
    lay.positions = lay.next_pos = None
    q, lse = randn(52, 2, 6, 4, 64, dtype=torch.bfloat16), randn(53, 2, 4, 6) + 4
    for window in (-1, 70):
        c = gpu_cache(lay)
        swa.cache_weigh(c, dev(q), dev(lse), scale=0.125, window_left=window, check_status=True)
        w, tol = R.weigh(lay, q, lse, scale=0.125, window=window)
        held = ~torch.isnan(lay.weights)
        close("weights", c.weights.cpu()[held], w[held], tol[held])


def test_weigh_reports_bad_pages_and_lengths():
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(54, [200, 100], 2, 128, "bf16", 16, tracked=True)
    q, lse = randn(55, 2, 3, 4, 128, dtype=torch.bfloat16), randn(56, 2, 4, 3) + 4
    w, tol = R.weigh(lay, q, lse, scale=0.1)
    for bad in (-1, lay.k.shape[0], 2 ** 31 - 1):
        c = gpu_cache(lay)
        c.page_table[0, 2] = bad             # keys 32..47
        swa.cache_weigh(c, dev(q), dev(lse), scale=0.1)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BOUNDS
        got = c.weights.cpu()
        same("left out", got[0, :, 32:48], lay.weights[0, :, 32:48])
        close("others", got[0, :, 48:200], w[0, :, 48:200], tol[0, :, 48:200])
        close("others", got[1, :, :100], w[1, :, :100], tol[1, :, :100])
    for n in (-1, lay.cap + 1):
        c = gpu_cache(lay)
        c.lengths[1] = n
        swa.cache_weigh(c, dev(q), dev(lse), scale=0.1)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
        close("others", c.weights.cpu()[0, :, :200], w[0, :, :200], tol[0, :, :200])


# ------------------------------------------------------------------------- evict

@pytest.mark.parametrize("lens,keep,first,recent,d,page", [
    ([300, 100, 0, 1, 129], 100, 4, 20, 64, 16),
    ([300, 100, 0, 1, 129], 99, 0, 0, 128, 7),
    ([300, 257], 256, 4, 252, 64, 64),
    ([300, 257], 1, 0, 1, 64, 64),
    ([300, 257], 1, 0, 0, 64, 0),
    ([300, 257], 0, 0, 0, 64, 64),
    ([50], 50, 2, 2, 64, 64),
    ([5000, 1024, 1025, 2048], 1024, 4, 100, 64, 64),
    ([5000, 4096, 3], 4000, 4, 100, 128, 128),
    ([70001], 30000, 10, 1000, 64, 256),
    ([70001], 69999, 10, 1000, 64, 256),
    ([3] * 40, 2, 0, 1, 64, 16),
])
def test_evict(lens, keep, first, recent, d, page):
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(61 + keep % 50, lens, 2, d, "bf16", page, evicted=True)
    want = R.evict(lay, keep, first, recent)
    c = gpu_cache(lay)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    swa.cache_evict(c, keep, first=first, recent=recent, workspace=ws, check_status=True)
    same_cache(c, want)
    # at the budget: a second call changes nothing
    swa.cache_evict(c, keep, first=first, recent=recent, check_status=True)
    same_cache(c, want)


@pytest.mark.parametrize("lens,cap", [([5000], 900000), ([20, 100, 101, 300] * 20, 50000), ([20, 100, 101, 300] * 20, 40000)])
def test_evict_with_room_for_many_keys(lens, cap):
    """The room, not the keys, says how a head is cut and whether its ranks are
    kept: few heads with much room, many heads with more than shared memory
    holds and with less."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(90, lens, 2, 64, "bf16", 64, evicted=True)
    more = -(-cap // 64) - lay.table.shape[1]
    b, h_kv = len(lens), 2
    lay.table = torch.cat([lay.table, torch.full((b, more), -1, dtype=torch.int32)], 1)
    lay.positions = torch.cat([lay.positions, torch.full((b, h_kv, more * 64), -5, dtype=torch.int32)], 2)
    lay.weights = torch.cat([lay.weights, torch.full((b, h_kv, more * 64), math.nan)], 2)
    c = gpu_cache(lay)
    swa.cache_evict(c, 100, first=4, recent=20, check_status=True)
    same_cache(c, R.evict(lay, 100, 4, 20))


@pytest.mark.parametrize("kind", ["all_equal", "special", "close", "negative"])
def test_evict_orders_of_weights(kind):
    """Ties go to the lowest slot; NaN above every number; -0 counts as 0."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(71, [700, 1500], 3, 64, "f16", 32, evicted=True)
    for i, n in enumerate([700, 1500]):
        g = torch.Generator().manual_seed(72 + i)
        if kind == "all_equal":
            w = torch.zeros(3, n)
        elif kind == "special":
            pick = torch.randint(0, 7, (3, n), generator=g)
            w = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45])[pick]
        elif kind == "close":
            w = 1 + torch.randint(0, 5, (3, n), generator=g) * 2.0 ** -23
        else:
            w = -torch.rand(3, n, generator=g)
        lay.weights[i, :, :n] = w
    for keep in (1, 333, 699):
        c = gpu_cache(lay)
        swa.cache_evict(c, keep, first=1, recent=0, check_status=True)
        same_cache(c, R.evict(lay, keep, 1, 0))


def test_evict_more_protected_than_the_budget():
    """Positions that repeat: the protected ones in the lowest slots stay."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(81, [600], 2, 64, "bf16", 64, evicted=True)
    lay.positions[0, :, :600] = 0
    c = gpu_cache(lay)
    swa.cache_evict(c, 100, first=4, recent=4, check_status=True)
    same_cache(c, R.evict(lay, 100, 4, 4))


def test_evict_reports_bad_pages_and_lengths():
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(82, [300, 300], 2, 64, "bf16", 16, evicted=True)
    c = gpu_cache(lay)
    c.lengths[0] = lay.cap + 1
    swa.cache_evict(c, 100)
    with pytest.raises(swa.SdpaError) as e:
        c.check_status()
    assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
    want = R.evict(lay, 100, 0, 0)
    for f in ("positions", "weights"):
        same(f, getattr(c, f)[0], getattr(lay, f)[0])
        same(f, getattr(c, f)[1], getattr(want, f)[1])
    assert c.lengths.tolist() == [lay.cap + 1, 100]
    for bad, entry in ((-1, 1), (lay.k.shape[0], 15), (2 ** 31 - 1, 15)):
        c = gpu_cache(lay)
        c.page_table[0, entry] = bad
        swa.cache_evict(c, 100)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BOUNDS
        for f in ("lengths", "positions", "weights"):
            same(f, getattr(c, f), getattr(want, f))
        n1 = [lay.where(1, s) for s in ([s] for s in range(100))]
        for pg, at in n1:
            same("k", c.k[pg, at], want.k[pg, at])


# ------------------------------------------------------------------------- large offsets

def test_offsets_behind_32_bits():
    """Pages that lie more than 2^32 bytes into the pool, and more than 2^31
    elements: written, read, weighed and moved there."""
    import sliding_window_attention_sdpa_gb300 as swa
    h_kv, d, page = 2, 128, 64
    n_pages = 2 ** 31 // (h_kv * d * page) + 300
    k, v = (torch.empty(n_pages, page, h_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = R.make(91, [400, 130], h_kv, d, "bf16", page, room=30, tracked=True, wild=False)
    # the small cache's pages, put at the far end of the pool
    base = n_pages - small.k.shape[0]
    k[base:], v[base:] = dev(small.k), dev(small.v)
    c = swa.KVCache(k, v, dev(small.lengths), page_table=dev(small.table + base), next_pos=dev(small.next_pos),
                    positions=dev(small.positions), weights=dev(small.weights))
    for t in (2, 40):
        q, kn, vn = inputs(92, 2, t, 4, h_kv, d, "bf16")
        o, lse = swa.cache_forward(c, dev(q), dev(kn), dev(vn), scale=0.1, check_status=True)
        ref = R.forward(small, q, kn, vn, scale=0.1)
        close("o", o, ref.o, ref.tol_o)
    q, kn, vn = inputs(93, 2, 30, 4, h_kv, d, "bf16")
    swa.cache_append(c, dev(kn), dev(vn), check_status=True)
    small = R.append(small, kn, vn)
    lse = randn(94, 2, 4, 30) + 4
    swa.cache_weigh(c, dev(q), dev(lse), scale=0.1, check_status=True)
    w, tol = R.weigh(small, q, lse, scale=0.1)
    held = ~torch.isnan(small.weights)
    close("weights", c.weights.cpu()[held], w[held], tol[held])
    small.weights = c.weights.cpu()
    swa.cache_evict(c, 128, first=4, recent=8, check_status=True)
    want = R.evict(small, 128, 4, 8)
    same("k", c.k[base:], want.k)
    same("v", c.v[base:], want.v)
    same("positions", c.positions, want.positions)


# ------------------------------------------------------------------------- together

def decode_step(swa, c, x, budget):
    o, lse = swa.cache_forward(c, x["q"], x["k"], x["v"], scale=0.125, window_left=500, tree=x["tree"], sink=x["sink"])
    swa.cache_append(c, x["k"], x["v"], index=x["index"], counts=x["counts"])
    swa.cache_weigh(c, x["q"], lse, scale=0.125, window_left=500, q_pos=x["q_pos"])
    swa.cache_evict(c, budget, first=2, recent=10)
    return o, lse


def draft(seed, lay, t, h_q, h_kv, d):
    """Drafted trees, and the accepted paths: row indexes, their number, and the
    positions of the rows (negative where a row was not accepted)."""
    b = len(lay.lengths)
    q, k, v = inputs(seed, b, t, h_q, h_kv, d, "bf16")
    tree = R.tree_masks(seed, b, t)
    index, counts = torch.zeros(b, t, dtype=torch.int32), torch.zeros(b, dtype=torch.int32)
    q_pos = torch.full((b, t), -1, dtype=torch.int32)
    for i in range(b):
        leaf = int(torch.randint(0, t, (1,), generator=torch.Generator().manual_seed(seed + i)))
        path = [u for u in range(t) if int(tree[i, leaf]) >> u & 1]
        index[i, :len(path)] = torch.tensor(path, dtype=torch.int32)
        counts[i] = len(path)
        for n, u in enumerate(path):
            q_pos[i, u] = int(lay.next_pos[i]) + n
    return dict(q=q, k=k, v=v, tree=tree, index=index, counts=counts, q_pos=q_pos, sink=randn(seed + 9, h_q))


@pytest.mark.parametrize("captured", [False, True])
def test_decoding_loop(captured):
    """Prompt, then drafting steps with eviction, eager and as one replayed
    graph, against the plain forms step by step."""
    import sliding_window_attention_sdpa_gb300 as swa
    b, t, h_q, h_kv, d, budget = 3, 6, 4, 2, 64, 60
    lay = R.make(200, [0, 0, 0], h_kv, d, "bf16", 16, room=100, tracked=True)
    off = torch.tensor([0, 70, 75, 130], dtype=torch.int32)
    kp, vp = (randn(s, 130, h_kv, d, dtype=torch.bfloat16) for s in (201, 202))
    c = gpu_cache(lay)
    swa.cache_append(c, dev(kp), dev(vp), offsets=dev(off), max_seqlen=70, check_status=True)
    lay = R.append(lay, kp, vp, offsets=off)
    same_cache(c, lay)
    graph, x = None, None
    for step in range(4):
        new = draft(300 + 20 * step, lay, t, h_q, h_kv, d)
        if x is None:
            x = {n: dev(y) for n, y in new.items()}
        else:
            for n, y in new.items():
                x[n].copy_(y)
        if captured and graph is None:
            s = torch.cuda.Stream()
            state = [y.clone() for y in (c.k, c.v, c.lengths, c.next_pos, c.positions, c.weights)]
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                decode_step(swa, c, x, budget)       # modules load before the capture
            torch.cuda.current_stream().wait_stream(s)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o, lse = decode_step(swa, c, x, budget)
            for y, z in zip((c.k, c.v, c.lengths, c.next_pos, c.positions, c.weights), state):
                y.copy_(z)
        if captured:
            graph.replay()
        else:
            o, lse = decode_step(swa, c, x, budget)
        c.check_status()
        ref = R.forward(lay, new["q"], new["k"], new["v"], scale=0.125, window=500, tree=new["tree"], sink=new["sink"])
        close("o", o, ref.o, ref.tol_o)
        close("lse", lse, ref.lse, ref.tol_lse)
        lay = R.append(lay, new["k"], new["v"], index=new["index"], counts=new["counts"])
        # the weights that the GPU holds decide the eviction; they are checked before it is repeated here
        before = lay
        w, tol = R.weigh(before, new["q"], lse.cpu(), scale=0.125, window=500, q_pos=new["q_pos"])
        lay = R.evict(before_with(before, w), budget, 2, 10)
        same("lengths", c.lengths, lay.lengths)
        same("next_pos", c.next_pos, lay.next_pos)
        for i in range(b):
            n = int(lay.lengths[i])
            for g in range(h_kv):
                # as sets: a tie of rounded weights may swap two keys
                got = c.positions[i, g, :n].cpu()
                assert sorted(got.tolist()) == sorted(lay.positions[i, g, :n].tolist()), (step, i, g)
        same("k", c.k, lay.k)
        same("positions", c.positions, lay.positions)
        held = ~torch.isnan(lay.weights)
        # off by the rounding of each step so far
        close("weights", c.weights.cpu()[held], lay.weights[held].double(), (4e-5 * (lay.weights[held].double().abs() + 1)))
        lay.weights = c.weights.cpu()


def before_with(lay, w):
    out = lay.clone()
    out.weights = w.float()
    return out


def test_other_streams_and_concurrent_calls():
    """Two caches on two streams at once, each call on torch's current stream."""
    import sliding_window_attention_sdpa_gb300 as swa
    todo = []
    for n, name in enumerate(("tree_37_gqa8", "long", "lengths_around_tiles", "tree_64")):
        lay, q, k, v, kw, dtype = forward_case(name)
        todo.append((lay, gpu_cache(lay), [dev(x) for x in (q, k, v)], kw, torch.cuda.Stream(), (q, k, v), dtype))
    torch.cuda.synchronize()
    got = [[] for _ in todo]
    for _ in range(5):
        for i, (lay, c, x, kw, s, _, _) in enumerate(todo):
            with torch.cuda.stream(s):
                got[i].append(call_forward(c, *x, kw))
    torch.cuda.synchronize()
    for i, (lay, c, x, kw, s, cpu, dtype) in enumerate(todo):
        ref = R.forward(lay, *cpu, dtype=dtype, **kw)
        for o, lse in got[i]:
            close("o", o, ref.o, ref.tol_o)
            assert torch.equal(o, got[i][0][0]) and torch.equal(lse, got[i][0][1])
        c.check_status()
