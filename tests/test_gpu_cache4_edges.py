"""The cache in 4 bits where its kernels could go wrong: every kernel and block
form, bad pages and lengths, keys that do not count and may hold anything, extreme
values, strides, far offsets, streams, waits that run out, and a decoding loop
(rotation, append, forward, read) eager and captured."""
import math

import numpy as np
import pytest
import torch

import cache4_ref as Q
import cache_ref as R
import test_gpu_cache as T
from test_gpu_cache4 import layout, read_all

pytestmark = pytest.mark.gpu

dev, randn, close, same = T.dev, T.randn, T.close, T.same


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# lens, t, h_q, h_kv, d, dtype, page, window, extras: rows per kv-head are t * h_q / h_kv
FORMS = {
    "rows_9": ([300, 40], 9, 2, 2, 128, "bf16", 64, -1, dict(tree=True)),
    "rows_17": ([300, 40], 17, 2, 2, 128, "f16", 16, -1, dict(tree=True)),
    "rows_32_long": ([5000, 17, 0], 4, 16, 2, 128, "bf16", 64, -1, dict(sink=True)),
    "rows_33": ([1300, 17, 0], 11, 6, 2, 128, "bf16", 48, -1, {}),
    "d64_rows_33": ([1300, 17, 0], 11, 6, 2, 64, "f16", 48, 200, {}),
    "d64_rows_80": ([2300, 300], 10, 8, 1, 64, "bf16", 64, -1, dict(tree=True)),
    "d64_rows_81": ([2300, 300], 27, 3, 1, 64, "bf16", 64, -1, dict(tree=True)),
    "tile_window": ([2300, 300, 5], 40, 3, 1, 128, "f16", 32, 700, dict(tree=True, sink=True)),
    "tile_positions": ([700, 300, 5], 40, 3, 1, 64, "bf16", 32, 150, dict(tree=True, evicted=True)),
    "tile_positions_d128": ([700, 300, 5], 40, 3, 1, 128, "f16", 16, 150, dict(evicted=True)),
    "tile_300_rows": ([900, 64, 65, 63], 50, 6, 1, 128, "bf16", 0, -1, dict(tree=True)),
    "tile_q_lens": ([900, 64, 0, 300], 50, 4, 2, 64, "f16", 64, -1, dict(q_lens=[50, 0, 1, 33])),
    "tile_padding": ([90, 10, 300], 45, 3, 1, 128, "bf16", 16, 30, dict(tree=True, empty=0.4)),
    "rows_positions": ([1700, 300, 5], 3, 4, 2, 128, "bf16", 32, 150, dict(tree=True, evicted=True)),
    "one_long": ([40000], 1, 4, 2, 64, "f16", 128, -1, {}),
    "rows_positions_cut": ([3700, 300, 5], 3, 4, 2, 128, "bf16", 32, 150, dict(tree=True, evicted=True)),
    "rows_ragged_cut": ([4000, 0, 90, 2500], 4, 8, 2, 128, "f16", 64, -1, dict(q_lens=[4, 0, 1, 3], sink=True)),
    "d64_rows_window_cut": ([9000, 300], 2, 8, 2, 64, "bf16", 16, 5000, {}),
    "d64_rows_padding_cut": ([6000, 17], 4, 8, 2, 64, "f16", 48, -1, dict(tree=True, empty=0.4)),
    "d64_rows_64": ([2300, 300], 8, 8, 1, 64, "f16", 64, -1, dict(tree=True)),
    "d64_rows_65": ([2300, 300], 13, 5, 1, 64, "bf16", 16, 90, dict(tree=True)),
    "d64_tiles_both": ([3900, 0, 130, 64], 37, 16, 2, 64, "bf16", 64, -1, dict(tree=True)),
    "d64_tiles_both_f16": ([6000, 500], 33, 8, 1, 64, "f16", 16, 4000, dict(sink=True)),
    "d64_tiles_three": ([2500, 1, 300], 60, 10, 1, 64, "bf16", 32, -1, dict(q_lens=[60, 3, 0])),
    "d64_tiles_many": ([1500, 70, 0, 900, 2500, 64, 65], 40, 14, 2, 64, "f16", 48, -1, {}),
    # units of one step and of many in one part; more sequences than a CTA has threads
    "short_cut_rows": ([3, 60, 64, 65, 1, 0, 7, 130, 20, 5] * 6 + [2300], 1, 8, 2, 128, "bf16", 64, -1, {}),
    "short_cut_blocks": ([3, 60, 64, 65, 1, 0, 7, 130, 20, 5] * 6 + [2300], 3, 8, 1, 64, "f16", 16, -1, dict(tree=True)),
    "short_cut_tiles": ([3, 60, 1, 0, 130, 5, 64, 65] * 5 + [1300], 37, 8, 1, 64, "bf16", 16, -1, dict(tree=True)),
    "short_cut_tiles_d128": ([3, 60, 1, 0, 130, 5, 64, 65] * 5 + [1300], 37, 8, 1, 128, "f16", 64, -1, {}),
    "b_200_cut": ([(37 * i) % 40 for i in range(200)] + [2300], 1, 2, 1, 64, "bf16", 64, -1, {}),
    "b_520_tiles_cut": ([(37 * i) % 40 for i in range(520)] + [1100], 9, 8, 1, 64, "bf16", 64, -1, {}),
}


def case(name):
    lens, t, h_q, h_kv, d, dtype, page, window, x = FORMS[name]
    seed = 3000 + 13 * list(FORMS).index(name)
    lay = layout(seed, lens, h_kv, d, dtype, page, evicted=x.get("evicted", False))
    q_lens = x.get("q_lens")
    q, k, v = T.inputs(seed + 1, len(lens), t, h_q, h_kv, d, dtype, q_lens)
    tree = R.tree_masks(seed, len(lens), t, x.get("empty", 0.0)) if x.get("tree") else None
    return lay, q, k, v, dict(scale=d ** -0.5, window=window, tree=tree, q_lens=q_lens,
                              sink=randn(seed + 4, h_q) if x.get("sink") else None), dtype


@pytest.mark.parametrize("name", FORMS)
def test_forward_forms(name):
    lay, q, k, v, kw, dtype = case(name)
    o, lse = T.call_forward(Q.gpu_cache(lay), dev(q), dev(k), dev(v), kw, check_status=True)
    ref = Q.forward(Q.held_layout(lay), q, k, v, dtype=dtype, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("t,d,page", [(1, 64, 16), (1, 128, 64), (5, 128, 16), (40, 128, 64), (50, 64, 16)])
def test_forward_reports_bad_pages_and_lengths(t, d, page):
    import sliding_window_attention_sdpa_gb300 as swa
    lay = layout(19, [200, 100, 64], 2, d, "bf16", page)
    q, k, v = T.inputs(20, 3, t, 4, 2, d, "bf16")
    kw = dict(scale=0.125, window=-1, tree=None, q_lens=None, sink=None)
    held = Q.held_layout(lay)
    last = 199 // page
    for bad in (-1, lay.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        c = Q.gpu_cache(lay)
        c.page_table[0, last] = bad
        o, lse = T.call_forward(c, dev(q), dev(k), dev(v), kw)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BOUNDS
        c.check_status()                   # cleared
        cut = held.clone()
        cut.lengths[0] = last * page
        cut.next_pos = lay.lengths.clone()  # positions stay those of 200 keys
        cut.positions = torch.arange(cut.cap, dtype=torch.int32).expand(3, 2, -1)
        ref = Q.forward(cut, q, k, v, dtype="bf16", **kw)
        close("lse", lse, ref.lse, ref.tol_lse)
        close("o", o, ref.o, ref.tol_o)
    full = layout(21, [200 // page * page + page, 100, 64], 2, d, "bf16", page)
    ref = Q.forward(Q.held_layout(full), q, k, v, dtype="bf16", **kw)
    for n in (-1, full.cap + 1, 2 ** 31 - 1, -2 ** 31):
        c = Q.gpu_cache(full)
        c.lengths[0] = n
        o, lse = T.call_forward(c, dev(q), dev(k), dev(v), kw)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
        close("lse", lse[1:], ref.lse[1:], ref.tol_lse[1:])
        close("o", o[1:], ref.o[1:], ref.tol_o[1:])


@pytest.mark.parametrize("t", [1, 64])
def test_no_sequences_and_no_room(t):
    import sliding_window_attention_sdpa_gb300 as swa
    kw = dict(dtype=torch.bfloat16, device="cuda", bits=4)
    c = swa.KVCache.empty(0, 2, 64, 100, **kw)
    z = torch.zeros(0, t, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = swa.cache_forward(c, z, z, z, scale=1.0, check_status=True)
    assert o.shape == z.shape and lse.shape == (0, 2, t)
    swa.cache_append(c, z, z, check_status=True)
    assert swa.cache_read(c, check_status=True)[0].shape[0] == 0
    with pytest.raises(swa.SdpaError, match="total"):
        swa.cache_read(c, offsets=i32([0]), total=3)
    # room for no key: the new tokens attend over each other alone
    c = swa.KVCache.empty(3, 2, 64, 0, **kw)
    lay = layout(7, [0, 0, 0], 2, 64, "bf16", 16)
    q, k, v = T.inputs(8, 3, t, 4, 2, 64, "bf16")
    o, lse = swa.cache_forward(c, dev(q), dev(k), dev(v), scale=0.125, check_status=True)
    ref = Q.forward(lay, q, k, v, scale=0.125, dtype="bf16")
    close("o", o, ref.o, ref.tol_o)
    close("lse", lse, ref.lse, ref.tol_lse)
    assert swa.cache_read(c, check_status=True)[0].shape == (3, 0, 2, 64)
    swa.cache_append(c, dev(k), dev(v))
    with pytest.raises(swa.SdpaError):
        c.check_status()


@pytest.mark.parametrize("t,d", [(1, 64), (2, 128), (40, 128), (60, 64)])
def test_keys_and_tokens_that_do_not_count_may_hold_anything(t, d):
    """Keys in front of every row's window are held as NaN; new tokens that no row admits are NaN, infinite, huge."""
    import sliding_window_attention_sdpa_gb300 as swa
    lens, h_q, h_kv, w = [500, 130, 64], 4, 2, 100
    lay = layout(61, lens, h_kv, d, "bf16", 16)
    q, k, v = T.inputs(62, 3, t, h_q, h_kv, d, "bf16")
    tree = torch.tensor([[(1 << (r + 1)) - 1 for r in range(t)]] * 3, dtype=torch.uint64).view(torch.int64)
    if t > 2:
        # token 1 is listed by nobody (and itself an empty row)
        tree = tree & ~torch.tensor(2, dtype=torch.int64)
        tree[:, 1] = 0
        k[0, 1], v[0, 1] = math.nan, math.nan
        k[1, 1], v[1, 1] = math.inf, -math.inf
        k[2, 1], v[2, 1] = 3e38, -3e38
    kw = dict(scale=0.125, window=w, tree=tree, q_lens=None, sink=None)
    ref = Q.forward(Q.held_layout(lay), q, k, v, dtype="bf16", **kw)
    bad = lay.clone()
    for i, n in enumerate(lens):
        gone = np.arange(max(0, n - w))               # the shallowest row is at position n: it sees the last w keys
        pg, at = bad.where(i, gone)
        bad.k[pg, at], bad.v[pg, at] = math.nan, math.inf
    o, lse = T.call_forward(Q.gpu_cache(bad), dev(q), dev(k), dev(v), kw, check_status=True)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("t,d,dtype", [(1, 64, "bf16"), (3, 128, "bf16"), (40, 128, "bf16"), (60, 64, "bf16"), (2, 128, "f16"), (40, 64, "f16")])
def test_extreme_values(t, d, dtype):
    """Rows of q far beyond f16 and far below it (bf16), of unlike sizes, zero; NaN rows; keys and values from the
    smallest scales to the largest."""
    import sliding_window_attention_sdpa_gb300 as swa
    h_q, h_kv, lens = 4, 2, [300, 70]
    lay = layout(71, lens, h_kv, d, dtype, 16)
    g = torch.Generator().manual_seed(5)
    for i, n in enumerate(lens):
        pg, at = lay.where(i, np.arange(n))
        lay.v[pg, at] = (lay.v[pg, at].float() * 2.0 ** torch.randint(-10, 9, (n, 1, 1), generator=g).float()).to(R.DT[dtype])
        lay.k[pg, at] = (lay.k[pg, at].float() * 2.0 ** torch.randint(-8, 3, (n, 1, 1), generator=g).float()).to(R.DT[dtype])
    q, k, v = T.inputs(72, 2, t, h_q, h_kv, d, dtype)
    scale = 2.0 ** -3
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 2.0 ** -14
    if dtype == "bf16":
        q[0, 0, 2] *= 2.0 ** -60
        q[1, 0, 0] *= 2.0 ** -30
        q[1, 0, 2, ::3] *= 2.0 ** -20
        q[1, 0, 3] = 2.0 ** -126
    c = Q.gpu_cache(lay)
    kw = dict(scale=scale, window=-1, tree=None, q_lens=None, sink=None)
    o, lse = T.call_forward(c, dev(q), dev(k), dev(v), kw, check_status=True)
    ref = Q.forward(Q.held_layout(lay), q, k, v, dtype=dtype, **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)
    # beyond f16 and beyond what exponents hold: one key has all of the weight
    if dtype == "bf16":
        x = q.clone()
        x[0, 0, 0] = 2.0 ** 20 * randn(9, d).to(torch.bfloat16)
        o, lse = T.call_forward(c, dev(x), dev(k), dev(v), kw, check_status=True)
        held = Q.held_layout(lay)
        kk = torch.cat([held.rows(0, 0, lens[0])[0], k[0, :1, 0]]).double()
        vv = torch.cat([held.rows(0, 0, lens[0])[1], v[0, :1, 0]]).double()
        s = kk @ x[0, 0, 0].double() * scale
        best = int(s.argmax())
        assert abs(float(lse[0, 0, 0]) - float(s[best])) <= 2.0 ** -16 * float(s[best])
        assert ((o[0, 0, 0].double().cpu() - vv[best]).abs() <= R.U["bf16"] * vv[best].abs() + 2.0 ** -24).all()
    x = q.clone()
    x[1, t - 1, 1, 5] = math.nan
    o, lse = T.call_forward(c, dev(x), dev(k), dev(v), kw, check_status=True)
    assert torch.isnan(o[1, t - 1, 1]).all() and torch.isnan(lse[1, 1, t - 1])
    ok = torch.ones(2, t, h_q, dtype=torch.bool)
    ok[1, t - 1, 1] = False
    assert torch.isfinite(o.cpu()[ok]).all()


@pytest.mark.parametrize("t,h_q,d,dtype,most", [(1, 8, 128, "bf16", 1.1), (1, 16, 64, "f16", 1.1), (2, 8, 128, "f16", 1.1), (40, 8, 128, "bf16", 1.1),
                                                (40, 8, 128, "f16", 1.5)])
def test_precision(t, h_q, d, dtype, most):
    """O's error against 64 bits, relative to that of rounding the exact O: P is f16, with its remainder for f16 output
    in the rows kernel; without it (tiles), P's rounding adds as much as O's at most: sqrt(2) of it, 1.5 with a margin for the sample."""
    lay = layout(81, [700], 1, d, dtype, 64)
    q, k, v = T.inputs(82, 1, t, h_q, 1, d, dtype)
    kw = dict(scale=d ** -0.5, window=-1, tree=None, q_lens=None, sink=None)
    o, _ = T.call_forward(Q.gpu_cache(lay), dev(q), dev(k), dev(v), kw, check_status=True)
    ref = R.forward(Q.held_layout(lay), q, k, v, dtype=dtype, **kw).o
    rounded = ref.to(R.DT[dtype]).double()
    assert (o.double().cpu() - ref).norm() <= most * (rounded - ref).norm()


@pytest.mark.parametrize("t,d", [(1, 64), (9, 128), (40, 64)])
def test_strides(t, d):
    """K and V of the cache in one allocation, new tokens cut from one projection, O into a wider tensor."""
    import sliding_window_attention_sdpa_gb300 as swa
    h_q, h_kv, lens = 6, 2, [90, 300, 0]
    lay = layout(11, lens, h_kv, d, "bf16", 32)
    n_pages = lay.k.shape[0]
    pool = torch.full((h_kv, n_pages, 2, 2, 9 * d), 0xff, dtype=torch.uint8, device="cuda")   # heads, pages, K or V, groups
    pools = [pool[:, :, x].transpose(0, 1) for x in range(2)]
    c = swa.KVCache(*pools, torch.zeros_like(lay.lengths).cuda(), page_table=dev(lay.table), dtype=torch.bfloat16)
    rows = [torch.cat([x[lay.where(i, np.arange(n))] for i, n in enumerate(lens)]) for x in (lay.k, lay.v)]
    wide = [torch.full((len(r), h_kv + 3, d), 9.0, dtype=torch.bfloat16, device="cuda") for r in rows]
    for w, r in zip(wide, rows):
        w[:, 1:3] = r.cuda()
    swa.cache_append(c, wide[0][:, 1:3], wide[1][:, 1:3], offsets=i32(np.concatenate([[0], np.cumsum(lens)])), max_seqlen=300, check_status=True)
    plain = Q.gpu_cache(lay)
    for got, want in zip(read_all(c, lens), read_all(plain, lens)):
        assert torch.equal(got, want)
    qkv = randn(12, 3, t, (h_q + 2 * h_kv) * d + 8, dtype=torch.bfloat16).cuda()
    q, k, v = (x.unflatten(2, (-1, d)) for x in qkv[..., :(h_q + 2 * h_kv) * d].split([h_q * d, h_kv * d, h_kv * d], 2))
    out = torch.full((3, t, h_q + 1, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = swa.cache_forward(c, q, k, v, scale=0.1, out=out[:, :, 1:, :d], check_status=True)
    o2, lse2 = swa.cache_forward(plain, q.contiguous(), k.contiguous(), v.contiguous(), scale=0.1)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert (out[:, :, 0] == 7).all() and (out[..., d:] == 7).all()


def test_offsets_behind_32_bits():
    """Pages more than 4 GB into the pool, output rows more than 2^31 elements into a tensor."""
    import sliding_window_attention_sdpa_gb300 as swa
    d, h_kv, page = 128, 2, 16
    n_pages = (1 << 32) // (h_kv * 9 * d) + 100
    pools = [torch.empty(n_pages, h_kv, 1, 9 * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    far = [n_pages - 1, n_pages - 40, 3, n_pages - 2]
    c = swa.KVCache(*pools, torch.zeros(1, dtype=torch.int32, device="cuda"), page_table=i32([far]), dtype=torch.float16)
    k, v = randn(1, 1, 60, h_kv, d, dtype=torch.float16), randn(2, 1, 60, h_kv, d, dtype=torch.float16)
    swa.cache_append(c, dev(k), dev(v), check_status=True)
    near = swa.KVCache.empty(1, h_kv, d, 64, dtype=torch.float16, device="cuda", page_size=16, bits=4)
    swa.cache_append(near, dev(k), dev(v), check_status=True)
    out = [torch.empty(1, 60, 1 << 18, d, dtype=torch.float16, device="cuda")[:, :, -h_kv:] for _ in range(2)]
    got = swa.cache_read(c, max_rows=60, out=out, check_status=True)
    same("k", got[0], Q.held(k))
    same("v", got[1], Q.held(v))
    for t in (1, 40):
        q, kn, vn = (dev(randn(3 + i, 1, t, h, d, dtype=torch.float16)) for i, h in enumerate((4, h_kv, h_kv)))
        a, b = (swa.cache_forward(x, q, kn, vn, scale=0.1, check_status=True) for x in (c, near))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_and_graphs_with_a_workspace_each():
    import sliding_window_attention_sdpa_gb300 as swa
    lay = layout(91, [3000, 700], 2, 128, "bf16", 64)
    c = Q.gpu_cache(lay)
    calls = []
    for i, t in enumerate((1, 40, 3)):
        q, k, v = (dev(x) for x in T.inputs(92 + i, 2, t, 8, 2, 128, "bf16"))
        calls.append((q, k, v, swa.cache_forward(c, q, k, v, scale=0.1, check_status=True)))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = []
        for s, (q, k, v, _) in zip(streams, calls):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(swa.cache_forward(c, q, k, v, scale=0.1))
        torch.cuda.synchronize()
        for (a, b), (_, _, _, want) in zip(got, calls):
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    graphs, held = [], []
    for q, k, v, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(swa.cache_forward(c, q, k, v, scale=0.1))
        graphs.append(g)
    for s, g in zip(streams, graphs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for (a, b), (_, _, _, want) in zip(held, calls):
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


WAITS = {"few": ([30000, 10], 1, 8, 2, 128, "bf16", 64), "few_small_pages": ([60000, 10], 1, 8, 2, 64, "f16", 16),
         "few_uncut": ([900, 500], 1, 8, 2, 128, "f16", 16), "sixteen": ([30000, 10], 2, 8, 1, 128, "f16", 64),
         "tile": ([60000, 40], 5, 8, 1, 128, "bf16", 64), "tile_d64": ([30000, 40], 50, 8, 2, 64, "f16", 64),
         "tile_two": ([60000, 40], 32, 8, 1, 128, "bf16", 16), "tile_uncut": ([300, 200], 37, 16, 2, 64, "bf16", 64)}


@pytest.mark.parametrize("name", WAITS)
def test_waits_run_out(name):
    import sliding_window_attention_sdpa_gb300 as swa
    from test_gpu_cache_waits import runs_out
    lens, t, h_q, h_kv, d, dtype, page = WAITS[name]
    c = swa.KVCache.empty(2, h_kv, d, max(lens), dtype=R.DT[dtype], device="cuda", page_size=page, bits=4)
    rows = [randn(5 + i, sum(lens), h_kv, d, dtype=R.DT[dtype]).cuda() for i in range(2)]
    swa.cache_append(c, *rows, offsets=i32(np.concatenate([[0], np.cumsum(lens)])), max_seqlen=max(lens), check_status=True)
    x = [dev(y) for y in T.inputs(612, 2, t, h_q, h_kv, d, dtype)]
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")
    want = swa.cache_forward(c, *x, scale=0.1, workspace=ws, check_status=True)
    runs_out(c, lambda: swa.cache_forward(c, *x, scale=0.1, workspace=ws))
    got = swa.cache_forward(c, *x, scale=0.1, workspace=ws, check_status=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def serving_step(swa, c, x):
    """One step of a model with norms, rotation and a cache in 4 bits; all in place or into given tensors."""
    swa.qk_rotate(x["q0"], x["k0"], x["pos"], x["freq"], q_weight=x["wq"], k_weight=x["wk"], out=(x["q"], x["k"]))
    swa.cache_forward(c, x["q"], x["k"], x["v"], scale=0.125, window_left=300, tree=x["tree"], out=x["o"], lse=x["lse"], workspace=x["ws"])
    swa.cache_append(c, x["k"], x["v"], index=x["index"], counts=x["counts"])
    swa.cache_read(c, start=x["start"], counts=x["take"], max_rows=8, out=(x["kr"], x["vr"]))


@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(captured):
    import sliding_window_attention_sdpa_gb300 as swa
    import rope_ref as P
    b, t, h_q, h_kv, d, dt = 3, 5, 8, 2, 64, torch.bfloat16
    lens = [40, 333, 0]
    lay = layout(41, lens, h_kv, d, "bf16", 16, room=60)
    c = Q.gpu_cache(lay)
    ref = Q.held_layout(lay)
    new = lambda *s, dtype=dt: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    x = dict(q0=new(b, t, h_q, d), k0=new(b, t, h_kv, d), v=new(b, t, h_kv, d), q=new(b, t, h_q, d), k=new(b, t, h_kv, d),
             o=new(b, t, h_q, d), lse=new(b, h_q, t, dtype=torch.float32), pos=new(b, t, dtype=torch.int32),
             freq=(10000.0 ** (-torch.arange(32) / 32)).cuda(), wq=(1 + 0.1 * randn(1, d)).to(dt).cuda(), wk=(1 + 0.1 * randn(2, d)).to(dt).cuda(),
             tree=new(b, t, dtype=torch.int64), index=new(b, t, dtype=torch.int32), counts=new(b, dtype=torch.int32),
             start=new(b, dtype=torch.int32), take=new(b, dtype=torch.int32), kr=new(b, 8, h_kv, d), vr=new(b, 8, h_kv, d),
             ws=new(1 << 24, dtype=torch.uint8))
    graph = None
    for step in range(6):
        rs = np.random.RandomState(step)
        f = dict(q0=randn(100 + step, b, t, h_q, d, dtype=dt), k0=randn(200 + step, b, t, h_kv, d, dtype=dt), v=randn(300 + step, b, t, h_kv, d, dtype=dt),
                 tree=R.tree_masks(400 + step, b, t))
        deep = torch.tensor([[bin(m % 2 ** 64).count("1") - 1 for m in row] for row in f["tree"].tolist()])
        f["pos"] = (ref.lengths[:, None] + deep).to(torch.int32)
        f["index"] = torch.from_numpy(np.stack([rs.permutation(t) for _ in range(b)]).astype(np.int32))
        f["counts"] = torch.from_numpy(rs.randint(0, t + 1, b).astype(np.int32))
        # the last 8 keys after the step, as far as there are any
        after = ref.lengths + f["counts"]
        f["start"] = (after - 8).clamp(min=0).to(torch.int32)
        f["take"] = (after - f["start"]).to(torch.int32)
        for n, y in f.items():
            x[n].copy_(y)
        if captured and graph is None:
            # (modules load before the capture, on a copy of the state)
            keep = [z.clone() for z in (c.k, c.v, c.lengths)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                serving_step(swa, c, x)
            torch.cuda.current_stream().wait_stream(side)
            for z, y in zip((c.k, c.v, c.lengths), keep):
                z.copy_(y)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                serving_step(swa, c, x)
            for z, y in zip((c.k, c.v, c.lengths), keep):
                z.copy_(y)
        if captured:
            graph.replay()
        else:
            serving_step(swa, c, x)
        c.check_status()
        for n, w in (("q", x["wq"]), ("k", x["wk"])):
            close(n, x[n], *P.forward(f[n + "0"], w.cpu(), f["pos"], x["freq"].cpu()))
        want = Q.forward(ref, x["q"].cpu(), x["k"].cpu(), f["v"], scale=0.125, window=300, tree=f["tree"], dtype="bf16")
        close("o", x["o"], want.o, want.tol_o)
        close("lse", x["lse"], want.lse, want.tol_lse)
        ref = R.append(ref, Q.held(x["k"].cpu()), Q.held(f["v"]), index=f["index"], counts=f["counts"])
        same("lengths", c.lengths, ref.lengths)
        for i in range(b):
            n0, n = int(f["start"][i]), int(f["take"][i])
            pg, at = ref.where(i, np.arange(n0, n0 + n))
            same("kr", x["kr"][i, :n], ref.k[pg, at])
            same("vr", x["vr"][i, :n], ref.v[pg, at])
            assert (x["kr"][i, n:] == 0).all()
