"""Edges of the key/value cache's calls on the GPU: masks that list padding
tokens, keys that only the shallowest rows could see, light keys in f16, NaN
queries and infinite sinks, the precision that each forward kernel promises,
and every form in which the forward's work is cut and joined."""
import math

import numpy as np
import pytest
import torch

import cache_ref as R
from test_gpu_cache import close, dev, gpu_cache, inputs, randn

pytestmark = pytest.mark.gpu

F64 = torch.float64


def admitted(lay, i, g, t, tree, window):
    """Which cached keys [t, n] and new tokens [t, t] each row admits, by the
    header's words: a token's position counts all bits of its mask; a mask
    without its own bit admits nothing, but others may list its token."""
    n = int(lay.lengths[i])
    line = R.chain(t) if tree is None else [int(x) % 2 ** 64 & ((1 << t) - 1) for x in tree[i].tolist()]
    deep = torch.tensor([bin(x).count("1") - 1 for x in line])
    real = torch.tensor([x >> r & 1 for r, x in enumerate(line)], dtype=torch.bool)
    bit = torch.tensor([[x >> u & 1 for u in range(t)] for x in line], dtype=torch.bool)
    old = real[:, None].expand(t, n)
    new = bit & real[:, None]
    if window >= 0:
        pos = torch.from_numpy(lay.pos(i, g, n))
        old = old & (lay.next(i) + deep[:, None] - pos <= window)
        new = new & (deep[:, None] - deep <= window)
    return old, new


def form(lay, q, k, v, *, scale, window=-1, tree=None, sink=None, dtype="bf16", split=False):
    """O, LSE and their bounds in 64 bits, a (sequence, kv-head) at a time.
    `split`: P enters the product as a 16-bit value and its 16-bit remainder."""
    b, t, h_q, d = q.shape
    h_kv, u = k.shape[2], R.U[dtype]
    grp = h_q // h_kv
    o, tol_o = torch.zeros(b, t, h_q, d, dtype=F64), torch.zeros(b, t, h_q, d, dtype=F64)
    lse, tol_l = torch.full((b, h_q, t), -math.inf, dtype=F64), torch.zeros(b, h_q, t, dtype=F64)
    for i in range(b):
        n = int(lay.lengths[i])
        for g in range(h_kv):
            old, new = admitted(lay, i, g, t, tree, window)
            see = torch.cat([old, new], 1)
            ks, vs = lay.rows(i, g, n)
            kk, vv = torch.cat([ks, k[i, :, g]]).to(F64), torch.cat([vs, v[i, :, g]]).to(F64)
            none = ~see.any(0)
            kk[none], vv[none] = 0.0, 0.0
            for h in range(g * grp, (g + 1) * grp):
                qq = q[i, :, h].to(F64)
                s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
                z = torch.logsumexp(s, 1)
                if sink is not None:
                    z = torch.logaddexp(z, sink[h].to(F64))
                rows = see.any(1)
                p = torch.exp(s - z[:, None])
                p[~rows] = 0
                m = see.sum(1).to(F64) + 8
                mag = torch.where(see, (qq.abs() @ kk.abs().T) * scale, 0.0).amax(1)
                top = torch.where(see, s.abs(), 0.0).amax(1)
                # as in cache_ref.forward: scores off by es, exponentials within 2^-21, sums of m terms within m steps
                es = mag * (d + 8) * 2.0 ** -23 + top * 2.0 ** -22
                rel = (2 * es + 2.0 ** -20 + m * 2.0 ** -23)[:, None]
                o[i, :, h], lse[i, h] = p @ vv, z
                zf = torch.where(torch.isfinite(z), z.abs(), 0.0)
                tol_l[i, h] = es + 2.0 ** -20 + m * 2.0 ** -23 + zf * 2.0 ** -22
                # P in 16 bits (and its remainder: u of u); f16's smallest P is 2^-24 of which half is lost, next to a
                # largest P of 2^7 at least
                up = u * u if split else u
                small = 2.0 ** -32 * (m * p.amax(1))[:, None] * vv.abs().max() if dtype == "f16" and len(vv) else 0.0
                tol_o[i, :, h] = u * o[i, :, h].abs() + (up + rel) * (1 + u) * (p @ vv.abs()) + small + 2.0 ** -24
    return R.Forward(o, lse, tol_o, tol_l)


def few(t, h_q, h_kv, d):
    """Whether the kernel for few rows per kv-head takes the call (it splits P)."""
    return t * (h_q // h_kv) <= (8 if d == 128 else 16)


def call(c, q, k, v, **kw):
    import sliding_window_attention_sdpa_gb300 as swa
    kw = {n: dev(x) if torch.is_tensor(x) else x for n, x in kw.items()}
    return swa.cache_forward(c, dev(q), dev(k), dev(v), check_status=True, **kw)


# ------------------------------------------------------------------------- masks

def listed_padding(seed, b, t, share):
    """Trees of which some tokens' masks lack their own bit: those rows are
    empty, while the rows behind them list them as before."""
    tree = R.tree_masks(seed, b, t)
    rs = np.random.RandomState(seed + 1)
    for i in range(b):
        for r in range(t - 1):
            if rs.rand() < share:
                tree[i, r] = int(tree[i, r]) & ~(1 << r)
    return tree


@pytest.mark.parametrize("window", [-1, 2, 0, 40])
@pytest.mark.parametrize("t,d,h_q", [(7, 64, 2), (4, 128, 4), (11, 128, 8), (40, 64, 4), (63, 128, 4)])
def test_padding_tokens_that_others_list(t, d, h_q, window):
    """A mask without its own bit makes an empty row, and its token keeps the
    position that its bits say: others that list it admit it by that."""
    lens, h_kv = [90, 10, 0], 2
    lay = R.make(401, lens, h_kv, d, "bf16", 16)
    q, k, v = inputs(402, len(lens), t, h_q, h_kv, d, "bf16")
    tree = listed_padding(403, len(lens), t, 0.4)
    # the smallest such case in sequence 0: token 1 descends from 0 but is empty, token 2 lists both
    tree[0, 0], tree[0, 1], tree[0, 2] = 1, 1, 7
    kw = dict(scale=d ** -0.5, window=window, tree=tree)
    o, lse = call(gpu_cache(lay), q, k, v, scale=kw["scale"], window_left=window, tree=tree)
    ref = form(lay, q, k, v, split=few(t, h_q, h_kv, d), **kw)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("t,d,h_q", [(7, 64, 2), (4, 128, 4), (8, 64, 4), (30, 128, 4), (64, 64, 4)])
def test_tokens_out_of_every_window_hold_anything(t, d, h_q, wide):
    """Tokens that rows list but no row's window has, on a chain whose first
    ones are empty rows: NaN in them reaches no output."""
    lens, h_kv, gone = [90, 10, 0], 2, t // 2
    b, window = len(lens), gone - 1 if wide else 0
    lay = R.make(411, lens, h_kv, d, "bf16", 16)
    q, k, v = inputs(412, b, t, h_q, h_kv, d, "bf16")
    line = R.chain(t)
    for r in range(gone):
        line[r] &= ~(1 << r)
    tree = torch.tensor([[x - 2 ** 64 if x >= 2 ** 63 else x for x in line]] * b, dtype=torch.int64)
    new = admitted(lay, 0, 0, t, tree, window)[1]
    out = torch.nonzero(~new.any(0)).flatten().tolist()
    assert out
    k[:, out], v[:, out] = math.nan, math.inf
    o, lse = call(gpu_cache(lay), q, k, v, scale=d ** -0.5, window_left=window, tree=tree)
    ref = form(lay, q, k, v, split=few(t, h_q, h_kv, d), scale=d ** -0.5, window=window, tree=tree)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("page", [0, 7, 16, 64])
@pytest.mark.parametrize("t,d,h_q", [(5, 64, 2), (3, 128, 4), (21, 128, 4), (40, 64, 4)])
def test_in_front_of_the_shallowest_window(t, d, h_q, page):
    """Rows whose shallowest is not at the next position (the tokens before it
    are padding): keys that only the padding's windows would have hold anything,
    and their pages may be gone."""
    lens, h_kv, window, gone = [301, 100, 76, 1000], 2, 77, t // 2
    b = len(lens)
    lay = R.make(421, lens, h_kv, d, "bf16", page)
    q, k, v = inputs(422, b, t, h_q, h_kv, d, "bf16")
    line = R.chain(t)
    for r in range(gone):
        line[r] = 0
    tree = torch.tensor([[x - 2 ** 64 if x >= 2 ** 63 else x for x in line]] * b, dtype=torch.int64)
    for i, n in enumerate(lens):
        first = max(0, min(n, n + gone - window))
        pg, at = lay.where(i, np.arange(first))
        lay.k[pg, at], lay.v[pg, at] = math.nan, math.nan
        if page:
            lay.table[i, :first // page] = -1
    o, lse = call(gpu_cache(lay), q, k, v, scale=d ** -0.5, window_left=window, tree=tree)
    ref = form(lay, q, k, v, split=few(t, h_q, h_kv, d), scale=d ** -0.5, window=window, tree=tree)
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


# ------------------------------------------------------------------------- values

def ladder(lay, i, powers, values):
    """Keys of sequence i whose scores, with q = (1, 0, ..) and scale 1, are
    log(2) times `powers` (rounded to the type), and V of `values` in every
    feature."""
    n = len(powers)
    dt = lay.k.dtype
    pg, at = lay.where(i, np.arange(n))
    x = (torch.tensor(powers, dtype=F64) * math.log(2)).to(dt)
    lay.k[pg, at], lay.v[pg, at] = 0, torch.tensor(values, dtype=dt)[:, None, None]
    lay.k[pg, at, :, 0] = x[:, None]


@pytest.mark.parametrize("heavy", ["first", "last", "amid"])
@pytest.mark.parametrize("light", [-15.0, -24.3, -26.1, -29.6])
@pytest.mark.parametrize("t,d,n", [(1, 64, 2000), (1, 128, 300), (1, 128, 5000), (20, 128, 300), (20, 64, 5000)])
def test_light_keys_in_f16(t, d, n, light, heavy):
    """One heavy key whose V is 0 next to many light ones whose V is 1: O is the
    light ones' mass, far below f16's smallest number relative to the heavy P."""
    lay = R.make(431, [n], 1, d, "f16", 16)
    q, k, v = inputs(432, 1, t, 1, 1, d, "f16")
    q[:], k[:], v[:] = 0, 0, 0
    q[..., 0] = 1
    k[..., 0] = light * math.log(2)
    powers, values = [light] * n, [1.0] * n
    at = dict(first=0, last=n - 1, amid=n // 2 + 5)[heavy]
    powers[at], values[at] = 0.0, 0.0
    ladder(lay, 0, powers, values)
    o, lse = call(gpu_cache(lay), q, k, v, scale=1.0)
    ref = form(lay, q, k, v, scale=1.0, dtype="f16", split=few(t, 1, 1, d))
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("t,d,lens", [(2, 64, [90, 0, 300]), (2, 128, [90, 0, 5000]), (9, 128, [90, 0, 300]),
                                      (40, 64, [90, 0, 5000]), (40, 128, [90, 3, 700])])
def test_nan_queries_are_seen(t, d, lens, sink):
    """A row whose q holds a NaN has NaN for every score: O and LSE are NaN,
    those of the other rows what they are; a padding row is still empty."""
    h_q, h_kv, b = 4, 2, len(lens)
    lay = R.make(441, lens, h_kv, d, "bf16", 16)
    q, k, v = inputs(442, b, t, h_q, h_kv, d, "bf16")
    tree = R.tree_masks(443, b, t)
    tree[0, 1] = 0                                     # an empty row, NaN or not
    s = randn(444, h_q) if sink else None
    ref = form(lay, q, k, v, scale=d ** -0.5, tree=tree, sink=s, split=few(t, h_q, h_kv, d))
    bad = torch.zeros(b, t, h_q, dtype=torch.bool)
    bad[0, 0, 1] = bad[1, t - 1, 3] = bad[2, 0, 0] = bad[2, t // 2, 2] = True
    q[bad, d - 1] = math.nan
    q[0, 1, 2] = math.nan
    o, lse = call(gpu_cache(lay), q, k, v, scale=d ** -0.5, tree=tree, sink=s)
    o, lse = o.cpu(), lse.cpu()
    assert torch.isnan(o[bad]).all() and torch.isnan(lse.transpose(1, 2)[bad]).all()
    close("lse", lse.transpose(1, 2)[~bad], ref.lse.transpose(1, 2)[~bad], ref.tol_lse.transpose(1, 2)[~bad])
    close("o", o[~bad], ref.o[~bad], ref.tol_o[~bad])


@pytest.mark.parametrize("t,d,n", [(1, 64, 90), (2, 128, 3000), (40, 64, 90), (40, 128, 3000), (1, 64, 0)])
def test_infinite_sinks(t, d, n):
    """exp(-inf) = 0: no sink; a sink of +inf takes all of the weight."""
    h_q, h_kv = 4, 2
    lay = R.make(451, [n, 30], h_kv, d, "bf16", 16)
    q, k, v = inputs(452, 2, t, h_q, h_kv, d, "bf16")
    sink = torch.tensor([math.inf, -math.inf, 0.3, math.inf])
    o, lse = call(gpu_cache(lay), q, k, v, scale=d ** -0.5, sink=sink)
    ref = form(lay, q, k, v, scale=d ** -0.5, sink=sink, split=few(t, h_q, h_kv, d))
    assert torch.isinf(ref.lse[:, [0, 3]]).all() and (ref.o[:, :, [0, 3]] == 0).all()
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


def rms_ratio(got, exact, dtype):
    """Root mean square error relative to that of rounding the exact O."""
    rms = lambda x: float(x.double().square().mean().sqrt())  # noqa: E731
    return rms(got.cpu().double() - exact) / rms(exact.to(R.DT[dtype]).double() - exact)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t,d,h_q", [(2, 64, 8), (4, 64, 8), (2, 128, 8), (4, 128, 8), (37, 128, 16)])
def test_precision_of_each_kernel(t, d, h_q, dtype):
    """With V of zero mean both O and the sum of P's rounding errors are random
    walks over p v: P in 16 bits adds an error of the size of O's own rounding,
    1.41 times it together; with P's remainder O's own rounding is all (the next
    term is u of it). The bounds are apart from both by a few per cent of 10^4
    samples and more."""
    b, h_kv, n = 2, 2, 900
    split = few(t, h_q, h_kv, d)
    lay = R.make(461, [n] * b, h_kv, d, dtype, 64)
    q, k, v = inputs(462, b, t, h_q, h_kv, d, dtype)
    o, lse = call(gpu_cache(lay), q, k, v, scale=d ** -0.5)
    exact = form(lay, q, k, v, scale=d ** -0.5, dtype=dtype, split=split).o
    assert rms_ratio(o, exact, dtype) < (1.01 if split else 1.5)
    # and that a lost remainder would show: the same sums with P rounded once
    i, g = 0, 0
    ks, vs = lay.rows(i, g, n)
    qq = q[i, :, :h_q // h_kv].transpose(0, 1).reshape(-1, d).double()
    s = qq @ ks.double().T * d ** -0.5
    p = torch.exp(s - s.amax(1, keepdim=True))
    whole, once = (x @ vs.double() / p.sum(1, keepdim=True) for x in (p, p.to(R.DT[dtype]).double()))
    assert rms_ratio(once.to(R.DT[dtype]), whole, dtype) > 1.2


# ------------------------------------------------------------------------- work cut between parts

# lens, t, h_q, h_kv, d, dtype: more units (sequence, kv-head, block of 256 or 8 rows) than parts (152, few rows 304)
# and room for more than 512 keys, so that cut units are named by their part
PARTS = {
    "blocks_of_two_and_one": ([(37 * i) % 90 for i in range(42)] + [1500, 700], 37, 16, 2, 128, "bf16"),
    "blocks_of_two_and_one_d64": ([(37 * i) % 90 for i in range(42)] + [1500, 700], 37, 16, 2, 64, "f16"),
    "two_blocks_of_two": ([(53 * i) % 70 for i in range(40)] + [900, 1300], 64, 16, 2, 128, "f16"),
    "two_blocks_of_two_d64": ([(53 * i) % 70 for i in range(40)] + [900, 1300], 64, 16, 2, 64, "bf16"),
    "one_block_of_two": ([(37 * i) % 90 for i in range(60)] + [1500], 32, 24, 3, 64, "bf16"),
    "one_block_of_one": ([(37 * i) % 90 for i in range(90)] + [1500, 40, 2000], 5, 16, 2, 128, "bf16"),
    "three_blocks": ([(37 * i) % 90 for i in range(30)] + [1500], 60, 18, 2, 64, "bf16"),
    "few_rows": ([(37 * i) % 90 for i in range(170)] + [900, 5, 2500], 1, 8, 2, 128, "bf16"),
    "few_rows_d64": ([(37 * i) % 90 for i in range(110)] + [900, 5, 2500], 2, 24, 3, 64, "f16"),
    # and by unit: several kv-heads, mixed blocks, fewer units than parts
    "by_unit_mixed": ([1500, 3, 700, 4000], 37, 16, 2, 128, "bf16"),
    "by_unit_three_blocks": ([1500, 3, 700], 60, 18, 2, 64, "f16"),
}


@pytest.mark.parametrize("name", PARTS)
def test_units_cut_between_parts(name):
    lens, t, h_q, h_kv, d, dtype = PARTS[name]
    seed, b, rows = 500 + 7 * list(PARTS).index(name), len(lens), t * (h_q // h_kv)
    units = b * h_kv * -(-rows // (256 if not few(t, h_q, h_kv, d) else rows))
    assert name.startswith("by_unit") == (units <= (304 if few(t, h_q, h_kv, d) else 152))
    lay = R.make(seed, lens, h_kv, d, dtype, 64)
    q, k, v = inputs(seed + 1, b, t, h_q, h_kv, d, dtype)
    tree = R.tree_masks(seed + 2, b, t)
    o, lse = call(gpu_cache(lay), q, k, v, scale=d ** -0.5, tree=tree)
    ref = form(lay, q, k, v, scale=d ** -0.5, tree=tree, dtype=dtype, split=few(t, h_q, h_kv, d))
    close("lse", lse, ref.lse, ref.tol_lse)
    close("o", o, ref.o, ref.tol_o)


# ------------------------------------------------------------------------- lengths

@pytest.mark.parametrize("d,window", [(64, -1), (128, 100)])
def test_more_than_64_tokens_in_several_calls(d, window):
    """A call refuses them and says how: in calls of up to 64, appended in between."""
    import sliding_window_attention_sdpa_gb300 as swa
    t, h_q, h_kv, lens = 150, 8, 2, [90, 0]
    lay = R.make(481, lens, h_kv, d, "bf16", 16, room=t)
    q, k, v = inputs(482, 2, t, h_q, h_kv, d, "bf16")
    c = gpu_cache(lay)
    with pytest.raises(swa.SdpaError, match="appended in between"):
        call(c, q, k, v, scale=d ** -0.5, window_left=window)
    for a in range(0, t, 64):
        x = [y[:, a:a + 64].contiguous() for y in (q, k, v)]
        o, lse = call(c, *x, scale=d ** -0.5, window_left=window)
        swa.cache_append(c, dev(x[1]), dev(x[2]), check_status=True)
        ref = form(lay, *x, scale=d ** -0.5, window=window)
        close("lse", lse, ref.lse, ref.tol_lse)
        close("o", o, ref.o, ref.tol_o)
        lay = R.append(lay, x[1], x[2])


@pytest.mark.parametrize("keep", [64, 65, 2 ** 31 - 1])
def test_evict_looks_at_lengths_whatever_the_budget(keep):
    """A budget of all of the room moves nothing; lengths out of range are
    reported all the same."""
    import sliding_window_attention_sdpa_gb300 as swa
    lay = R.make(471, [64, 30], 2, 64, "bf16", 16, evicted=True)
    c = gpu_cache(lay)
    swa.cache_evict(c, keep, check_status=True)
    assert c.lengths.tolist() == [64, 30]
    for wrong in (-1, 65, 2 ** 31 - 1):
        c.lengths[1] = wrong
        swa.cache_evict(c, keep)
        with pytest.raises(swa.SdpaError) as e:
            c.check_status()
        assert e.value.code == swa.SDPA_ERR_BAD_LENGTHS
        assert c.lengths.tolist() == [64, wrong]
