"""Cases and plain forms of the operators around attention: what goes into it, and a cache held in 4 bits.

Five operators prepare and serve what the attention of this package computes:

  rotate    each head's RMS norm of queries and keys and their position rotation (one axis, or time, height and width),
            in one pass
  rotback   its backward pass: gradients of the queries, the keys and the norms' weights
  store     keys and values are quantised as they go into the cache (4 bits, a scale for each 16 features), and the
            rows that went in are read back as the values they stand for
  read      the cached keys and values of each sequence, or those in reach of a window, come out in one run, for a
            prompt's next part
  attend    attention of a few new tokens of each sequence over its cached keys held in 4 bits and over each other:
            O and LSE

A block of 16 features is held as whole numbers c from -8 to 7 and a scale s: s is the largest magnitude / 7, rounded to
a floating-point number of 3 mantissa bits (normal from 2^-14 on, steps of 2^-17 below, 240 at most), c is x / s, rounded
(ties to even). `run` computes the operators in plain torch operations, or through the package where `own` is true.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # One user's next token: its queries and keys are normed and rotated. Only latency counts.
        dict(name="rotate-token", op="rotate", dtype="bf16", b=1, t=1, h_q=16, h_kv=16, d=64, r=64, axes=1,
             interleaved=False, norm=True, packed=False, far=16384),
        # Prompts with images and video of 16 users, packed: three axes, grouped heads.
        dict(name="rotate-prompts", op="rotate", dtype="bf16", b=16, t=4096, h_q=48, h_kv=6, d=128, r=128, axes=3,
             interleaved=False, norm=True, packed=True, far=4096),
        # A training step of the windowed layer that the benchmark's backward runs on: its gradients go on to the projections.
        dict(name="rotback-layer", op="rotback", dtype="bf16", b=2, t=8192, h_q=16, h_kv=16, d=64, r=64, axes=1,
             interleaved=False, norm=True, packed=False, far=0),
        # Packed texts of ragged lengths, adjacent pairs rotated in half of each head, far into a document.
        dict(name="rotback-packed", op="rotback", dtype="f16", b=7, t=8191, h_q=48, h_kv=6, d=128, r=64, axes=1,
             interleaved=True, norm=True, packed=True, far=1000003),
        # The accepted ones of 5 drafted tokens for 48 users.
        dict(name="store-accepted", op="store", dtype="bf16", b=48, t=5, h_kv=8, d=64, len_lo=40, len_hi=8192, page=64,
             picked=True),
        # Prompts of 16 users enter the cache at once, packed.
        dict(name="store-prompts", op="store", dtype="bf16", b=16, t=8192, h_kv=8, d=128, len_lo=0, len_hi=0, page=64,
             picked=False),
        # The keys that a windowed layer's next part of a prompt reaches back to.
        dict(name="read-window", op="read", dtype="bf16", b=4, h_kv=8, d=64, len_lo=300, len_hi=8192, page=64, window=128),
        # Whole caches for the next part of long prompts.
        dict(name="read-long", op="read", dtype="f16", b=12, h_kv=6, d=128, len_lo=16484, len_hi=16484, page=64, window=-1),
        # One user, one token, a short text: a chat's first answers. Only latency counts.
        dict(name="attend-first-tokens", op="attend", dtype="bf16", b=1, t=1, h_q=16, h_kv=16, d=64, len_lo=301,
             len_hi=301, page=64, window=-1, sink=False),
        # Full attention of a busy server: 64 users with texts from a few tokens to the longest.
        dict(name="attend-ragged", op="attend", dtype="bf16", b=64, t=1, h_q=48, h_kv=6, d=128, len_lo=5, len_hi=16484,
             page=128, window=-1, sink=True),
        # Verification of 37 drafted tokens for each of 12 users.
        dict(name="attend-tree", op="attend", dtype="bf16", b=12, t=37, h_q=48, h_kv=6, d=128, len_lo=16484, len_hi=16484,
             page=64, window=-1, sink=False),
        # One long document, four drafted tokens at a time, in a contiguous cache.
        dict(name="attend-long", op="attend", dtype="f16", b=1, t=4, h_q=32, h_kv=8, d=64, len_lo=262161, len_hi=262161,
             page=0, window=-1, sink=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotback", "store", "read", "attend", "attend"])
    top = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        d = rng.choice([64, 128])
        c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), b=_log(rng, 1, 64), d=d, h_kv=rng.choice([1, 2, 3, 4, 6, 8, 16]))
        if op in ("rotate", "rotback"):
            c["h_q"] = c["h_kv"] * rng.choice([1, 2, 4, 5, 8])
            c["t"] = _log(rng, 1, 16384)
            c["r"] = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
            c["axes"] = rng.choice([1, 1, 2, 3])
            c["interleaved"] = rng.random() < 0.5
            c["norm"] = rng.random() < 0.8
            c["packed"] = rng.random() < 0.5
            c["far"] = rng.choice([0, 0, _log(rng, 1, 2 ** 30)])
            elements = c["b"] * c["t"] * (c["h_q"] + c["h_kv"]) * d
            if _cost(c) <= top and elements <= 2 ** 29:
                return c
            continue
        c["page"] = rng.choice([0, 16, 48, 64, 128, 256])
        c["len_hi"] = _log(rng, 1, 262144)
        c["len_lo"] = rng.choice([0, c["len_hi"], rng.randint(0, c["len_hi"])])
        if op == "attend":
            c["h_q"] = c["h_kv"] * rng.choice([1, 2, 4, 5, 8, 16])
            c["t"] = rng.choice([1, _log(rng, 1, 64)])
            c["window"] = rng.choice([-1, -1, _log(rng, 1, 8192)])
            c["sink"] = rng.random() < 0.3
        if op == "read":
            c["window"] = rng.choice([-1, _log(rng, 1, 8192)])
        if op == "store":
            c["picked"] = rng.random() < 0.5
            c["t"] = _log(rng, 1, 64) if c["picked"] else _log(rng, 1, 8192)
        pool = c["b"] * (c["len_hi"] + c.get("t", 0)) * c["h_kv"] * d
        scores = c["b"] * c.get("h_q", 0) * c.get("t", 0) * c["len_hi"]
        if _cost(c) <= top and pool <= 2 ** 29 and scores <= 2 ** 28 * 1.5:
            return c


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def _lengths(case):
    """Cached keys of each sequence: spread over the logarithm from len_lo to len_hi, in an order of no kind."""
    b, lo, hi = case["b"], case["len_lo"], case["len_hi"]
    if b == 1:
        return [hi]
    got = [int(round(math.exp(math.log(lo + 1) + (math.log(hi + 1) - math.log(lo + 1)) * i / (b - 1)))) - 1 for i in range(b)]
    np.random.RandomState(7).shuffle(got)
    return got


def _counts(case):
    """Rows of each sequence that a call takes: 1 to t, the last of them t."""
    got = np.random.RandomState(11).randint(1, case["t"] + 1, case["b"]).tolist()
    return got[:-1] + [case["t"]]


def work(case):
    """Each input that counts read once, each output written once; a cached row is d / 2 bytes and d / 16 of scales."""
    d, h_kv, op = case["d"], case["h_kv"], case["op"]
    row = d // 2 + d // 16
    if op in ("rotate", "rotback"):
        tokens, heads = sum(_counts(case)), case["h_q"] + h_kv
        passes = 2 if op == "rotate" or not case["norm"] else 3
        return {"bytes": float(tokens * (heads * d * 2 * passes + 4 * case["axes"])), "flops": float(tokens * heads * d * 4 * passes)}
    if op == "store":
        rows = sum(_counts(case)) * h_kv
        # the rows in, in 4 bits into the cache, out of it, and out in the type they came in
        return {"bytes": float(rows * 2 * (4 * d + 2 * row)), "flops": 0.0}
    lens = _lengths(case)
    if op == "read":
        rows = sum(n if case["window"] < 0 else min(n, case["window"]) for n in lens) * h_kv
        return {"bytes": float(rows * 2 * (row + 2 * d)), "flops": 0.0}
    b, t, h_q = case["b"], case["t"], case["h_q"]
    reach = [n if case["window"] < 0 else min(n, case["window"] + t - 1) for n in lens]
    q = b * t * h_q * d * 2
    return {"bytes": float(sum(reach) * h_kv * 2 * row + b * t * h_kv * 4 * d + 2 * q + b * h_q * t * 4),
            "flops": float(sum(reach) * t * h_q * 4 * d + b * t * t * h_q * 4 * d)}


# ----------------------------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1013 + 5)
    return _prepare_rotate(case, g) if case["op"] in ("rotate", "rotback") else _prepare_cache(case, g, seed)


def _normal(g, dt, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dt)


def _prepare_rotate(case, g):
    dev, dt = torch.device("cuda"), DTYPES[case["dtype"]]
    b, t, d, r, axes = case["b"], case["t"], case["d"], case["r"], case["axes"]
    counts = _counts(case)
    lens = torch.tensor(counts, dtype=torch.int32, device=dev)
    # each token's place in its text; images and video after a first stretch, in frames of 8 x 12
    place = torch.arange(t, device=dev, dtype=torch.int32).expand(b, t)
    pos = [place, place // 96, (place // 12) % 8][:axes] if axes > 1 else [place]
    if axes == 3:
        pos = [place // 96, (place // 12) % 8 + place // 96, place % 12 + place // 96]
    start = torch.randint(0, case["far"] + 1, (b, 1), generator=g, device=dev, dtype=torch.int32)
    pos = torch.stack([p + start for p in pos])
    # features of unlike sizes, as projections give them
    size = lambda: (0.4 * _normal(g, torch.float32, d)).exp().to(dt)  # noqa: E731
    here = (torch.arange(t, device=dev) < lens[:, None]).view(-1)
    tensors = {}
    for name, heads in (("q", case["h_q"]), ("k", case["h_kv"])):
        tensors[name] = _normal(g, dt, b, t, heads, d) * size()
        if case["op"] == "rotback":
            tensors["d" + name] = _normal(g, dt, b, t, heads, d) * 0.02
    if case["packed"]:
        tensors = {n: x.flatten(0, 1)[here] for n, x in tensors.items()}
        pos = pos.flatten(1)[:, here]
    else:
        # rows of padding: a gradient of zero, and values of no meaning
        for n, x in tensors.items():
            if n.startswith("d"):
                x.view(b * t, -1)[~here] = 0
    s = dict(case=case, pos=pos[0].contiguous() if axes == 1 else pos.contiguous(), **tensors)
    s["lens"] = None if case["packed"] else lens
    s["freq"] = (10000.0 ** (-torch.arange(r // 2, dtype=torch.float64) * 2 / r)).float().to(dev)
    s["axis"] = None if axes == 1 else (torch.arange(r // 2, device=dev) * axes // (r // 2)).to(torch.int32)
    s["eps"] = 1e-6
    for n in ("q", "k"):
        s[n + "_weight"] = (1 + 0.2 * _normal(g, torch.float32, d)).to(dt) if case["norm"] else None
    return s


def _prepare_cache(case, g, seed):
    dev, dt = torch.device("cuda"), DTYPES[case["dtype"]]
    b, h_kv, d, op = case["b"], case["h_kv"], case["d"], case["op"]
    t = case.get("t", 0)
    lens = _lengths(case)
    room = max(1, max(lens) + (t if op == "store" else 0))
    page = case["page"] or -(-room // 16) * 16
    table_w = -(-room // page)
    n_pages = b * table_w
    # keys have a few features that are larger than the others, whatever the token; values do not
    wide = (0.5 * _normal(g, torch.float32, h_kv, d)).exp().to(dt)
    keys = lambda *shape: _normal(g, dt, *shape, h_kv, d) * wide  # noqa: E731
    values = lambda *shape: _normal(g, dt, *shape, h_kv, d)  # noqa: E731
    s = dict(case=case, page=page)
    s["table"] = (torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).view(b, table_w) if case["page"]
                  else torch.arange(b, device=dev, dtype=torch.int32).view(b, 1))
    s["lengths0"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["lengths"] = s["lengths0"].clone()
    s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    total = sum(lens)
    old = (keys(total), values(total)) if total else None
    if own:
        import sliding_window_attention_sdpa_gb300 as swa
        s["cache"] = swa.KVCache.empty(b, h_kv, d, room, dtype=dt, device=dev, page_size=page, bits=4)
        s["cache"].page_table.copy_(s["table"])
        if total:
            swa.cache_append(s["cache"], *old, offsets=s["offsets"], max_seqlen=max(lens))
        s["lengths"] = s["cache"].lengths
    else:
        s["pools"] = [(torch.zeros(n_pages, page, h_kv, d, dtype=torch.int8, device=dev),
                       torch.zeros(n_pages, page, h_kv, d // 16, dtype=torch.float32, device=dev)) for _ in range(2)]
        if total:
            seq = torch.repeat_interleave(torch.arange(b, device=dev), s["lengths0"].long())
            slots = torch.arange(total, device=dev) - s["offsets"].long()[seq]
            _put(s, seq, slots, old)
    if op == "store":
        cnt = _counts(case)
        s["counts"] = torch.tensor(cnt, dtype=torch.int32, device=dev)
        s["new_offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32, device=dev)
        s["longest"], s["total"] = max(cnt), sum(cnt)
        rows = (b, t) if case["picked"] else (sum(cnt),)
        s["k_new"], s["v_new"] = keys(*rows), values(*rows)
        if case["picked"]:
            s["index"] = torch.rand(b, t, generator=g, device=dev).argsort(1).to(torch.int32).contiguous()
    if op == "read":
        cnt = [n if case["window"] < 0 else min(n, case["window"]) for n in lens]
        s["start"] = torch.tensor([n - c for n, c in zip(lens, cnt)], dtype=torch.int32, device=dev)
        s["new_offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32, device=dev)
        s["total"] = sum(cnt)
    if op == "attend":
        s["q"] = _normal(g, dt, b, t, case["h_q"], d)
        s["k_new"], s["v_new"] = keys(b, t), values(b, t)
        s["scale"] = d ** -0.5
        s["sink"] = _normal(g, torch.float32, case["h_q"]) if case["sink"] else None
        # a tree: each node hangs from one of the few nodes before it
        masks, rs = [], np.random.RandomState(int(seed) % 2 ** 31)
        for _ in range(b):
            m = []
            for i in range(t):
                m.append((1 << i) | (m[max(0, i - 1 - int(rs.randint(0, 4)))] if i else 0))
            masks.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in m])
        s["tree"] = torch.tensor(masks, dtype=torch.int64, device=dev)
    return s


# ---------------------------------------------------------------------------------------------------- the operators

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rotate": _own_rotate, "rotback": _own_rotback, "store": _own_store, "read": _own_read,
                "attend": _own_attend}[op](s)
    return {"rotate": _rotate, "rotback": _rotback, "store": _store, "read": _read, "attend": _attend}[op](s)


def _own_rotate(s):
    import sliding_window_attention_sdpa_gb300 as swa
    return swa.qk_rotate(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                         axis=s["axis"], interleaved=s["case"]["interleaved"], seq_lens=s["lens"])


def _own_rotback(s):
    import sliding_window_attention_sdpa_gb300 as swa
    out = swa.qk_rotate_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freq"], q_weight=s["q_weight"],
                                 k_weight=s["k_weight"], eps=s["eps"], axis=s["axis"],
                                 interleaved=s["case"]["interleaved"], seq_lens=s["lens"])
    return out if s["case"]["norm"] else out[:2]


def _own_store(s):
    import sliding_window_attention_sdpa_gb300 as swa
    s["lengths"].copy_(s["lengths0"])  # each pass starts from the same cache
    if s["case"]["picked"]:
        swa.cache_append(s["cache"], s["k_new"], s["v_new"], index=s["index"], counts=s["counts"])
        k, v = swa.cache_read(s["cache"], start=s["lengths0"], counts=s["counts"], max_rows=s["case"]["t"])
    else:
        swa.cache_append(s["cache"], s["k_new"], s["v_new"], offsets=s["new_offsets"], max_seqlen=s["longest"])
        k, v = swa.cache_read(s["cache"], start=s["lengths0"], offsets=s["new_offsets"], total=s["total"])
    return k, v, s["lengths"]


def _own_read(s):
    import sliding_window_attention_sdpa_gb300 as swa
    return swa.cache_read(s["cache"], start=s["start"], offsets=s["new_offsets"], total=s["total"])


def _own_attend(s):
    import sliding_window_attention_sdpa_gb300 as swa
    return swa.cache_forward(s["cache"], s["q"], s["k_new"], s["v_new"], scale=s["scale"], window_left=s["case"]["window"],
                             tree=s["tree"], sink=s["sink"])


# -- rotation

def _turns(s):
    """Cosine and sine of each token and pair, and which tokens are there: angles in 64 bits, far positions turn often."""
    pos = s["pos"] if s["axis"] is None else s["pos"][s["axis"].long()].movedim(0, -1)
    angle = (pos.double()[..., None] if s["axis"] is None else pos.double()) * s["freq"].double()
    here = None
    if s["lens"] is not None:
        here = torch.arange(angle.shape[1], device=angle.device) < s["lens"][:, None]
    return angle.cos().float()[..., None, :], angle.sin().float()[..., None, :], here


def _halves(x, case):
    r = case["r"]
    return (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])


def _joined(lo, hi, rest, case):
    pairs = torch.stack([lo, hi], -1).flatten(-2) if case["interleaved"] else torch.cat([lo, hi], -1)
    return torch.cat([pairs, rest], -1)


def _turned(x, cos, sin, case):
    lo, hi = _halves(x, case)
    return _joined(lo * cos - hi * sin, hi * cos + lo * sin, x[..., case["r"]:], case)


def _rotate(s):
    case = s["case"]
    cos, sin, here = _turns(s)
    out = []
    for n in ("q", "k"):
        x = s[n].float()
        if case["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s[n + "_weight"].float()
        y = _turned(x, cos, sin, case)
        if here is not None:
            y = y.masked_fill(~here[..., None, None], 0.0)
        out.append(y.to(s[n].dtype))
    return tuple(out)


def _rotback(s):
    case = s["case"]
    cos, sin, here = _turns(s)
    grads, weights = [], []
    for n in ("q", "k"):
        dy = _turned(s["d" + n].float(), cos, -sin, case)
        if here is not None:
            dy = dy.masked_fill(~here[..., None, None], 0.0)
        if case["norm"]:
            x = s[n].float()
            if here is not None:
                x = x.masked_fill(~here[..., None, None], 0.0)
            r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
            x = x * r
            weights.append((dy * x).flatten(0, -2).sum(0))
            dy = dy * s[n + "_weight"].float()
            dy = (dy - x * (dy * x).mean(-1, keepdim=True)) * r
        grads.append(dy.to(s[n].dtype))
    return tuple(grads + weights)


# -- the cache in 4 bits

def _quantised(x):
    """Whole numbers and scales of rows [.., d]."""
    x = x.float().unflatten(-1, (-1, 16))
    a = x.abs().amax(-1, keepdim=True)
    a = a / torch.full_like(a, 7.0)  # (a plain 7 would be a product with 1 / 7, which is not exact at a border)
    # the power of two in front of a, from its exponent's bits: powers and logarithms need not be exact
    step = (a.clamp(min=2.0 ** -14).view(torch.int32) & 0x7f800000).view(torch.float32) / 8
    scale = ((a / step).round() * step).clamp(max=240.0)
    c = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0).round().clamp(-8, 7)
    return c.flatten(-2).to(torch.int8), scale[..., 0]


def _places(s, seq, slots):
    return s["table"].long()[seq, slots // s["page"]], slots % s["page"]


def _put(s, seq, slots, rows):
    pg, at = _places(s, seq, slots)
    for (codes, scales), x in zip(s["pools"], rows):
        codes[pg, at], scales[pg, at] = _quantised(x)


def _get(s, seq, slots):
    pg, at = _places(s, seq, slots)
    return [(codes[pg, at].float().unflatten(-1, (-1, 16)) * scales[pg, at][..., None]).flatten(-2) for codes, scales in s["pools"]]


def _store(s):
    case = s["case"]
    dt, dev = s["k_new"].dtype, s["k_new"].device
    s["lengths"].copy_(s["lengths0"])
    fresh = torch.arange(case["t"], device=dev, dtype=torch.int32) < s["counts"][:, None]
    seq, i = fresh.nonzero(as_tuple=True)
    rows = (s["k_new"], s["v_new"])
    if case["picked"]:
        rows = tuple(x[seq, s["index"].long()[seq, i]] for x in rows)
    slots = s["lengths"].long()[seq] + i
    _put(s, seq, slots, rows)
    s["lengths"] += s["counts"]
    out = [x.to(dt) for x in _get(s, seq, slots)]
    if case["picked"]:
        full = [torch.zeros_like(s["k_new"]) for _ in out]
        for f, x in zip(full, out):
            f[seq, i] = x
        out = full
    return out[0], out[1], s["lengths"]


def _read(s):
    dt, dev = DTYPES[s["case"]["dtype"]], s["table"].device
    n = (s["new_offsets"][1:] - s["new_offsets"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(n), device=dev), n, output_size=s["total"])
    slots = torch.arange(s["total"], device=dev) - s["new_offsets"].long()[seq] + s["start"].long()[seq]
    return tuple(x.to(dt) for x in _get(s, seq, slots))


def _attend(s):
    case, q = s["case"], s["q"]
    b, t, h_q, d = q.shape
    h_kv, w, dev = case["h_kv"], case["window"], q.device
    # the latest n slots of each sequence hold every key that a row can see
    n = min(max(1, case["len_hi"] if w < 0 else min(case["len_hi"], w)), s["table"].shape[1] * s["page"])
    slots = (s["lengths"].long() - n).clamp(min=0)[:, None] + torch.arange(n, device=dev)
    k, v = _get(s, torch.arange(b, device=dev)[:, None].expand(b, n), slots)
    k, v = torch.cat([k, s["k_new"].float()], 1), torch.cat([v, s["v_new"].float()], 1)
    bit = (s["tree"][:, :, None] >> torch.arange(t, device=dev)) & 1
    depth = bit.sum(-1) - 1
    see = (slots < s["lengths"][:, None])[:, None].expand(b, t, n)
    see_new = bit == 1
    if w >= 0:
        see = see & ((s["lengths"][:, None] + depth)[:, :, None] - slots[:, None] <= w)
        see_new = see_new & (depth[:, :, None] - depth[:, None] <= w)
    see = torch.cat([see, see_new], 2)
    score = torch.einsum("btkgd,bnkd->bkgtn", q.float().view(b, t, h_kv, h_q // h_kv, d), k) * s["scale"]
    score = score.masked_fill(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, h_kv, h_q // h_kv, 1, 1)
        top = torch.maximum(top, sink)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + (sink - top).exp()
    o = torch.einsum("bkgtn,bnkd->btkgd", p / total, v).reshape(b, t, h_q, d).to(q.dtype)
    return o, (top + total.log()).view(b, h_q, t)


# ------------------------------------------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    # (the inputs as a plain program holds them: nothing below calls the package)
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1013 + 5)
    if case["op"] in ("rotate", "rotback"):
        return _exact_rotate(_prepare_rotate(case, g))
    global own
    was, own = own, False
    try:
        s = _prepare_cache(case, g, seed)
    finally:
        own = was
    return {"store": _exact_store, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _exact_rotate(s):
    """A pair of features is a complex number, its rotation a product with exp(i angle)."""
    case = s["case"]
    b, t, d, r = case["b"], case["t"], case["d"], case["r"]
    i = torch.arange(r // 2, device=s["q"].device)
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
    pos = s["pos"] if s["pos"].dim() > 1 + (not case["packed"]) else s["pos"][None]
    axis = torch.zeros_like(i) if s["axis"] is None else s["axis"].long()
    spin = torch.polar(torch.ones((), dtype=torch.float64, device=i.device),
                       torch.stack([pos[a].double() for a in axis.tolist()], -1) * s["freq"].double())
    if case["op"] == "rotback":
        spin = spin.conj()
    outs, weights = [], []
    for n in ("q", "k"):
        out = torch.zeros(s[n].shape, dtype=torch.float64, device=i.device)
        w = torch.ones(d, dtype=torch.float64, device=i.device) if s[n + "_weight"] is None else s[n + "_weight"].double()
        dw = torch.zeros_like(w)
        # head by head: 64 bits of one head at a time
        for h in range(s[n].shape[-2]):
            x = s[n][..., h, :].double()
            inv = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / d + s["eps"]) if case["norm"] else torch.ones_like(x[..., :1])
            y = s["d" + n][..., h, :].double() if case["op"] == "rotback" else x * inv * w
            z = torch.complex(y[..., lo], y[..., hi]) * spin
            y[..., lo], y[..., hi] = z.real, z.imag
            if not case["packed"]:
                y[torch.arange(t, device=i.device) >= s["lens"][:, None]] = 0
            if case["op"] == "rotback":
                dw += (y * x * inv).reshape(-1, d).sum(0)
                if case["norm"]:
                    y = y * w
                    y = inv * y - x * inv ** 3 * ((x * y).sum(-1, keepdim=True) / d)
            out[..., h, :] = y
        outs.append(out)
        weights.append(dw)
    return tuple(outs + (weights if case["op"] == "rotback" and case["norm"] else []))


def _exact_held(x):
    """The values that rows stand for once they are held: the border cases by comparison of whole multiples."""
    x = x.double().unflatten(-1, (-1, 16))
    a = x.abs().amax(-1, keepdim=True)
    # all scales there are, and seven times the borders between them; on a border the even one counts
    table = [m / 2 ** 17 for m in range(8)] + [(8 + m) / 2 ** 17 * 2 ** e for e in range(22) for m in range(8)]
    table = torch.tensor([z for z in table if z <= 240], dtype=torch.float64, device=x.device)
    borders = 7 * (table[1:] + table[:-1]) / 2
    at, behind = torch.searchsorted(borders, a), torch.searchsorted(borders, a, right=True)
    scale = table[torch.where(at % 2 == 0, at, behind)]
    # x lies at c if it is behind the border below c and not behind the one above it
    c = torch.zeros_like(x)
    for k in range(1, 9):
        border = (k - 0.5) * scale
        over = (x.abs() > border) | ((x.abs() == border) & (k % 2 == 0))
        c += (over & (scale > 0)).double()
    c = torch.where(x < 0, -c.clamp(max=8), c.clamp(max=7))
    return (c * scale).flatten(-2)


def _exact_store(s):
    case = s["case"]
    out, start = [torch.zeros_like(s["k_new"], dtype=torch.float64) for _ in range(2)], 0
    for i, n in enumerate(_counts(case)):
        for o, x in zip(out, (s["k_new"], s["v_new"])):
            if case["picked"]:
                o[i, :n] = _exact_held(x[i, s["index"][i, :n].long()])
            else:
                o[start:start + n] = _exact_held(x[start:start + n])
        start += n
    lengths = torch.tensor([n + c for n, c in zip(_lengths(case), _counts(case))], dtype=torch.int32, device=out[0].device)
    return out[0], out[1], lengths


def _held_rows(s, i, lo, hi):
    """Sequence i's cached rows lo to hi in 64 bits."""
    pages = s["table"][i].long()
    first, last = lo // s["page"], -(-hi // s["page"])
    at = slice(lo - first * s["page"], hi - first * s["page"])
    return [(codes[pages[first:last]].flatten(0, 1)[at].double().unflatten(-1, (-1, 16)) *
             scales[pages[first:last]].flatten(0, 1)[at].double()[..., None]).flatten(-2) for codes, scales in s["pools"]]


def _exact_read(s):
    lens, start = _lengths(s["case"]), s["start"].tolist()
    rows = [_held_rows(s, i, start[i], n) for i, n in enumerate(lens)]
    return tuple(torch.cat([r[j] for r in rows]) for j in range(2))


def _exact_attend(s):
    case = s["case"]
    q = s["q"].double()
    b, t, h_q, d = q.shape
    group, w, dev = h_q // case["h_kv"], case["window"], q.device
    o = torch.zeros(b, t, h_q, d, dtype=torch.float64, device=dev)
    lse = torch.full((b, h_q, t), -math.inf, dtype=torch.float64, device=dev)
    lines = [[x % 2 ** 64 for x in row] for row in s["tree"].tolist()]
    for i, n in enumerate(_lengths(case)):
        lo = max(0, n - w) if w >= 0 else 0
        deep = [bin(x).count("1") - 1 for x in lines[i]]
        see = np.zeros((t, n - lo + t), dtype=bool)
        for r in range(t):
            see[r, max(0, n + deep[r] - w - lo) if w >= 0 else 0:n - lo] = True
            for u in range(t):
                see[r, n - lo + u] = bool(lines[i][r] >> u & 1) and (w < 0 or deep[r] - deep[u] <= w)
        see = torch.from_numpy(see).to(dev)
        held = _held_rows(s, i, lo, n)
        for kv in range(case["h_kv"]):
            k, v = (torch.cat([x[:, kv], y[i, :, kv].double()]) for x, y in zip(held, (s["k_new"], s["v_new"])))
            heads = slice(kv * group, (kv + 1) * group)
            a = torch.einsum("tgd,nd->gtn", q[i, :, heads], k) * s["scale"]
            a = a.masked_fill(~see, -math.inf)
            z = torch.logsumexp(a, -1)
            if s["sink"] is not None:
                z = torch.logaddexp(z, s["sink"][heads].double()[:, None])
            o[i, :, heads] = torch.einsum("gtn,nd->tgd", torch.exp(a - z[..., None]), v)
            lse[i, heads] = z
    return o, lse
