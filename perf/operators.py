"""Cases and plain forms of the operators on a key/value cache.

Four operators serve a model trained with the sliding-window attention of this package:

  forward   attention of a few new tokens of each sequence (one token, a chain, or a tree of drafted tokens)
            over its cached keys and over each other: O and LSE
  append    the keys and values of accepted tokens (or of whole prompts) go behind each sequence's cached ones
  weigh     each cached key's attention weight, summed over given query rows and the heads of its group, is added
            to the key's account
  evict     each sequence that holds more keys than a budget keeps the first, the latest and the heaviest ones;
            keys kept behind the budget move into the places that became free

`run` computes them in plain torch operations, or through the package where `own` is true. Sequences live in pages
([n_pages, page_size, h_kv, d]) named by a table; `page` 0 stands for one contiguous run of slots per sequence.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # One user, one token, a short text: a chat's first answers. Only latency counts.
        dict(name="forward-first-tokens", op="forward", dtype="bf16", b=1, t=1, h_q=16, h_kv=16, d=64, len_lo=301,
             len_hi=301, page=64, window=-1, sink=False),
        # A windowed layer with sinks of a model served to 16 users: the key range is the window, whatever the length.
        dict(name="forward-window-sink", op="forward", dtype="bf16", b=16, t=1, h_q=64, h_kv=8, d=64, len_lo=700,
             len_hi=8192, page=64, window=128, sink=True),
        # Full attention of a busy server: 64 users with texts from a few tokens to the longest.
        dict(name="forward-ragged", op="forward", dtype="f16", b=64, t=1, h_q=48, h_kv=6, d=128, len_lo=5,
             len_hi=16484, page=128, window=-1, sink=False),
        # Verification of 37 drafted tokens for each of 12 users.
        dict(name="forward-tree", op="forward", dtype="bf16", b=12, t=37, h_q=48, h_kv=6, d=128, len_lo=16484,
             len_hi=16484, page=64, window=-1, sink=False),
        # One long document, four drafted tokens at a time, in a contiguous cache.
        dict(name="forward-long", op="forward", dtype="bf16", b=1, t=4, h_q=16, h_kv=2, d=128, len_lo=262161,
             len_hi=262161, page=0, window=-1, sink=False),
        # The accepted ones of 5 drafted tokens for 48 users.
        dict(name="append-accepted", op="append", dtype="bf16", b=48, t=5, h_kv=8, d=64, len_lo=40, len_hi=8192,
             page=64, picked=True),
        # Prompts of 16 users enter the cache at once, packed.
        dict(name="append-prompts", op="append", dtype="bf16", b=16, t=8192, h_kv=8, d=128, len_lo=0, len_hi=0,
             page=64, picked=False),
        # One decoded token of 16 users weighs its keys.
        dict(name="weigh-token", op="weigh", dtype="bf16", b=16, t=1, h_q=64, h_kv=8, d=64, len_lo=1000, len_hi=8192,
             page=64, window=-1),
        # The last 32 rows of a prompt say which of its keys matter.
        dict(name="weigh-prompt-end", op="weigh", dtype="bf16", b=12, t=32, h_q=48, h_kv=6, d=128, len_lo=16484,
             len_hi=16484, page=64, window=-1),
        # A short cache goes back to its budget after some tokens.
        dict(name="evict-step", op="evict", dtype="bf16", b=2, h_kv=8, d=64, len_lo=1100, len_hi=1100, page=64,
             keep=1024, first=4, recent=128),
        # After the prompt, half of each cache goes.
        dict(name="evict-half", op="evict", dtype="bf16", b=12, h_kv=6, d=128, len_lo=16484, len_hi=16484, page=64,
             keep=8192, first=4, recent=512),
        # One long document down to a quarter.
        dict(name="evict-long", op="evict", dtype="f16", b=1, h_kv=8, d=128, len_lo=262161, len_hi=262161, page=128,
             keep=65536, first=16, recent=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "append", "weigh", "evict"])
    top = {o: max(_cost(c) for c in listed() if c["op"] == o) for o in ("forward", "append", "weigh", "evict")}
    while True:
        c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), b=_log(rng, 1, 64), d=rng.choice([64, 128]),
                 h_kv=rng.choice([1, 2, 3, 4, 6, 8, 16]), page=rng.choice([0, 16, 24, 64, 128, 256]))
        c["len_hi"] = _log(rng, 1, 262144)
        c["len_lo"] = rng.choice([0, c["len_hi"], rng.randint(0, c["len_hi"])])
        if op in ("forward", "weigh"):
            c["h_q"] = c["h_kv"] * rng.choice([1, 2, 4, 5, 8, 16])
            c["t"] = rng.choice([1, _log(rng, 1, 64)])
            c["window"] = rng.choice([-1, -1, _log(rng, 1, 8192)])
        if op == "forward":
            c["sink"] = rng.random() < 0.3
        if op == "append":
            c["picked"] = rng.random() < 0.5
            c["t"] = _log(rng, 1, 64) if c["picked"] else _log(rng, 1, 8192)
        if op == "evict":
            c["keep"] = _log(rng, 1, c["len_hi"])
            c["first"] = rng.randint(0, min(16, c["keep"]))
            c["recent"] = rng.randint(0, (c["keep"] - c["first"]) // 2)
        pool = c["b"] * (c["len_hi"] + c.get("t", 0)) * c["h_kv"] * c["d"]
        scores = c["b"] * c.get("h_q", 0) * c.get("t", 0) * c["len_hi"]
        if _cost(c) <= top[op] and pool <= 2 ** 30 and scores <= 2 ** 28 * 1.5:
            return c


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def _lengths(case):
    """Cached keys of each sequence: spread over the logarithm from len_lo to len_hi, in an order of no kind."""
    b, lo, hi = case["b"], case["len_lo"], case["len_hi"]
    if b == 1:
        return [hi]
    got = [int(round(math.exp(math.log(lo + 1) + (math.log(hi + 1) - math.log(lo + 1)) * i / (b - 1)))) - 1
           for i in range(b)]
    np.random.RandomState(7).shuffle(got)
    return got


def _counts(case):
    """Rows that each sequence appends: 1 to t."""
    return np.random.RandomState(11).randint(1, case["t"] + 1, case["b"]).tolist()


def work(case):
    """Each key and value row that the masks reach read once, each output written once."""
    lens, d, h_kv, b = _lengths(case), case["d"], case["h_kv"], case["b"]
    if case["op"] == "append":
        rows = sum(_counts(case)) * h_kv
        return {"bytes": float(rows * (8 * d + 8)), "flops": 0.0}
    if case["op"] == "evict":
        # the accounts of weights and positions, and the rows that move: weights of no order free the budget's places
        # in the share that is evicted
        over = [n for n in lens if n > case["keep"]]
        moved = sum(case["keep"] * (n - case["keep"]) / n for n in over) * h_kv
        return {"bytes": float(sum(over) * h_kv * 8 + moved * (8 * d + 8)), "flops": 0.0}
    t, h_q = case["t"], case["h_q"]
    reach = [n if case["window"] < 0 else min(n, case["window"] + t - 1) for n in lens]
    keys = sum(reach) * h_kv
    pairs = sum(reach) * t * h_q
    q = b * t * h_q * d * 2
    if case["op"] == "weigh":
        return {"bytes": float(keys * (2 * d + 8) + q + b * h_q * t * 4), "flops": float(pairs * 2 * d)}
    return {"bytes": float(keys * 4 * d + b * t * h_kv * 4 * d + 2 * q + b * h_q * t * 4),
            "flops": float(pairs * 4 * d + b * t * t * h_q * 4 * d)}


# ----------------------------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 1009 + 1)
    dt = DTYPES[case["dtype"]]
    b, h_kv, d, op = case["b"], case["h_kv"], case["d"], case["op"]
    lens = _lengths(case)
    room = max(lens) + (case["t"] if op == "append" else 0)
    page = case["page"] or max(1, room)
    table_w = max(1, -(-room // page))
    n_pages = b * table_w
    cap = table_w * page

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = dict(case=case, k_pages=normal(n_pages, page, h_kv, d), v_pages=normal(n_pages, page, h_kv, d))
    s["table"] = (torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).view(b, table_w)
                  if case["page"] else torch.arange(b, device=dev, dtype=torch.int32).view(b, 1))
    # lengths, next positions, positions and weights lie in one buffer, so that a pass can put back what it changes
    kept = op in ("append", "evict", "weigh")
    r4 = lambda n: -(-n // 4) * 4  # noqa: E731
    sizes = [r4(b), r4(b)] + ([b * h_kv * cap, b * h_kv * cap] if kept else [])
    meta = torch.zeros(sum(r4(n) for n in sizes), device=dev, dtype=torch.int32)
    at = np.cumsum([0] + [r4(n) for n in sizes]).tolist()
    s["meta"] = meta
    s["lengths"] = meta[:b]
    s["next_pos"] = meta[at[1]:at[1] + b]
    s["lengths"].copy_(torch.tensor(lens, dtype=torch.int32))
    s["next_pos"].copy_(s["lengths"])
    s["positions"] = s["weights"] = None
    if kept:
        s["positions"] = meta[at[2]:at[2] + sizes[2]].view(b, h_kv, cap)
        s["weights"] = meta[at[3]:at[3] + sizes[3]].view(torch.float32).view(b, h_kv, cap)
        slot = torch.arange(cap, device=dev, dtype=torch.int32)
        held = slot < s["lengths"][:, None, None]
        if op == "evict":
            # what earlier evictions left: growing positions with gaps, in another order for each head
            pos = torch.randint(1, 4, (b, cap), generator=g, device=dev).cumsum(1).to(torch.int32)
            last = torch.where(s["lengths"] > 0, pos.gather(1, (s["lengths"].long() - 1).clamp(min=0)[:, None])[:, 0], -1)
            s["next_pos"].copy_(last + 1)
            mix = torch.where(held, torch.rand(b, h_kv, cap, generator=g, device=dev), 2.0).argsort(-1)
            s["positions"].copy_(torch.where(held, pos[:, None].expand(b, h_kv, cap).gather(2, mix), -1))
            # a few heavy keys, many light ones, and ties among the lightest
            heavy = (normal(b, h_kv, cap, dtype=torch.float32) * 2).exp()
            s["weights"].copy_(torch.where(held, torch.floor(heavy * 64) / 64, 0.0))
        else:
            s["positions"].copy_(torch.where(held, slot, -1))
            s["weights"].copy_(torch.where(held, normal(b, h_kv, cap, dtype=torch.float32).abs(), 0.0))
    if op in ("forward", "weigh"):
        t, h_q = case["t"], case["h_q"]
        s["q"] = normal(b, t, h_q, d)
        s["scale"] = d ** -0.5
    if op == "forward":
        s["k_new"], s["v_new"] = normal(b, t, h_kv, d), normal(b, t, h_kv, d)
        s["sink"] = normal(h_q, dtype=torch.float32) if case["sink"] else None
        # a tree: each node hangs from one of the few nodes before it
        masks = []
        rs = np.random.RandomState(int(seed) % 2 ** 31)
        for _ in range(b):
            m = []
            for i in range(t):
                m.append((1 << i) | (m[max(0, i - 1 - int(rs.randint(0, 4)))] if i else 0))
            masks.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in m])
        s["tree"] = torch.tensor(masks, dtype=torch.int64, device=dev)
    if op == "weigh":
        # the rows are the last ones; their LSE is what scores of unit variance give
        s["q_pos"] = (s["next_pos"][:, None] - t + torch.arange(t, device=dev, dtype=torch.int32)).clamp(min=-1).contiguous()
        n = (s["q_pos"] + 1).clamp(min=1).float()
        if case["window"] >= 0:
            n = n.clamp(max=case["window"] + 1)
        s["lse"] = (n.log() + 0.5)[:, None] + 0.1 * normal(b, h_q, t, dtype=torch.float32)
    if op == "append":
        t = case["t"]
        cnt = _counts(case)
        s["counts"] = torch.tensor(cnt, dtype=torch.int32, device=dev)
        if case["picked"]:
            s["k_new"], s["v_new"] = normal(b, t, h_kv, d), normal(b, t, h_kv, d)
            s["index"] = torch.rand(b, t, generator=g, device=dev).argsort(1).sort(1)[1].to(torch.int32).contiguous()
        else:
            s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32, device=dev)
            s["k_new"], s["v_new"] = normal(sum(cnt), h_kv, d), normal(sum(cnt), h_kv, d)
            s["longest"] = max(cnt)
    s["meta0"] = s["meta"].clone()
    if own:
        import sliding_window_attention_sdpa_gb300 as swa
        s["cache"] = swa.KVCache(s["k_pages"], s["v_pages"], s["lengths"], page_table=s["table"] if case["page"] else None,
                                 next_pos=s["next_pos"] if kept else None, positions=s["positions"], weights=s["weights"])
    return s


# ---------------------------------------------------------------------------------------------------- the operators

def run(s):
    case = s["case"]
    op = case["op"]
    if op != "forward":
        s["meta"].copy_(s["meta0"])  # each pass starts from the same account
    if own:
        import sliding_window_attention_sdpa_gb300 as swa
        if op == "forward":
            return swa.cache_forward(s["cache"], s["q"], s["k_new"], s["v_new"], scale=s["scale"],
                                     window_left=case["window"], tree=s["tree"], sink=s["sink"])
        if op == "append":
            if case["picked"]:
                swa.cache_append(s["cache"], s["k_new"], s["v_new"], index=s["index"], counts=s["counts"])
            else:
                swa.cache_append(s["cache"], s["k_new"], s["v_new"], offsets=s["offsets"], max_seqlen=s["longest"])
        if op == "weigh":
            swa.cache_weigh(s["cache"], s["q"], s["lse"], scale=s["scale"], window_left=case["window"], q_pos=s["q_pos"])
            return s["weights"]
        if op == "evict":
            swa.cache_evict(s["cache"], case["keep"], first=case["first"], recent=case["recent"])
    elif op == "forward":
        return _forward(s)
    elif op == "append":
        _append(s)
    elif op == "weigh":
        return _weigh(s)
    else:
        _evict(s)
    return [s["k_pages"], s["v_pages"], s["lengths"], s["next_pos"], s["positions"], s["weights"]]


def _rows(s, slots):
    """Page and place of each sequence's slots ([b, n])."""
    page = s["k_pages"].shape[1]
    slots = slots.long()
    return s["table"].long().gather(1, slots // page), slots % page


def _forward(s):
    case, q = s["case"], s["q"]
    b, t, h_q, d = q.shape
    h_kv, w = case["h_kv"], case["window"]
    dev = q.device
    # the latest n slots of each sequence hold every key that a row can see
    n = max(1, case["len_hi"] if w < 0 else min(case["len_hi"], w))
    n = min(n, s["table"].shape[1] * s["k_pages"].shape[1])
    first = (s["lengths"] - n).clamp(min=0)
    slots = first[:, None] + torch.arange(n, device=dev, dtype=torch.int32)
    pg, at = _rows(s, slots)
    k, v = s["k_pages"][pg, at].float(), s["v_pages"][pg, at].float()
    k = torch.cat([k, s["k_new"].float()], 1)
    v = torch.cat([v, s["v_new"].float()], 1)
    bit = (s["tree"][:, :, None] >> torch.arange(t, device=dev)) & 1
    depth = bit.sum(-1) - 1
    back = (s["lengths"][:, None] + depth)[:, :, None] - slots[:, None]
    see = (slots < s["lengths"][:, None])[:, None].expand(b, t, n)
    see_new = bit == 1
    if w >= 0:
        see = see & (back <= w)
        see_new = see_new & (depth[:, :, None] - depth[:, None] <= w)
    see = torch.cat([see, see_new], 2)
    qg = q.float().view(b, t, h_kv, h_q // h_kv, d)
    score = torch.einsum("btkgd,bnkd->bkgtn", qg, k) * s["scale"]
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
    lse = (top + total.log()).view(b, h_q, t)
    return o, lse


def _append(s):
    case = s["case"]
    dev = s["k_pages"].device
    i = torch.arange(case["t"], device=dev, dtype=torch.int32)
    fresh = i < s["counts"][:, None]
    if case["picked"]:
        k, v = (x[torch.arange(case["b"], device=dev)[:, None], s["index"].long()] for x in (s["k_new"], s["v_new"]))
        k, v = k[fresh], v[fresh]
    else:
        k, v = s["k_new"], s["v_new"]
    slots = (s["lengths"][:, None] + i)
    cap = s["positions"].shape[2]
    pg, at = _rows(s, slots.clamp(max=cap - 1))
    s["k_pages"][pg[fresh], at[fresh]] = k
    s["v_pages"][pg[fresh], at[fresh]] = v
    seq = torch.arange(case["b"], device=dev)[:, None].expand_as(slots)[fresh]
    s["positions"].transpose(1, 2)[seq, slots[fresh].long()] = (s["next_pos"][:, None] + i)[fresh][:, None].expand(-1, case["h_kv"])
    s["weights"].transpose(1, 2)[seq, slots[fresh].long()] = 0.0
    s["lengths"] += s["counts"]
    s["next_pos"] += s["counts"]


def _weigh(s):
    case, q = s["case"], s["q"]
    b, t, h_q, d = q.shape
    h_kv, w = case["h_kv"], case["window"]
    cap = s["weights"].shape[2]
    slots = torch.arange(cap, device=q.device, dtype=torch.int32).expand(b, cap)
    pg, at = _rows(s, slots)
    k = s["k_pages"][pg, at].float()
    qg = q.float().view(b, t, h_kv, h_q // h_kv, d)
    score = torch.einsum("btkgd,bnkd->bktgn", qg, k) * s["scale"]
    pos, q_pos = s["positions"][:, :, None], s["q_pos"][:, None, :, None]
    see = (slots < s["lengths"][:, None])[:, None, None] & (pos <= q_pos) & (q_pos >= 0)
    if w >= 0:
        see = see & (q_pos - pos <= w)
    p = (score - s["lse"].view(b, h_kv, h_q // h_kv, t).transpose(2, 3)[..., None]).exp()
    s["weights"] += p.masked_fill(~see[:, :, :, None], 0.0).sum((2, 3))
    return s["weights"]


def _evict(s):
    case = s["case"]
    keep, w, pos = case["keep"], s["weights"], s["positions"]
    b, h_kv, cap = w.shape
    slot = torch.arange(cap, device=w.device)
    n = s["lengths"][:, None, None]
    held = slot < n
    must = held & ((pos < case["first"]) | (pos >= s["next_pos"][:, None, None] - case["recent"]))
    rank = w.masked_fill(must, math.inf).masked_fill(~held, -math.inf).sort(dim=-1, descending=True, stable=True)[1]
    kept = torch.zeros_like(w, dtype=torch.bool).scatter_(2, rank[:, :, :keep], True) & held
    kept = torch.where(n > keep, kept, held)
    # the i-th free place below the budget takes the i-th key kept behind it; the other places take themselves
    most = min(keep, cap - keep)
    if most > 0:
        hole, tail = ~kept & (slot < keep) & (n > keep), kept & (slot >= keep)
        dst = (~hole).to(torch.uint8).sort(dim=-1, stable=True)[1][:, :, :most]
        src = (~tail).to(torch.uint8).sort(dim=-1, stable=True)[1][:, :, :most]
        real = torch.arange(most, device=w.device) < hole.sum(-1, keepdim=True)
        src = torch.where(real, src, dst)
        head = torch.arange(h_kv, device=w.device)[None, :, None].expand_as(src)
        (sp, sa), (dp, da) = (_rows(s, x.reshape(b, -1)) for x in (src, dst))
        head = head.reshape(b, -1)
        for pool in (s["k_pages"], s["v_pages"]):
            pool[dp, da, head] = pool[sp, sa, head]
        pos.scatter_(2, dst, pos.gather(2, src))
        w.scatter_(2, dst, w.gather(2, src))
    s["lengths"].clamp_(max=keep)


# ------------------------------------------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"forward": _exact_forward, "append": _exact_append, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _keys(s, pool, i, head):
    """Sequence i's slots of one head, in order, in 64 bits."""
    return pool[s["table"][i].long(), :, head].flatten(0, 1).double()


def _exact_forward(s):
    case = s["case"]
    q = s["q"].double()
    b, t, h_q, d = q.shape
    group, w = h_q // case["h_kv"], case["window"]
    o = torch.zeros(b, t, h_q, d, dtype=torch.float64, device=q.device)
    lse = torch.full((b, h_q, t), -math.inf, dtype=torch.float64, device=q.device)
    lens = _lengths(case)
    for i in range(b):
        n = lens[i]
        lines = [int(x) % 2 ** 64 for x in s["tree"][i].tolist()]
        see = np.zeros((t, n + t), dtype=bool)
        deep = [bin(x).count("1") - 1 for x in lines]
        for r in range(t):
            see[r, max(0, n + deep[r] - w) if w >= 0 else 0:n] = True
            for u in range(t):
                see[r, n + u] = bool(lines[r] >> u & 1) and (w < 0 or deep[r] - deep[u] <= w)
        lo = int(see.any(0).argmax())
        see = torch.from_numpy(see[:, lo:]).to(q.device)
        for kv in range(case["h_kv"]):
            k = torch.cat([_keys(s, s["k_pages"], i, kv)[:n], s["k_new"][i, :, kv].double()])[lo:]
            v = torch.cat([_keys(s, s["v_pages"], i, kv)[:n], s["v_new"][i, :, kv].double()])[lo:]
            rows = q[i, :, kv * group:(kv + 1) * group].transpose(0, 1).reshape(group * t, d)
            a = (rows @ k.T * s["scale"]).view(group, t, -1).masked_fill(~see, -math.inf)
            z = torch.logsumexp(a, -1)
            if s["sink"] is not None:
                z = torch.logaddexp(z, s["sink"][kv * group:(kv + 1) * group].double()[:, None])
            o[i, :, kv * group:(kv + 1) * group] = (torch.exp(a - z[..., None]).view(group * t, -1) @ v).view(group, t, d).transpose(0, 1)
            lse[i, kv * group:(kv + 1) * group] = z
    return o, lse


def _exact_append(s):
    case = s["case"]
    pools = [s["k_pages"], s["v_pages"]]
    page = pools[0].shape[1]
    start = 0
    for i, (n, c) in enumerate(zip(_lengths(case), _counts(case))):
        rows = s["index"][i, :c].long() if case["picked"] else torch.arange(start, start + c, device=pools[0].device)
        start += c
        slots = np.arange(n, n + c)
        pg = s["table"][i].long()[torch.from_numpy(slots // page).to(rows.device)]
        at = torch.from_numpy(slots % page).to(rows.device)
        for pool, new in zip(pools, (s["k_new"], s["v_new"])):
            pool[pg, at] = (new[i] if case["picked"] else new)[rows]
        s["positions"][i, :, n:n + c] = torch.arange(n, n + c, device=rows.device, dtype=torch.int32)
        s["weights"][i, :, n:n + c] = 0
        s["lengths"][i] = n + c
        s["next_pos"][i] = n + c
    return pools + [s["lengths"], s["next_pos"], s["positions"], s["weights"]]


def _exact_weigh(s):
    case = s["case"]
    w = s["weights"].double()
    group = case["h_q"] // case["h_kv"]
    for i, n in enumerate(_lengths(case)):
        for kv in range(case["h_kv"]):
            k = _keys(s, s["k_pages"], i, kv)[:n]
            pos = s["positions"][i, kv, :n]
            for r, p in enumerate(s["q_pos"][i].tolist()):
                if p < 0 or n == 0:
                    continue
                heads = slice(kv * group, (kv + 1) * group)
                a = (s["q"][i, r, heads].double() @ k.T * s["scale"] - s["lse"][i, heads, r].double()[:, None]).exp().sum(0)
                a[pos > p] = 0
                if case["window"] >= 0:
                    a[pos < p - case["window"]] = 0
                w[i, kv, :n] += a
    return w


def _exact_evict(s):
    case = s["case"]
    keep = case["keep"]
    page = s["k_pages"].shape[1]
    pos, w = s["positions"].cpu().numpy(), s["weights"].cpu().numpy()
    table, after = s["table"].cpu().numpy(), s["next_pos"].cpu().numpy()
    seqs, heads, src, dst = [], [], [], []
    lens = _lengths(case)
    for i, n in enumerate(lens):
        if n <= keep:
            continue
        s["lengths"][i] = keep
        for kv in range(case["h_kv"]):
            p = pos[i, kv, :n]
            light = np.flatnonzero((p >= case["first"]) & (p < after[i] - case["recent"]))
            order = light[np.lexsort((light, -w[i, kv, light].astype(np.float64)))]
            gone = order[keep - (n - len(light)):]
            free = np.sort(gone[gone < keep])
            stay = np.ones(n, dtype=bool)
            stay[gone] = False
            come = np.flatnonzero(stay[keep:])[:len(free)] + keep
            seqs.append(np.full(len(free), i))
            heads.append(np.full(len(free), kv))
            src.append(come)
            dst.append(free)
    if seqs:
        seqs, heads, src, dst = (np.concatenate(x) for x in (seqs, heads, src, dst))
        dev = s["k_pages"].device
        on = lambda x: torch.from_numpy(np.ascontiguousarray(x)).long().to(dev)  # noqa: E731
        sp, dp = on(table[seqs, src // page]), on(table[seqs, dst // page])
        sa, da, hh, ss = on(src % page), on(dst % page), on(heads), on(seqs)
        for pool in (s["k_pages"], s["v_pages"]):
            pool[dp, da, hh] = pool[sp, sa, hh]
        s["positions"][ss, hh, on(dst)] = s["positions"][ss, hh, on(src)]
        s["weights"][ss, hh, on(dst)] = s["weights"][ss, hh, on(src)]
    return [s["k_pages"], s["v_pages"], s["lengths"], s["next_pos"], s["positions"], s["weights"]]
