"""Plain 64-bit forms of the cache in 4 bits, for the tests: what rows are held
as, by a search over all scales and all codes (every distance below is exact in
64 bits), sharing no code with the CUDA path."""
from __future__ import annotations

import numpy as np
import torch

import cache_ref as R

# all scales: 3 mantissa bits, normal from 2^-14 on, up to 240
SCALES = np.array([m * 2.0 ** -17 for m in range(8)] +
                  [z for e in range(22) for z in ((8 + m) * 2.0 ** (e - 17) for m in range(8)) if z <= 240])
CODES = np.arange(-8, 8)


def held(x: torch.Tensor) -> torch.Tensor:
    """The values [.., d] that rows stand for, in their type (NaN blocks as NaN)."""
    f = x.double().numpy().reshape(-1, 16)
    bad = ~np.isfinite(f).all(1)
    f = np.where(bad[:, None], 0.0, f)
    a = np.abs(f).max(1)
    # the nearest scale to a / 7; of two, the one with the even mantissa (the even place in the table)
    far = np.abs(a[:, None] - 7 * SCALES)
    near = far == far.min(1, keepdims=True)
    even = near & (np.arange(len(SCALES)) % 2 == 0)
    s = SCALES[np.where(even.any(1), even.argmax(1), near.argmax(1))]
    far = np.abs(f[:, :, None] - s[:, None, None] * CODES)
    near = far == far.min(2, keepdims=True)
    even = near & (CODES % 2 == 0)
    c = CODES[np.where(even.any(2), even.argmax(2), near.argmax(2))]
    out = np.where(bad[:, None], np.nan, c * s[:, None])
    return torch.from_numpy(out.reshape(x.shape)).to(x.dtype)


def held_layout(lay: R.Layout) -> R.Layout:
    """The same cache with its keys' rows as they are held."""
    out = lay.clone()
    for i, n in enumerate(lay.lengths.tolist()):
        pg, at = lay.where(i, np.arange(n))
        out.k[pg, at], out.v[pg, at] = held(lay.k[pg, at]), held(lay.v[pg, at])
    return out


def gpu_cache(lay: R.Layout, fill=0xff):
    """A cache in 4 bits on the GPU that has taken in the layout's rows; every
    byte that no row's codes have is `fill` (0xff: scales that are NaN)."""
    import sliding_window_attention_sdpa_gb300 as swa
    n_pages, page, h_kv, d = lay.k.shape
    assert page % 16 == 0
    lens = lay.lengths.tolist()
    pools = [torch.full((n_pages, h_kv, page // 16, 9 * d), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    c = swa.KVCache(*pools, torch.zeros_like(lay.lengths).cuda(), page_table=dev(lay.table), next_pos=dev(lay.next_pos),
                    positions=dev(lay.positions), weights=dev(lay.weights), dtype=lay.k.dtype)
    rows = [[], []]
    for i, n in enumerate(lens):
        pg, at = lay.where(i, np.arange(n))
        rows[0].append(lay.k[pg, at])
        rows[1].append(lay.v[pg, at])
    if lay.next_pos is not None:
        c.next_pos.zero_()
    if sum(lens):
        off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
        swa.cache_append(c, torch.cat(rows[0]).cuda(), torch.cat(rows[1]).cuda(), offsets=off, max_seqlen=max(lens),
                         check_status=True)
    if lay.next_pos is not None:
        c.next_pos.copy_(lay.next_pos)
        c.positions.copy_(lay.positions)
        c.weights.copy_(lay.weights)
    return c


def forward(lay4, q, k, v, *, dtype, **kw):
    """R.forward over the held rows. P is f16 whatever the type: for bf16 output
    its rounding and its smallest step come on top, which are those of f16 output's bound."""
    ref = R.forward(lay4, q, k, v, dtype=dtype, **kw)
    if dtype == "bf16":
        ref.tol_o = ref.tol_o + R.forward(lay4, q, k, v, dtype="f16", **kw).tol_o
    return ref
