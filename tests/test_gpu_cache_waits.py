"""Bounded waits of the key/value cache's kernels: a wait that runs out is
reported, not hung on. The library's test hook shortens the limit to a few
milliseconds and leaves an early copy out; the kernel must then report
SDPA_ERR_TIMEOUT, end what it has in flight and leave the device usable, and the
same call without the hook must give the bits that it gave before."""
import pytest
import torch

import cache_ref as R
import sliding_window_attention_sdpa_gb300 as swa


def test_hook_rejects_unknown_flags():
    swa._build.build()
    assert swa.sdpa_cache_test_hook(0, 2) == swa.SDPA_ERR_INVALID_ARG
    assert "flags" in swa.last_error()
    assert swa.sdpa_cache_test_hook(0, 0) == swa.SDPA_OK


def runs_out(cache, call):
    assert swa.sdpa_cache_test_hook(2_000_000, 1) == swa.SDPA_OK
    try:
        call()
    finally:
        swa.sdpa_cache_test_hook(0, 0)
    with pytest.raises(swa.SdpaError) as e:
        cache.check_status()
    assert e.value.code == swa.SDPA_ERR_TIMEOUT, str(e.value)
    cache.check_status()               # cleared, and the device answers


# lens, t, h_q, h_kv, d, dtype, page, long enough for several copies in each CTA's part: the kernel for few rows
# (boxes, single rows; cut, uncut), then the tile kernel (one row tile, two, both; boxes, gathered rows; cut, uncut)
FORWARD = {
    "few": ([30000, 10], 1, 8, 2, 128, "bf16", 64), "few_odd_pages": ([60000, 10], 1, 8, 2, 64, "f16", 7),
    "few_uncut": ([300, 200], 1, 8, 2, 128, "f16", 16),
    "tile": ([60000, 40], 5, 8, 1, 128, "bf16", 64), "tile_d64": ([30000, 40], 40, 8, 2, 64, "f16", 64),
    "tile_odd_pages": ([15000, 40], 37, 16, 2, 128, "bf16", 7), "tile_two": ([60000, 40], 32, 8, 1, 128, "bf16", 16),
    "tile_uncut": ([300, 200], 37, 16, 2, 64, "bf16", 64),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", FORWARD)
def test_forward_waits_run_out(name):
    from test_gpu_cache import dev, gpu_cache, inputs, same_cache
    lens, t, h_q, h_kv, d, dtype, page = FORWARD[name]
    lay = R.make(611, lens, h_kv, d, dtype, page)
    q, k, v = inputs(612, len(lens), t, h_q, h_kv, d, dtype)
    c, x = gpu_cache(lay), [dev(y) for y in (q, k, v)]
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")
    want = swa.cache_forward(c, *x, scale=0.1, workspace=ws, check_status=True)
    runs_out(c, lambda: swa.cache_forward(c, *x, scale=0.1, workspace=ws))
    got = swa.cache_forward(c, *x, scale=0.1, workspace=ws, check_status=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    same_cache(c, lay)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,t,d,page,window", [([700] * 300, 1, 64, 64, -1), ([700] * 300, 1, 128, 7, -1),
                                                  ([700] * 300, 40, 128, 64, -1), ([3000] * 160, 70, 64, 64, 1500)])
def test_weigh_waits_run_out(lens, t, d, page, window):
    """More sequences than CTAs: each has several to look after."""
    from test_gpu_cache import dev, gpu_cache, randn
    lay = R.make(621, lens, 1, d, "bf16", page, tracked=True)
    if window >= 0:
        lay.positions = lay.next_pos = None       # rows that reach some tiles only
    q, lse = (dev(x) for x in (randn(622, len(lens), t, 8, d, dtype=torch.bfloat16),
                           randn(623, len(lens), 8, t) + 4))

    def weighed(stall=False):
        c = gpu_cache(lay)
        if stall:
            runs_out(c, lambda: swa.cache_weigh(c, q, lse, scale=0.1, window_left=window))
        else:
            swa.cache_weigh(c, q, lse, scale=0.1, window_left=window, check_status=True)
        return torch.nan_to_num(c.weights)
    want = weighed()
    weighed(stall=True)
    assert torch.equal(weighed(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_evict_waits_run_out(d):
    """160 heads on 456 CTAs: each moves about 400 rows, several rounds of its
    warps."""
    from test_gpu_cache import gpu_cache, same_cache
    lay = R.make(601, [1600] * 40, 4, d, "bf16", 64, evicted=True)
    c = gpu_cache(lay)
    runs_out(c, lambda: swa.cache_evict(c, 800))
    c = gpu_cache(lay)
    swa.cache_evict(c, 800, check_status=True)
    same_cache(c, R.evict(lay, 800, 0, 0))
