"""Bounded waits of the key/value cache's kernels: a wait that runs out is
reported, not hung on. The library's test hook shortens the limit to a few
milliseconds and leaves an early copy out; the kernel must then report
SDPA_ERR_TIMEOUT, end what it has in flight and leave the device usable, and the
same call without the hook must give the right result."""
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
