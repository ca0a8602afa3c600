"""CPU checks of the cache in 4 bits and of reading a cache: every refusal that
needs no device (the C entry points check shapes before any pointer)."""
import ctypes

import pytest
import torch

import sliding_window_attention_sdpa_gb300 as swa
from test_cache_host import INVALID, UNSUP, append, cache, fwd, refused, weigh


@pytest.fixture(scope="module", autouse=True)
def lib():
    swa._build.build()
    return swa.load()


def test_struct_matches_binding(lib):
    assert lib.sdpa_cache_read_params_bytes() == ctypes.sizeof(swa.SdpaCacheReadParams)


GROUPS = swa._i64x3(4 * 9 * 64, 9 * 64, 9 * 64)


def cache4(**kw):
    return cache(**dict(dict(bits=4, page_size=16, k_stride=GROUPS, v_stride=GROUPS), **kw))


def read(**kw):
    p = swa.SdpaCacheReadParams()
    p.layout, p.s = swa.SDPA_BSHD, 5
    p.k_stride = p.v_stride = swa._i64x3(5 * 4 * 64, 4 * 64, 64)
    p.k = p.v = 4096
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code,needle", [
    (dict(bits=8), INVALID, "bits=8"), (dict(bits=-4), INVALID, "bits=-4"),
    (dict(page_size=24), UNSUP, "page_size=24"),
    (dict(k_stride=swa._i64x3(2304, 64, 576)), INVALID, "k_stride[1]=64"),
    (dict(v_stride=swa._i64x3(2304, 576, 584)), INVALID, "v_stride[2]=584"),
    (dict(v_stride=swa._i64x3(-2304, 576, 576)), INVALID, "v_stride[0]"),
    (dict(d=96), UNSUP, "d=96"), (dict(dtype=7), INVALID, "dtype"), (dict(page_table=0), INVALID, "page_table"),
])
def test_cache_refusals(kw, code, needle):
    c = cache4(**kw)
    refused(code, swa.sdpa_cache_fwd(c, fwd(), 4096, 1 << 40, 0), needle)
    refused(code, swa.sdpa_cache_append(c, append(), 0), needle)
    refused(code, swa.sdpa_cache_read(c, read(), 0), needle)
    assert swa.sdpa_cache_fwd_workspace_bytes(c, fwd()) == 0


def test_what_it_does_not_do():
    refused(UNSUP, swa.sdpa_cache_weigh(cache4(), weigh(), 0), "4 bits")
    refused(UNSUP, swa.sdpa_cache_evict(cache4(), swa.SdpaCacheEvictParams(4, 0, 0), 4096, 1 << 40, 0), "4 bits")
    assert swa.sdpa_cache_evict_workspace_bytes(cache4(), swa.SdpaCacheEvictParams(4, 0, 0)) == 0 and "4 bits" in swa.last_error()
    refused(UNSUP, swa.sdpa_cache_fwd(cache4(), fwd(s_q=65), 4096, 1 << 40, 0), "s_q=65")


@pytest.mark.parametrize("bits", [0, 4, 16])
@pytest.mark.parametrize("kw,code,needle", [
    (dict(layout=4), INVALID, "layout"), (dict(s=-1), INVALID, "s=-1"), (dict(s=2 ** 31), INVALID, "s="),
    (dict(layout=1, total=-1, offsets=4096), INVALID, "total=-1"), (dict(layout=1, total=4), INVALID, "offsets"),
    (dict(k_stride=swa._i64x3(8, 12, 8)), INVALID, "k_stride[1]"), (dict(v_stride=swa._i64x3(8, 8, -8)), INVALID, "v_stride[2]"),
])
def test_read_refusals(bits, kw, code, needle):
    refused(code, swa.sdpa_cache_read(cache4() if bits == 4 else cache(bits=bits), read(**kw), 0), needle)
    assert swa.sdpa_cache_read(cache4() if bits == 4 else cache(bits=bits), None, 0) == INVALID


def test_read_refuses_more_rows_than_a_launch_has():
    for c in (cache4(b=1 << 20), cache(b=1 << 20)):
        refused(UNSUP, swa.sdpa_cache_read(c, read(s=1 << 20), 0), "rows")


def test_workspace_follows_the_work():
    """None for short units (one CTA each), else two partials of a part's rows."""
    assert swa.sdpa_cache_fwd_workspace_bytes(cache4(max_pages=20), fwd()) == 0 and swa.last_error() == ""
    few = swa.sdpa_cache_fwd_workspace_bytes(cache4(max_pages=1000, n_pages=2000), fwd(s_q=1))
    tile = swa.sdpa_cache_fwd_workspace_bytes(cache4(max_pages=1000, n_pages=2000), fwd(s_q=64))
    assert 0 < few < tile


def test_calls_refuse_wrong_tensors():
    u8, i32 = torch.uint8, torch.int32
    k = torch.zeros(4, 2, 2, 9 * 64, dtype=u8)
    n, table = torch.zeros(2, dtype=i32), torch.zeros(2, 2, dtype=i32)
    c = swa.KVCache(k, k.clone(), n, page_table=table, dtype=torch.bfloat16)
    assert (c.bits, c.d, c.h_kv, c.capacity, c.dtype) == (4, 64, 2, 64, torch.bfloat16)
    for kw, needle in [(dict(k=k, v=k.clone()), "needs that of"), (dict(k=k, v=k.clone(), dtype=torch.float32), "unsupported dtype"),
                       (dict(k=k[0], v=k[0], dtype=torch.float16), "expected"), (dict(k=k[..., :-1], v=k, dtype=torch.float16), "groups of 9 d"),
                       (dict(k=k[:, :, ::2].repeat(1, 1, 2, 1)[:, :, ::1], v=torch.zeros(4, 2, 4, 576, dtype=u8)[:, :, ::2], dtype=torch.float16),
                        "must follow one another"),
                       (dict(k=torch.zeros(4, 16, 2, 64, dtype=torch.float16), v=torch.zeros(4, 16, 2, 64, dtype=torch.float16), dtype=torch.bfloat16),
                        "k is torch.float16")]:
        with pytest.raises(ValueError, match=needle):
            swa.KVCache(kw["k"], kw["v"], n, page_table=table, dtype=kw.get("dtype"))
    for kw, needle in [(dict(bits=8), "bits=8"), (dict(bits=4, page_size=24), "page_size=24")]:
        with pytest.raises(ValueError, match=needle):
            swa.KVCache.empty(2, 2, 64, 100, dtype=torch.float16, device="cpu", **kw)
    with pytest.raises(AttributeError, match="bits"):
        c.bits = 16
    off = torch.zeros(3, dtype=i32)
    for kw, needle in [(dict(offsets=off), "total"), (dict(total=4), "only with offsets"), (dict(offsets=off, total=4, max_rows=2), "max_rows"),
                       (dict(max_rows=-1), "max_rows"), (dict(offsets=off[:2], total=4), "offsets: expected shape"),
                       (dict(start=off), "start: expected shape"), (dict(counts=n.long()), "counts: expected dtype"),
                       (dict(max_rows=3, out=(torch.zeros(2, 3, 2, 64),) * 2), "out k: expected dtype"),
                       (dict(max_rows=3, out=(torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16).expand(2, 3, 2, 64),) * 2), "share memory")]:
        with pytest.raises(ValueError, match=needle):
            swa.cache_read(c, **kw)
