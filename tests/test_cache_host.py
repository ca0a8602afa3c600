"""CPU checks of the key/value cache's calls: struct sizes, and every refusal
that needs no device (the C entry points check shapes before any pointer)."""
import ctypes

import pytest
import torch

import sliding_window_attention_sdpa_gb300 as swa


@pytest.fixture(scope="module", autouse=True)
def lib():
    swa._build.build()
    return swa.load()


def test_structs_match_binding(lib):
    for name, cls in (("sdpa_cache_bytes", swa.SdpaCache), ("sdpa_cache_fwd_params_bytes", swa.SdpaCacheFwdParams),
                      ("sdpa_cache_append_params_bytes", swa.SdpaCacheAppendParams),
                      ("sdpa_cache_weigh_params_bytes", swa.SdpaCacheWeighParams),
                      ("sdpa_cache_evict_params_bytes", swa.SdpaCacheEvictParams)):
        assert getattr(lib, name)() == ctypes.sizeof(cls), name


def cache(**kw):
    c = swa.SdpaCache()
    c.dtype, c.b, c.h_kv, c.d, c.n_pages, c.page_size, c.max_pages = swa.SDPA_BF16, 2, 4, 64, 8, 16, 4
    st = swa._i64x3(16 * 4 * 64, 4 * 64, 64)
    c.k_stride = c.v_stride = st
    c.k = c.v = c.page_table = c.lengths = c.status = 4096
    c.positions = c.next_pos = c.weights = 4096
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def fwd(**kw):
    p = swa.SdpaCacheFwdParams()
    p.s_q, p.h_q, p.window_left, p.scale = 3, 8, -1, 0.125
    p.q_stride = p.o_stride = swa._i64x3(3 * 8 * 64, 8 * 64, 64)
    p.k_stride = p.v_stride = swa._i64x3(3 * 4 * 64, 4 * 64, 64)
    p.q = p.k = p.v = p.o = p.lse = 4096
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def append(**kw):
    p = swa.SdpaCacheAppendParams()
    p.layout, p.s = swa.SDPA_BSHD, 3
    p.k_stride = p.v_stride = swa._i64x3(3 * 4 * 64, 4 * 64, 64)
    p.k = p.v = 4096
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def weigh(**kw):
    p = swa.SdpaCacheWeighParams()
    p.s_q, p.h_q, p.window_left, p.scale = 3, 8, -1, 0.125
    p.q_stride = swa._i64x3(3 * 8 * 64, 8 * 64, 64)
    p.q = p.lse = 4096
    for k, v in kw.items():
        setattr(p, k, v)
    return p


INVALID, UNSUP, WS = swa.SDPA_ERR_INVALID_ARG, swa.SDPA_ERR_UNSUPPORTED, swa.SDPA_ERR_WORKSPACE
ODD = swa._i64x3(16 * 4 * 64, 4 * 64 + 4, 64)
MINUS = swa._i64x3(-8, 8, 8)


def refused(code, got, needle):
    assert got == code and needle in swa.last_error(), (got, swa.last_error())


@pytest.mark.parametrize("kw,code,needle", [
    (dict(dtype=5), INVALID, "dtype"),
    (dict(d=96), UNSUP, "d=96"),
    (dict(h_kv=0), INVALID, "h_kv=0"),
    (dict(b=-1), INVALID, "b=-1"),
    (dict(page_size=0), INVALID, "page_size=0"),
    (dict(max_pages=-1), INVALID, "max_pages=-1"),
    (dict(max_pages=2 ** 20, page_size=2 ** 11), UNSUP, "capacity"),
    (dict(max_pages=2 ** 40, page_size=2 ** 40), UNSUP, "capacity"),
    (dict(b=2 ** 30), UNSUP, "b * h_kv"),
    (dict(h_kv=4097), UNSUP, "b * h_kv"),
    (dict(page_table=0), INVALID, "without a page_table"),
    (dict(page_table=0, max_pages=1, n_pages=1), INVALID, "without a page_table"),
    (dict(positions=0), INVALID, "positions and next_pos"),
    (dict(next_pos=0), INVALID, "positions and next_pos"),
    (dict(k_stride=ODD), INVALID, "cache k_stride[1]"),
    (dict(v_stride=MINUS), INVALID, "cache v_stride[0]"),
])
def test_cache_refusals(kw, code, needle):
    c = cache(**kw)
    refused(code, swa.sdpa_cache_fwd(c, fwd(), 4096, 1 << 40, 0), needle)
    refused(code, swa.sdpa_cache_append(c, append(), 0), needle)
    refused(code, swa.sdpa_cache_weigh(c, weigh(), 0), needle)
    refused(code, swa.sdpa_cache_evict(c, swa.SdpaCacheEvictParams(4, 0, 0), 4096, 1 << 40, 0), needle)
    assert swa.sdpa_cache_fwd_workspace_bytes(c, fwd()) == 0
    assert swa.sdpa_cache_evict_workspace_bytes(c, swa.SdpaCacheEvictParams(4, 0, 0)) == 0


@pytest.mark.parametrize("kw,code,needle", [
    (dict(s_q=0), UNSUP, "s_q=0"), (dict(s_q=65), UNSUP, "s_q=65"),
    (dict(h_q=6), INVALID, "h_q=6"), (dict(h_q=0), INVALID, "h_q=0"),
    (dict(h_q=2 ** 33), UNSUP, "rows"),
    (dict(window_left=-2), INVALID, "window_left=-2"),
    (dict(scale=0.0), INVALID, "scale"), (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(q_stride=ODD), INVALID, "q_stride[1]"), (dict(o_stride=MINUS), INVALID, "o_stride[0]"),
    (dict(k_stride=ODD), INVALID, "k_stride[1]"), (dict(v_stride=ODD), INVALID, "v_stride[1]"),
])
def test_forward_refusals(kw, code, needle):
    refused(code, swa.sdpa_cache_fwd(cache(), fwd(**kw), 4096, 1 << 40, 0), needle)
    assert swa.sdpa_cache_fwd_workspace_bytes(cache(), fwd(**kw)) == 0


@pytest.mark.parametrize("kw,code,needle", [
    (dict(layout=3), INVALID, "layout"), (dict(s=-1), INVALID, "s=-1"),
    (dict(index=4096, n=-1), INVALID, "n=-1"),
    (dict(layout=swa.SDPA_THD), INVALID, "offsets"),
    (dict(layout=swa.SDPA_THD, offsets=4096, index=4096), INVALID, "index"),
    (dict(layout=swa.SDPA_THD, offsets=4096, total=-1), INVALID, "total=-1"),
    (dict(k_stride=ODD), INVALID, "k_stride[1]"), (dict(v_stride=MINUS), INVALID, "v_stride[0]"),
])
def test_append_refusals(kw, code, needle):
    refused(code, swa.sdpa_cache_append(cache(), append(**kw), 0), needle)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(s_q=0), INVALID, "s_q=0"), (dict(s_q=2 ** 40), UNSUP, "rows"), (dict(h_q=6), INVALID, "h_q=6"),
    (dict(window_left=-2), INVALID, "window_left=-2"), (dict(scale=-1.0), INVALID, "scale"),
    (dict(q_stride=ODD), INVALID, "q_stride[1]"),
])
def test_weigh_refusals(kw, code, needle):
    refused(code, swa.sdpa_cache_weigh(cache(), weigh(**kw), 0), needle)


def test_weigh_and_evict_need_their_accounts():
    refused(INVALID, swa.sdpa_cache_weigh(cache(weights=0), weigh(), 0), "weights")
    e = swa.SdpaCacheEvictParams(4, 0, 0)
    refused(INVALID, swa.sdpa_cache_evict(cache(weights=0), e, 4096, 1 << 40, 0), "weights")
    refused(INVALID, swa.sdpa_cache_evict(cache(positions=0, next_pos=0), e, 4096, 1 << 40, 0), "positions")


@pytest.mark.parametrize("keep,first,recent", [(-1, 0, 0), (4, -1, 0), (4, 0, -1), (4, 3, 2), (4, 5, 0), (2 ** 31, 0, 0),
                                               (4, 2, 2 ** 63 - 1)])
def test_evict_refusals(keep, first, recent):
    e = swa.SdpaCacheEvictParams(keep, first, recent)
    refused(INVALID, swa.sdpa_cache_evict(cache(), e, 4096, 1 << 40, 0), "keep=")
    assert swa.sdpa_cache_evict_workspace_bytes(cache(), e) == 0


def test_workspace_refusals():
    big = cache(max_pages=1000)
    n = swa.sdpa_cache_fwd_workspace_bytes(big, fwd())
    assert n > 0 and n % 256 == 0
    refused(WS, swa.sdpa_cache_fwd(big, fwd(), 0, n, 0), "workspace")
    refused(WS, swa.sdpa_cache_fwd(big, fwd(), 4096 + 16, n, 0), "aligned")
    refused(WS, swa.sdpa_cache_fwd(big, fwd(), 4096, n - 1, 0), "need")
    # short ranges need none: 0 bytes and no message
    for c, p in ((cache(), fwd()), (cache(max_pages=1000), fwd(window_left=64)), (cache(b=0), fwd())):
        c.positions = c.next_pos = 0
        assert swa.sdpa_cache_fwd_workspace_bytes(c, p) == 0 and swa.last_error() == ""
    e = swa.SdpaCacheEvictParams(4, 0, 0)
    n = swa.sdpa_cache_evict_workspace_bytes(cache(), e)
    assert n > 0
    refused(WS, swa.sdpa_cache_evict(cache(), e, 0, n, 0), "workspace")
    refused(WS, swa.sdpa_cache_evict(cache(), e, 4096, n - 1, 0), "need")


def test_null_arguments():
    lib = swa.load()
    for got in (lib.sdpa_cache_fwd(None, None, 4096, 0, 0), lib.sdpa_cache_append(None, None, 0),
                lib.sdpa_cache_weigh(None, None, 0), lib.sdpa_cache_evict(None, None, 4096, 0, 0),
                lib.sdpa_cache_check_status(None, 0)):
        refused(INVALID, got, "cache is NULL")
    for got in (lib.sdpa_cache_fwd(cache(), None, 4096, 0, 0), lib.sdpa_cache_append(cache(), None, 0),
                lib.sdpa_cache_weigh(cache(), None, 0), lib.sdpa_cache_evict(cache(), None, 4096, 0, 0)):
        refused(INVALID, got, "params is NULL")


# ------------------------------------------------------------- torch helpers

def tensors(**kw):
    t = dict(k=torch.zeros(8, 16, 4, 64, dtype=torch.bfloat16), v=torch.zeros(8, 16, 4, 64, dtype=torch.bfloat16),
             lengths=torch.zeros(2, dtype=torch.int32), page_table=torch.zeros(2, 4, dtype=torch.int32))
    t.update(kw)
    k, v, n = t.pop("k"), t.pop("v"), t.pop("lengths")
    return swa.KVCache(k, v, n, **t)


@pytest.mark.parametrize("kw,needle", [
    (dict(k=torch.zeros(8, 16, 64, dtype=torch.bfloat16)), "n_pages"),
    (dict(k=torch.zeros(8, 16, 4, 64)), "dtype"),
    (dict(v=torch.zeros(8, 16, 4, 64, dtype=torch.float16)), "v: expected dtype"),
    (dict(v=torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)), "v: expected shape"),
    (dict(k=torch.zeros(8, 16, 64, 4, dtype=torch.bfloat16).transpose(2, 3)), "contiguous"),
    (dict(k=torch.zeros(1, 16, 4, 64, dtype=torch.bfloat16).expand(8, 16, 4, 64)), "share memory"),
    (dict(lengths=torch.zeros(2, dtype=torch.int64)), "lengths: expected dtype"),
    (dict(page_table=torch.zeros(3, 4, dtype=torch.int32)), "page_table: expected shape"),
    (dict(page_table=torch.zeros(4, 2, dtype=torch.int32).t()), "page_table: must be contiguous"),
    (dict(page_table=None, lengths=torch.zeros(9, dtype=torch.int32)), "needs a page"),
    (dict(next_pos=torch.zeros(2, dtype=torch.int32)), "both or neither"),
    (dict(weights=torch.zeros(2, 4, 63)), "weights: expected shape"),
    (dict(positions=torch.zeros(2, 4, 64), next_pos=torch.zeros(2, dtype=torch.int32)), "positions: expected dtype"),
])
def test_cache_constructor_refusals(kw, needle):
    with pytest.raises(ValueError, match=needle):
        tensors(**kw)


def test_calls_refuse_wrong_tensors():
    c = tensors()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q, k = bf(2, 3, 8, 64), bf(2, 3, 4, 64)
    for args, kw, needle in [
            ((bf(2, 8, 64), k, k), {}, "s_q, h_q"),
            ((bf(3, 3, 8, 64), k, k), {}, "q: expected shape"),
            ((q, bf(2, 2, 4, 64), k), {}, "k: expected shape"),
            ((q, k, k.float()), {}, "v: expected dtype"),
            ((q, k, k), dict(tree=torch.zeros(2, 3, dtype=torch.int32)), "tree: expected dtype"),
            ((q, k, k), dict(tree=torch.zeros(3, dtype=torch.int64)), "tree: expected shape"),
            ((q, k, k), dict(seq_q_lens=torch.zeros(3, dtype=torch.int32)), "seq_q_lens"),
            ((q, k, k), dict(sink=torch.zeros(4)), "sink"),
            ((q, k, k), dict(out=bf(2, 3, 8, 128)), "out"),
            ((q, k, k), dict(out=bf(2, 3, 1, 64).expand(2, 3, 8, 64)), "share memory"),
            ((q, k, k), dict(lse=torch.zeros(2, 3, 8)), "lse"),
            ((q, k, k), dict(workspace=torch.zeros(4)), "workspace")]:
        with pytest.raises(ValueError, match=needle):
            swa.cache_forward(c, *args, scale=0.1, **kw)
    for args, kw, needle in [
            ((bf(2, 3, 2, 64), k), {}, "k: expected shape"), ((k, k[:, :2]), {}, "v: expected shape"),
            ((bf(5, 4, 64), bf(5, 4, 64)), {}, "offsets and max_seqlen"), ((k[0, 0], k), {}, "expected"),
            ((k, k), dict(offsets=torch.zeros(3, dtype=torch.int32)), "offsets"),
            ((k, k), dict(index=torch.zeros(2, dtype=torch.int32)), "index"),
            ((k, k), dict(counts=torch.zeros(2)), "counts")]:
        with pytest.raises(ValueError, match=needle):
            swa.cache_append(c, *args, **kw)
    for args, kw, needle in [((q[0], None), {}, "q: expected"), ((q, torch.zeros(2, 3, 8)), {}, "lse"),
                             ((q, torch.zeros(2, 8, 3)), dict(q_pos=torch.zeros(2, 3)), "q_pos")]:
        with pytest.raises(ValueError, match=needle):
            swa.cache_weigh(c, *args, scale=0.1, **kw)
    with pytest.raises(swa.SdpaError, match="weights"):
        swa.cache_evict(c, 4)


def test_cache_attributes_are_not_replaced():
    """The calls use the addresses that the constructor took."""
    c = tensors()
    for name in ("k", "v", "lengths", "page_table", "positions", "weights", "status", "capacity"):
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, torch.zeros(2, dtype=torch.int32))
    c.lengths[0] = 3
    assert c.lengths.tolist() == [3, 0]
    c.layer = 7                             # a user's own names are free
    assert c.layer == 7


def test_rows_up_to_the_32_bit_limit():
    refused(UNSUP, swa.sdpa_cache_weigh(cache(b=1, h_kv=1), weigh(s_q=2 ** 31 - 1023, h_q=1), 0), "rows")
    refused(UNSUP, swa.sdpa_cache_weigh(cache(b=0, h_kv=1), weigh(s_q=2 ** 31 - 1, h_q=2 ** 31 - 1), 0), "rows")
    p = swa.SdpaCacheEvictParams(2 ** 30, 0, 0)
    big = cache(b=2 ** 20, h_kv=1, max_pages=2 ** 20, page_size=2 ** 10 + 1)
    refused(UNSUP, swa.sdpa_cache_evict(big, p, 4096, 1 << 62, 0), "2^50")
    assert swa.sdpa_cache_evict_workspace_bytes(big, p) == 0


def test_empty_cache_helper():
    c = swa.KVCache.empty(3, 2, 64, 100, dtype=torch.float16, device="cpu", page_size=48, track=True)
    assert c.capacity == 144 and tuple(c.page_table.shape) == (3, 3) and c.k.shape[0] == 9
    assert c.positions.shape == c.weights.shape == (3, 2, 144)
    assert sorted(c.page_table.flatten().tolist()) == list(range(9))
