"""CPU checks of tensors that are missing: norm and rotation's calls, and reading a cache."""
import pytest
import torch

import sliding_window_attention_sdpa_gb300 as swa


@pytest.fixture(scope="module", autouse=True)
def lib():
    swa._build.build()
    return swa.load()


def test_missing_tensors_are_named():
    q, k = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    pos, freq, w = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(32), torch.zeros(64)
    kw = dict(q_weight=w, k_weight=w)
    for args, more, needle in [((q, k, None, k), kw, "q: needed"), ((q, k, q, None), kw, "k: needed"), ((q, k, None, None), kw, "q: needed"),
                               ((q, None, None, None), dict(q_weight=w), "q: needed"),
                               ((q, k, q, k), dict(kw, out=(None, k)), "out q: needed"), ((q, k, q, k), dict(kw, out=(q, None)), "out k: needed")]:
        with pytest.raises(ValueError, match=needle):
            swa.qk_rotate_backward(*args, pos, freq, **more)
    for out, needle in [((None, k), "out q: needed"), ((q, None), "out k: needed")]:
        with pytest.raises(ValueError, match=needle):
            swa.qk_rotate(q, k, pos, freq, out=out)


def test_missing_outputs_of_a_read_are_named():
    i32 = torch.int32
    k = torch.zeros(4, 2, 2, 9 * 64, dtype=torch.uint8)
    c = swa.KVCache(k, k.clone(), torch.zeros(2, dtype=i32), page_table=torch.zeros(2, 2, dtype=i32), dtype=torch.bfloat16)
    o = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    for out, needle in [((None, o), "out k: needed"), ((o, None), "out v: needed")]:
        with pytest.raises(ValueError, match=needle):
            swa.cache_read(c, max_rows=3, out=out)
