"""CPU checks of the key/value cache's calls: refusals at the edges of their forms."""
import pytest
import torch

import sliding_window_attention_sdpa_gb300 as swa
from test_cache_host import lib, tensors  # noqa: F401  (the built library)


@pytest.mark.parametrize("width", [0, 3])
def test_packed_rows_take_no_index(width):
    """An index of no columns too (its address is NULL, so that the library
    could not see it)."""
    c, k = tensors(), torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="index"):
        swa.cache_append(c, k, k, offsets=torch.tensor([0, 2, 5], dtype=torch.int32), max_seqlen=3,
                         index=torch.zeros(2, width, dtype=torch.int32))
