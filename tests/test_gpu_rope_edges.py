"""Norm and rotation on the GPU at their edges."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,interleaved,axes", [(64, 0, 1), (128, 0, 3), (128, 1, 1)])
@pytest.mark.parametrize("packed", [False, True])
def test_no_rows_and_no_arrays(packed, d, interleaved, axes):
    """A backward pass over no rows needs no positions and no frequencies (NULL through the C
    ABI): the weights' gradients are zeros."""
    import sliding_window_attention_sdpa_gb300 as swa
    p = swa.SdpaRopeParams()
    p.dtype, p.layout, p.interleaved = swa.SDPA_BF16, swa.SDPA_THD if packed else swa.SDPA_BSHD, interleaved
    p.b, p.s, p.total, p.h_q, p.h_kv, p.d, p.rot, p.n_axes = (0, 0, 0, 4, 2, d, d, axes) if packed else (2, 0, 0, 4, 2, d, d, axes)
    p.eps, p.rot_scale = 1e-6, 1.0
    for n, h in (("q", 4), ("k", 2), ("gq", 4), ("gk", 2), ("oq", 4), ("ok", 2)):
        setattr(p, n + "_stride", swa._i64x3(0, h * d, d))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((2, d), math.nan, device="cuda")
    p.q_weight = p.k_weight = w.data_ptr()
    p.dq_weight, p.dk_weight = dw[0].data_ptr(), dw[1].data_ptr()
    n = swa.sdpa_rope_bwd_workspace_bytes(p)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert not p.freq and not p.positions
    assert swa.sdpa_rope_bwd(p, ws.data_ptr(), n, stream) == swa.SDPA_OK, swa.last_error()
    assert swa.sdpa_rope_fwd(p, stream) == swa.SDPA_OK, swa.last_error()
    torch.cuda.synchronize()
    assert (dw == 0).all()
