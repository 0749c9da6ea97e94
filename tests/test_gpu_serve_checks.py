"""Refusals and flags of the calls around the layer that need a GPU to be seen."""
import pytest
import torch

import any_precision_expert_gb300 as pw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream,error", [("no stream", AttributeError), (1 << 70, OverflowError),
                                          (type("S", (), {"cuda_stream": "x"})(), TypeError)])
def test_an_argument_that_is_no_stream_enqueues_nothing(stream, error):
    q = torch.ones(3, 4, 64, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 7.0)
    with pytest.raises(error):
        pw.qk_norm_rope(pw.Rotary(None), q, None, None, out, None, stream=stream)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
