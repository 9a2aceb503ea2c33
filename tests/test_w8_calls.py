"""Calls of the 8-bit binding that are refused or answered before any device is needed."""
import pytest
import torch

import weight_quantization_codec_amd as q


def test_the_residual_stream_keeps_its_history():
    """h of rmsnorm8 would carry a residual stream on, without its history: where h is not x itself, x or a residual
    that requires a gradient is refused while gradients are recorded, and only then."""
    x, r = torch.zeros((4, 64)), torch.zeros((4, 64))
    with pytest.raises(ValueError, match="device"):
        q.rmsnorm8(x.clone().requires_grad_())   # h is x, with its history
    for kw in (dict(x=x, residual=r.clone().requires_grad_()), dict(x=x.clone().requires_grad_(), residual=r),
               dict(x=(2 * x.clone().requires_grad_()), residual=r), dict(x=x.clone().requires_grad_(), sum_out=r)):
        with pytest.raises(ValueError, match="gradient"):
            q.rmsnorm8(**kw)
        with torch.no_grad(), pytest.raises(ValueError, match="device"):
            q.rmsnorm8(**kw)
        kw = {k: v.detach() for k, v in kw.items()}
        with pytest.raises(ValueError, match="device"):
            q.rmsnorm8(weight=torch.ones(64, requires_grad=True), **kw)   # a parameter: no output carries it on


def test_workspace_of_sizes_past_32_bits():
    """Sizes that gemm8 refuses need no workspace; none is taken for another that it equals in 32 bits."""
    need = q.gemm8_workspace(77, 4096, 11008)
    assert need > 0
    for past in (2**32, -2**32, 2**31, 2**63, 2**64):
        assert q.gemm8_workspace(past + 77, 4096, 11008) == 0
        assert q.gemm8_workspace(77, past + 4096, 11008) == 0
        assert q.gemm8_workspace(77, 4096, past + 11008) == 0
    assert q.gemm8_workspace(77, 4096, 11008) == need
