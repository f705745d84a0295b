"""Host-only checks of the operators around the mixer at unusual arguments."""
import pytest
import torch

from rank_latent_routing_flare_b200 import Status

from .test_attention_host import bwd, fwd


@pytest.mark.parametrize("call", [fwd, bwd])
def test_scales_that_fp32_does_not_hold(call):
    """1e-60 would round to 0, which stands for 1 / sqrt(D); 1e39 to infinity."""
    for scale in (1e-60, 1e-46, 1e-31, 1e31, 1e39, 1e300):
        assert call(scale=scale) == Status.ERR_UNSUPPORTED, scale
    if torch.cuda.is_available():
        return                                    # the pointers are not real
    for scale in (0.0, -1.0, 1e-30, 0.1, 1e30):
        assert call(scale=scale) not in (Status.ERR_UNSUPPORTED, Status.ERR_SHAPE), scale
