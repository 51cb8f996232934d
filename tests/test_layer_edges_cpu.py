"""Refusals of the state space layer's calls at the ends of their ranges, before any CUDA call."""
import pytest

import gated_deltanet_recurrence_gb300 as gdn
from tests.test_layer_cpu import ARG, CONV, CONVB

MOST = 2 ** 31 - 1 - 2048  # tokens of a convolution: runs and the rows asked for ahead are counted in 32 bits


@pytest.mark.parametrize("tokens", [MOST + 1, 2 ** 31 - 16, 2 ** 31 - 1])
def test_convolutions_whose_counters_would_wrap_are_refused(tokens):
    L = gdn.lib()
    assert L.gdn_short_conv_fwd(*dict(CONV, T=tokens, dim=8, xs=8).values()) == ARG
    assert L.gdn_short_conv_bwd(*dict(CONVB, T=tokens, dim=8, xs=8).values()) == ARG
    assert L.gdn_short_conv_bwd_workspace_size(1, tokens, 8) == 0
    assert L.gdn_short_conv_bwd_workspace_size(1, MOST, 8) > 0
