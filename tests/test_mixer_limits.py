"""Sizes at the far end of what the calls of the layers around the delta rule take. CPU only."""

from gated_deltanet_chunkwise_gdn_gb300 import _lib
from test_mixer_abi import CONV, SSM, SSM_IN, _by_order

MOST = (1 << 31) - 1024


def test_most_tokens():
    L = _lib.load()
    for f in (L.gdn_conv_workspace_size, L.gdn_conv_backward_workspace_size):
        assert f(MOST, 1, 1, 4) > 0 and f(MOST, 1100, 1, 4) > 0 and f(MOST + 1, 1, 1, 4) == 0
    for f in (L.gdn_ssm_workspace_size, L.gdn_ssm_backward_workspace_size):
        assert f(MOST, 1, 1, 1, 1) > 0 and f(MOST, 1100, 1, 1, 1) > 0 and f(MOST + 1, 1, 1, 1, 1) == 0
    order = "x xs dtype w b pool size idx cu batch out T D W silu ws bytes stream"
    assert _by_order(L.gdn_conv_extend, order, CONV, dict(T=MOST + 1)) == 1
    assert _by_order(L.gdn_ssm_extend, SSM_IN + "cu batch out T Dm G N sp ws bytes stream", SSM, dict(T=MOST + 1)) == 1
