"""Sizes at the far end of what the calls of the layers around the delta rule take. CPU only."""

from gated_deltanet_chunkwise_gdn_gb300 import _lib
from test_mixer_abi import CONV, NORM, SSM, SSM_IN, _by_order

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


def test_most_columns():
    L, most = _lib.load(), 1 << 30
    size = L.gdn_layer_norm_backward_workspace_size
    assert size(2, most) > 0
    for n in (most + 1, (1 << 31) - 8, (1 << 31) - 1):
        over = dict(n=n, xs=n, ds=n)
        assert size(2, n) == 0
        assert _by_order(L.gdn_layer_norm, "x xs dtype w b out mean rstd rows n eps stream", NORM, dict(over, rows=0)) == 2
        assert _by_order(L.gdn_layer_norm_backward, "dy ds x xs dtype w mean rstd dx dw db rows n ws bytes stream", NORM,
                         dict(over, rows=0)) == 2
