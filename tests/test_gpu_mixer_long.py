"""Batches whose segments are long or many: the layers around the delta rule far from their shortest segments."""

import pytest
import torch

import gated_deltanet_chunkwise_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU runs, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("B", [1, 1100])
def test_most_tokens_of_one_channel(B):
    """As many tokens as a call takes, in one sequence and in more than one block checks. The first tap alone hands
    on the input before; a decay of nothing and unit B and C hand on the input itself: both exactly."""
    T = (1 << 31) - 1024
    cu = torch.arange(B + 1, device="cuda") * (T // B)
    cu[B] = T
    idx = torch.arange(B, device="cuda").flip(0)
    x = torch.empty(T, 1, dtype=torch.bfloat16, device="cuda").normal_()
    old = torch.randn(B, 1, 1, device="cuda").bfloat16()
    pool = old.clone()
    out = gdn.gdn_conv_extend(x, torch.tensor([[1.0, 0.0]], device="cuda"), None, pool, idx, cu, activation=None, check=True)
    assert torch.equal(out[cu[:-1]], old[idx, 0]) and torch.equal(pool[idx, 0], x[cu[1:] - 1])
    out[cu[:-1]] = x[cu[:-1] - 1]  # (the first sequence's: the last token, as in a roll)
    assert torch.equal(out, x.roll(1, 0))
    one = torch.ones(T, 1, dtype=torch.bfloat16, device="cuda")
    state = torch.ones(B, 1, 1, device="cuda")
    gdn.gdn_ssm_extend(x, one, torch.full((1, 1), -200.0, device="cuda"), one[:, None], one[:, None], None, None, None, state, idx,
                       cu, softplus=False, out=out, check=True)
    assert torch.equal(out, x) and torch.equal(state[idx, 0], x[cu[1:] - 1].float())


def test_longest_row_of_layer_norm():
    """2^30 columns of one value but for two: the mean, the variance and the gradients follow by hand."""
    n = 1 << 30
    x = torch.full((1, n), 2.0, dtype=torch.bfloat16, device="cuda")
    x[0, 5], x[0, n - 1] = 4.0, 0.0                    # mean 2, variance 8 / n
    out, mean, rstd = gdn.gdn_layer_norm(x, eps=1.0, return_stats=True)
    assert float(mean) == 2.0 and float(rstd) == 1.0   # (8 / n is under half a step of 1)
    assert float(out[0, 5]) == 2.0 and float(out[0, n - 1]) == -2.0 and int((out == 0).sum()) == n - 2
    g = gdn.gdn_layer_norm_backward(out, x, None, mean, rstd)  # the output as its own gradient: mean 0, mean of dy xh 8 / n
    assert torch.equal(g.dx, out) and torch.equal(g.dbias, out[0].float())
    assert float(g.dweight[5]) == 4.0 and float(g.dweight[n - 1]) == 4.0 and int((g.dweight == 0).sum()) == n - 2
