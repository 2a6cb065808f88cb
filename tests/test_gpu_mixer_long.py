"""Batches whose segments are long or many: the layers around the delta rule far from their shortest segments."""

import numpy as np
import pytest
import torch

import gated_deltanet_chunkwise_gdn_gb300 as gdn
from gated_deltanet_chunkwise_gdn_gb300 import GdnError
from oracle import mixer

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU runs, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_mixer import BF16, FP16, FP32, SSM_KEYS, check, check_ssm, conv_inputs, cuda, ssm_inputs  # noqa: E402


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


# ----------------------------------------------------------------------------- long segments, many sequences


def check_conv(lengths, D, W, dtype, pad=0, silu=True):
    d = conv_inputs(lengths, D, W, dtype, seed=D + W, pad=pad)
    g = cuda(d)
    act, T = "silu" if silu else None, int(d["cu"][-1])
    val, size = mixer.conv(d["x"], d["weight"], d["bias"], d["pool"], d["idx"], d["cu"], silu, d["d_out"], d["d_state"])
    pool = g["pool"].clone()
    out = gdn.gdn_conv_extend(g["x"], g["weight"], g["bias"], pool, g["idx"], g["cu"], activation=act, check=True)
    check("out", out, val["out"], size["out"], 2.0 ** -19)
    assert torch.equal(pool.cpu().double(), torch.from_numpy(val["pool"]))
    gr = gdn.gdn_conv_backward(g["x"], g["weight"], g["bias"], g["pool"], g["idx"], g["cu"], g["d_out"], g["d_state"],
                               activation=act, check=True)
    check("dx", gr.dx, val["dx"], size["dx"], 2.0 ** -19)
    check("d_pool", gr.d_state_pool, val["d_pool"], size["d_pool"], 2.0 ** -19)
    check("dweight", gr.dweight, val["dweight"], size["dweight"], (T + 32) * 2.0 ** -23)
    check("dbias", gr.dbias, val["dbias"], size["dbias"], (T + 32) * 2.0 ** -23)


def crowd(B, most):
    """B short sequences, empty ones among them, and a long one in between."""
    return [(i * 7) % 4 for i in range(B // 2)] + [most] + [(i * 5) % 3 for i in range(B - B // 2 - 1)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N,channels,G,pad", [(16, 4, 80, 0), (16, 2, 160, 0), (16, 1, 304, 0), (8, 4, 80, 0), (8, 3, 101, 1),
                                              (24, 2, 160, 0), (32, 4, 80, 0), (32, 1, 160, 1), (64, 2, 160, 0), (21, 4, 80, 0)])
def test_ssm_long_segments(dtype, N, channels, G, pad):
    """So many groups that the card is full with few segments: each is hundreds of tokens long, many tiles and chunks."""
    check_ssm(ssm_inputs([700, 0, 333, 1], channels * G, N, G, dtype, seed=N + G, pad=pad))


@pytest.mark.parametrize("dtype,N,Dm,pad", [(BF16, 16, 32, 0), (FP32, 16, 6, 0), (FP16, 8, 7, 1), (BF16, 33, 8, 0)])
@pytest.mark.parametrize("B", [1025, 2500])
def test_ssm_of_many_sequences(B, dtype, N, Dm, pad):
    """More sequences than one block checks, a long one among them, which is not cut."""
    check_ssm(ssm_inputs(crowd(B, 500), Dm, N, 1, dtype, seed=B, pad=pad))


@pytest.mark.parametrize("B", [33, 500, 1024])
def test_ssm_of_a_block_of_sequences(B):
    check_ssm(ssm_inputs(crowd(B, 300), 20, 16, 2, BF16, seed=B))


@pytest.mark.parametrize("dtype,W,D,pad", [(BF16, 4, 64, 0), (FP16, 3, 6, 0), (FP32, 2, 12, 0), (BF16, 4, 7, 1)])
@pytest.mark.parametrize("B", [33, 500, 1024, 1025, 2500])
def test_conv_of_many_sequences_and_a_long_one(B, dtype, W, D, pad):
    check_conv(crowd(B, 500), D, W, dtype, pad=pad)


@pytest.mark.parametrize("dtype,D", [(BF16, 4), (FP32, 3)])
def test_conv_segments_of_the_device_s_choice(dtype, D):
    """Tokens enough that the even share of the segments is longer than the shortest segment, in the backward pass."""
    check_conv([9000, 0, 17, 6001], D, 4, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_conv_forward_segments_of_the_device_s_choice(dtype):
    """The same in the forward pass, against the sum over shifted rows in 64 bits."""
    lengths, D, W = [70001, 3, 0, 9000], 2, 4
    d = conv_inputs(lengths, D, W, dtype, seed=1)
    g = cuda(d)
    out = gdn.gdn_conv_extend(g["x"], g["weight"], g["bias"], g["pool"], g["idx"], g["cu"], activation=None, check=True)
    x, w = mixer.f64(d["x"]), mixer.f64(d["weight"])
    for s, slot in enumerate(d["idx"].tolist()):
        t0, t1 = int(d["cu"][s]), int(d["cu"][s + 1])
        line = np.concatenate([mixer.f64(d["pool"][slot]), x[t0:t1]])
        terms = [w[:, j] * line[j:j + t1 - t0] for j in range(W)] + [mixer.f64(d["bias"])]
        check("out", out[t0:t1], sum(terms), sum(np.abs(t) for t in terms), 2.0 ** -19)
        assert torch.equal(g["pool"][slot].cpu().double(), torch.from_numpy(line[t1 - t0:]))


@pytest.mark.parametrize("B", [33, 500, 1024, 1025, 2500])
@pytest.mark.parametrize("fault", ["repeated", "next to it", "high", "low", "order"])
def test_bad_batches_of_many_sequences_touch_nothing(B, fault):
    """Faults past the first warp's share of the batch."""
    lengths = crowd(B, 20)
    d, c = ssm_inputs(lengths, 8, 16, 1, BF16, seed=B), conv_inputs(lengths, 8, 4, BF16, seed=B)
    idx, cu, status = d["idx"].clone(), d["cu"].clone(), 3
    if fault == "order":
        cu[B - 1], status = cu[B] + 1, 7
    else:
        idx[B - 1] = {"repeated": idx[0], "next to it": idx[B - 2], "high": d["pool"].shape[0], "low": -1}[fault]
    g, h, idx, cu = cuda(d), cuda(c), idx.cuda(), cu.cuda()
    par, cpar = [g[n] for n in SSM_KEYS[:8]], [h["x"], h["weight"], h["bias"]]
    out, cout = torch.full_like(g["x"], 5.0), torch.full_like(h["x"], 5.0)
    for call in (lambda: gdn.gdn_ssm_extend(*par, g["pool"], idx, cu, out=out, check=True),
                 lambda: gdn.gdn_conv_extend(*cpar, h["pool"], idx, cu, out=cout, check=True),
                 lambda: gdn.gdn_ssm_backward(*par, g["pool"], idx, cu, g["d_out"], g["d_state"], check=True),
                 lambda: gdn.gdn_conv_backward(*cpar, h["pool"], idx, cu, h["d_out"], h["d_state"], check=True)):
        with pytest.raises(GdnError) as e:
            call()
        assert e.value.status == status
    assert torch.equal(g["pool"].cpu(), d["pool"]) and torch.equal(h["pool"].cpu(), c["pool"])
    assert (out == 5).all() and (cout == 5).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,n", [(5000, 64), (5000, 512), (3000, 1000), (2000, 4096), (700, 8192), (900, 1538), (2000, 35)])
def test_layer_norm_of_many_rows(dtype, rows, n):
    """Rows enough that every block takes several: its loads ahead and its parameter sums go round more than once."""
    gen = torch.Generator().manual_seed(n)
    x, d_out = ((torch.randn(rows, n, generator=gen) * 2 + 1).to(dtype) for _ in "xd")
    w, b = 1 + 0.2 * torch.randn(n, generator=gen), torch.randn(n, generator=gen)
    val, size = mixer.layer_norm(x, w, b, 1e-5, d_out)
    out, mean, rstd = gdn.gdn_layer_norm(x.cuda(), w.cuda(), b.cuda(), return_stats=True)
    g = gdn.gdn_layer_norm_backward(d_out.cuda(), x.cuda(), w.cuda(), mean, rstd)
    k = 2.0 ** -19
    for name, got in (("out", out), ("mean", mean), ("rstd", rstd), ("dx", g.dx)):
        check(name, got, val[name], size[name], k)
    for name, got in (("dweight", g.dweight), ("dbias", g.dbias)):
        check(name, got, val[name], size[name], (rows + 32) * 2.0 ** -23 + k)
