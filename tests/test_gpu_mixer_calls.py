"""The calls of the layers around the delta rule from several host threads and streams, and captured in graphs."""

import threading

import pytest
import torch

import gated_deltanet_chunkwise_gdn_gb300 as gdn
from gated_deltanet_chunkwise_gdn_gb300 import _lib

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU runs, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def prompt(lengths, D=64, N=16, seed=0):
    """The arguments of a convolution and of a scan over one packed batch, with pools of their own."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    T, B = sum(lengths), len(lengths)
    cu = torch.tensor([0] + list(lengths), device="cuda").cumsum(0)
    idx = torch.randperm(B, generator=gen, device="cuda")
    x, bc = r(T, D).bfloat16(), r(T, 1, N).bfloat16()
    conv = (x, r(D, 4), r(D), r(B, 3, D).bfloat16(), idx, cu)
    scan = (x, x, -torch.rand(D, N, generator=gen, device="cuda"), bc, bc, r(D), x, r(D), r(B, D, N), idx, cu)
    return conv, scan


def outputs(conv, scan, stream=None):
    """Every call that keeps a workspace, on copies of the pools."""
    conv, scan = list(conv), list(scan)
    g = gdn.gdn_conv_backward(*conv, conv[0], stream=stream)
    conv[3], scan[8] = conv[3].clone(), scan[8].clone()
    return [gdn.gdn_conv_extend(*conv, stream=stream), conv[3], gdn.gdn_ssm_extend(*scan, stream=stream), scan[8], *g]


def in_threads(*jobs):
    errors = []

    def run(job):
        try:
            job()
        except BaseException as e:  # shown by the test, not by the thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_threads_on_one_stream():
    """Two threads issue calls of other batches on one stream: each gets its own batch's results."""
    batches = [prompt([700, 3, 41], seed=1), prompt([5, 1, 9, 0, 260, 2, 30], D=96, seed=2)]
    want = [outputs(*b) for b in batches]
    torch.cuda.synchronize()

    def job(i):
        for _ in range(30):
            got = outputs(*batches[i])
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    in_threads(*[lambda i=i: job(i) for i in (0, 1, 0, 1)])


def test_two_streams_at_once():
    batches = [prompt([700, 3, 41], seed=3), prompt([5, 1, 9, 0, 260, 2, 30], D=96, seed=4)]
    want = [outputs(*b) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = []
    for _ in range(20):
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                got.append(outputs(*b))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("N", [16, 5])
def test_steps_on_two_streams_keep_their_verdicts(N):
    """A good and a bad batch of steps side by side, both checked by a kernel before: the bad one touches nothing."""
    B, D = 600, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, bc, A = r(B, D), r(B, 1, N), -torch.rand(D, N, generator=gen, device="cuda")
    good = torch.randperm(2 * B, generator=gen, device="cuda")[:B]
    bad = good.clone()
    bad[B - 1] = bad[0]
    start = r(2 * B, D, N)
    pools, streams = [start.clone(), start.clone()], [torch.cuda.Stream(), torch.cuda.Stream()]
    step = lambda pool, idx: gdn.gdn_ssm_step(x, x, A, bc, bc, None, None, None, pool, idx)  # noqa: E731
    alone = start.clone()
    want = [step(alone, good) for _ in range(20)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            got.append(step(pools[0], good))
        with torch.cuda.stream(streams[1]):
            step(pools[1], bad)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(pools[0], alone)
    assert torch.equal(pools[1], start)


def test_threads_norm_rows_of_several_lengths():
    """Lengths that run on one kernel with other amounts of shared memory, all above what needs to be allowed. The
    library is called as closely as the interpreter can, so that calls fall between each other's host steps."""
    xs = [torch.randn(3, n, device="cuda").bfloat16() for n in (7168, 8192, 12288, 16384)]
    want = [gdn.gdn_layer_norm(x) for x in xs]
    outs = [torch.empty_like(x) for x in xs]
    norm, code = _lib.load().gdn_layer_norm, _lib.GDN_BF16
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]

    def job(i):
        x, n = xs[i], xs[i].shape[1]
        args = (x.data_ptr(), n, code, None, None, outs[i].data_ptr(), None, None, 3, n, 1e-5, streams[i].cuda_stream)
        status = {norm(*args) for _ in range(20000)}
        assert status == {0}, status
    in_threads(*[lambda i=i: job(i) for i in range(len(xs))])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_graphs_beside_calls_on_their_stream():
    """Two graphs captured on one stream after its workspace is made, replayed side by side on others, with larger calls
    on that stream in between, whose workspace replaces the one before."""
    batches = [prompt([300, 7, 41], seed=6), prompt([5, 1, 9, 0, 260, 2, 30], D=96, seed=7)]
    large = prompt([9000] + [5] * 700, seed=8)
    want = [outputs(*b) for b in batches]
    want_large = outputs(*large)
    main = torch.cuda.Stream()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        outputs(*batches[0])
    main.synchronize()
    graphs, results = [], []
    for b in batches:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=main):
            results.append(outputs(*b))
    for _ in range(10):
        for t in [t for r in results for t in r]:
            t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(main):
            got = outputs(*large)
            spare = [torch.full((1 << 18,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        for r, w in zip(results + [got], want + [want_large]):
            assert all(torch.equal(a, b) for a, b in zip(r, w))
        assert all(bool((t == 7).all()) for t in spare)


def test_a_replayed_step_reports_to_a_given_word():
    B, D = 400, 64
    x, w, pool = torch.randn(B, D, device="cuda"), torch.randn(D, 4, device="cuda"), torch.randn(B, 3, D, device="cuda")
    idx, word = torch.arange(B, device="cuda"), torch.full((1,), -1, dtype=torch.int32, device="cuda")
    gdn.gdn_conv_step(x, w, None, pool.clone(), idx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_conv_step(x, w, None, pool, idx, status=word)
    graph.replay()
    assert int(word) == 0
    before = pool.clone()
    idx[3] = idx[2]
    graph.replay()
    assert int(word) == 3 and torch.equal(pool, before)


def test_a_gradient_penalty_is_refused():
    x = torch.randn(5, 64, device="cuda", requires_grad=True)
    out = gdn.LayerNorm.apply(x, None, None)
    g, = torch.autograd.grad(out.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (out.sum() + g.square().sum()).backward()
