"""What the Python calls do on the host around the library's: workspaces, threads, streams and devices. CPU only: the
tensors say that they are on a GPU, and the library is a record of the calls made to it."""

import threading
import time
from types import SimpleNamespace

import pytest
import torch

import gated_deltanet_chunkwise_gdn_gb300 as gdn
from gated_deltanet_chunkwise_gdn_gb300 import _buffers, _lib, mixer


class OnGpu(torch.Tensor):
    """A host tensor that says it is on cuda:0."""
    device = property(lambda self: torch.device("cuda", 0))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


_zeros = torch.zeros


def on_gpu(*shape, dtype=torch.float32, device=None):
    return _zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    """Stands in for the library: each call takes a while and is recorded by its workspace's or status word's address."""

    def __init__(self):
        self.inside, self.overlaps, self.calls, self.lock = {}, 0, [], threading.Lock()

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 1024
        if name == "gdn_get_device_status":
            return lambda word, handle: 0

        def call(*args):
            key = args[-3] if args[-3] and args[-3] > 1 << 16 else args[-2]
            with self.lock:
                self.overlaps += self.inside.get(key, 0)
                self.inside[key] = self.inside.get(key, 0) + 1
                self.calls.append((name, key, args[-1]))
            time.sleep(0.02)
            with self.lock:
                self.inside[key] -= 1
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(_lib, "load", lambda *a: lib)
    for new in ("empty", "zeros"):  # a new tensor "on the GPU"
        monkeypatch.setattr(torch, new, on_gpu)
    lib.capturing = False
    lib.device = 0
    for module in (_buffers, mixer):
        monkeypatch.setattr(module, "current_device", lambda: lib.device)
    monkeypatch.setattr(torch, "zeros_like", lambda t: on_gpu(*t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: lib.capturing)
    for cache in ("_workspaces", "_locks", "_words"):
        monkeypatch.setattr(_buffers, cache, {})
    return lib


STREAM, OTHER = SimpleNamespace(cuda_stream=1 << 20), SimpleNamespace(cuda_stream=2 << 20)


def calls():
    """Every public call, on tensors of one sequence of two tokens."""
    idx, cu = on_gpu(1, dtype=torch.int64), on_gpu(2, dtype=torch.int64)
    x, w, pool = on_gpu(2, 8), on_gpu(8, 4), on_gpu(1, 3, 8)
    A, bc, state = on_gpu(8, 4), on_gpu(2, 1, 4), on_gpu(1, 8, 4)
    q, a, par, states = on_gpu(2, 1, 64, dtype=torch.bfloat16), on_gpu(2, 1), on_gpu(1), on_gpu(1, 1, 64, 64)
    out = on_gpu(2, 1, 64, dtype=torch.bfloat16)
    two, pool2, state2 = on_gpu(2, dtype=torch.int64), on_gpu(2, 3, 8), on_gpu(2, 8, 4)
    ssm = (x, x, A, bc, bc, None, None, None)
    return dict(
        extend=lambda **k: gdn.gdn_extend_chunkwise(q, q, q, a, a, par, par, states, idx, cu, out=out, **k),
        backward=lambda **k: gdn.gdn_chunkwise_backward(q, q, q, a, a, par, par, states, idx, cu, q, **k),
        decode=lambda **k: gdn.gdn_decode_step(q, q, q, a, a, par, par, states, two, out=out, **k),
        conv_extend=lambda **k: gdn.gdn_conv_extend(x, w, None, pool, idx, cu, **k),
        conv_step=lambda **k: gdn.gdn_conv_step(x, w, None, pool2, two, **k),
        conv_backward=lambda **k: gdn.gdn_conv_backward(x, w, None, pool, idx, cu, x, **k),
        ssm_extend=lambda **k: gdn.gdn_ssm_extend(*ssm, state, idx, cu, **k),
        ssm_step=lambda **k: gdn.gdn_ssm_step(*ssm, state2, two, **k),
        ssm_backward=lambda **k: gdn.gdn_ssm_backward(*ssm, state, idx, cu, x, **k),
        norm=lambda **k: gdn.gdn_layer_norm(x, **k),
        norm_backward=lambda **k: gdn.gdn_layer_norm_backward(x, x, None, on_gpu(2), on_gpu(2), **k))


def in_threads(*jobs):
    threads = [threading.Thread(target=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


KEPT = ("extend", "conv_extend", "conv_backward", "ssm_extend")


@pytest.mark.parametrize("name", KEPT)
@pytest.mark.parametrize("other", KEPT)
def test_threads_on_one_stream_take_turns_on_its_workspace(library, name, other):
    """A call's kernels are enqueued together: another thread's call on the stream would overwrite what they share."""
    c = calls()
    in_threads(*[lambda n=n: c[n](stream=STREAM) for n in (name, other, name)])
    assert len(library.calls) == 3 and len({key for _, key, _ in library.calls}) == 1
    assert library.overlaps == 0


STEPS = ("decode", "conv_step", "ssm_step")


@pytest.mark.parametrize("name", STEPS)
def test_steps_of_other_streams_and_threads_have_words_of_their_own(library, name):
    """A step's update may go by the verdict in the status word, so a step beside it must not write there."""
    step = calls()[name]
    for stream in (STREAM, STREAM, OTHER, OTHER):
        step(stream=stream)
    in_threads(lambda: step(stream=STREAM))
    words = [key for _, key, _ in library.calls]
    assert words[0] == words[1] and words[2] == words[3] and len({words[0], words[2], words[4]}) == 3


@pytest.mark.parametrize("name", STEPS)
def test_a_given_status_word_is_used(library, name):
    word = on_gpu(1, dtype=torch.int32)
    calls()[name](stream=STREAM, status=word)
    assert library.calls[0][1] == word.data_ptr()


def test_streams_do_not_wait_for_each_other(library):
    c = calls()
    c["conv_extend"](stream=STREAM), c["conv_extend"](stream=OTHER)
    with _buffers.workspace_lock(torch.device("cuda", 0), STREAM.cuda_stream):
        t = threading.Thread(target=lambda: c["conv_extend"](stream=OTHER))
        t.start()
        t.join(5)
        assert not t.is_alive()
    assert len({key for _, key, _ in library.calls}) == 2


@pytest.mark.parametrize("name", KEPT + STEPS)
def test_captured_calls_have_buffers_of_their_own(library, name):
    """A graph is replayed beside calls on the stream it was captured on, and after their buffer has grown."""
    call, kept = calls()[name], []
    call(stream=STREAM)
    library.capturing = True
    empty = torch.empty

    def keep(*a, **k):  # so that no two of them can have the same address by turns
        kept.append(empty(*a, **k))
        return kept[-1]
    torch.empty = keep
    try:
        call(stream=STREAM), call(stream=STREAM)
    finally:
        torch.empty = empty
    library.capturing = False
    call(stream=STREAM)
    at = [key for _, key, _ in library.calls]
    assert at[0] == at[3] and len(set(at)) == 3


@pytest.mark.parametrize("name", KEPT + ("ssm_backward", "norm_backward", "backward"))
def test_a_workspace_elsewhere_is_refused(library, name):
    """The kernels write there: host memory, gaps and other objects never reach the library."""
    call = calls()[name]
    room = on_gpu(8192, dtype=torch.uint8)
    for bad, error in ((_zeros(8192, dtype=torch.uint8), ValueError), (room[::2], ValueError), (room.data_ptr(), TypeError)):
        with pytest.raises(error, match="workspace"):
            call(stream=STREAM, workspace=bad)
    assert not library.calls
    call(stream=STREAM, workspace=room)
    assert library.calls[0][1] == room.data_ptr()


@pytest.mark.parametrize("name", ["extend", "backward", "decode", "conv_extend", "conv_step", "conv_backward", "ssm_extend", "ssm_step",
                                  "ssm_backward", "norm", "norm_backward"])
def test_inputs_off_the_current_device_are_refused(library, name):
    """The kernels would run on the current device with the other one's addresses."""
    library.device = 1
    with pytest.raises(ValueError, match="current device is cuda:1"):
        calls()[name](stream=STREAM)
    assert not library.calls
    library.device = 0
    calls()[name](stream=STREAM)
    assert len(library.calls) == 1


def _functions():
    """The autograd functions with the leaves of a small call."""
    leaf = lambda *shape: torch.ones(*shape, requires_grad=True)  # noqa: E731
    cu, q = torch.tensor([0, 2]), lambda: leaf(2, 1, 4)  # noqa: E731
    return dict(conv=(mixer.CausalConv, (leaf(2, 8), leaf(8, 4), leaf(8), leaf(1, 3, 8), cu)),
                ssm=(mixer.SelectiveScan, (leaf(2, 8), leaf(2, 8), leaf(8, 4), leaf(2, 1, 4), leaf(2, 1, 4), leaf(8), leaf(2, 8),
                                           leaf(8), leaf(1, 8, 4), cu)),
                norm=(mixer.LayerNorm, (leaf(2, 8), leaf(8), leaf(8))),
                delta=(gdn.GatedDeltaNetChunkwise, (q(), q(), q(), leaf(2, 1), leaf(2, 1), leaf(1), leaf(1), leaf(1, 1, 4, 4), cu)))


@pytest.mark.parametrize("name", ["conv", "ssm", "norm", "delta"])
def test_second_derivatives_are_refused(monkeypatch, name):
    """The gradients come from kernels: a loss on them would miss its part in silence."""
    zeros = lambda *ts: [torch.zeros_like(t) for t in ts]  # noqa: E731
    monkeypatch.setattr(mixer, "gdn_conv_extend", lambda x, *a, **k: x * 2)
    monkeypatch.setattr(mixer, "gdn_conv_backward", lambda x, w, b, p, *a, **k: gdn.GdnConvGrads(*zeros(x, w, b, p)))
    monkeypatch.setattr(mixer, "gdn_ssm_extend", lambda x, *a, **k: x * 2)
    monkeypatch.setattr(mixer, "gdn_ssm_backward", lambda *a, **k: gdn.GdnSsmGrads(*zeros(*a[:9])))
    monkeypatch.setattr(mixer, "gdn_layer_norm", lambda x, *a, **k: (x * 2, x[:, 0], x[:, 0]))
    monkeypatch.setattr(mixer, "gdn_layer_norm_backward", lambda d, x, w, *a, **k: gdn.GdnNormGrads(*zeros(x, w, w)))
    monkeypatch.setattr(gdn, "gdn_extend_chunkwise", lambda q, *a, **k: q * 2)
    monkeypatch.setattr(gdn, "gdn_chunkwise_backward", lambda *a, **k: gdn.GdnGrads(*zeros(*a[:8])))
    fn, leaves = _functions()[name]
    out = fn.apply(*leaves)
    out = out[0] if isinstance(out, tuple) else out
    g, = torch.autograd.grad((out * out).sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (out.sum() + g.square().sum()).backward()
    out = fn.apply(*leaves)
    (out[0] if isinstance(out, tuple) else out).sum().backward()
    assert all(t.grad is not None for t in leaves if t.requires_grad)
