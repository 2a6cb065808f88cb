"""The workspaces and status words that the Python calls keep between them."""

from __future__ import annotations

import contextlib
import threading

import torch

_workspaces: dict = {}
_locks: dict = {}
_words: dict = {}

UNSHARED = contextlib.nullcontext()  # in the place of a lock, for a workspace that is one call's alone


# What a call needs of CUDA on its way costs the host tenths of a microsecond a question, so the questions go straight
# to the binding where it has them.
current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def require_current(device: torch.device) -> None:
    """The library launches on the thread's current device: the inputs' has to be that one."""
    if current_device() != device.index:
        raise ValueError(f"the inputs are on {device}, but the current device is cuda:{current_device()}: make the call "
                         f"under torch.cuda.device({device.index})")


def _capturing(stream, handle: int) -> bool:
    """Whether a graph is being captured on the stream (None: the current one) of this handle. The default stream's is
    0, and it takes no part in captures: calls there are spared the question."""
    if handle == 0:
        return False
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _new(n: int, dtype, device: torch.device, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(n, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=dtype, device=device)


def workspace_for(device: torch.device, stream, handle: int, nbytes: int):
    """(workspace, lock to hold while the call is enqueued) of a call on the stream (None: the current one) of this
    handle, with room for `nbytes` at a 256-byte boundary.

    One kept buffer per stream: calls on one stream are ordered, so they may share it, while calls
    on two streams of a device run concurrently and must not. The buffer is allocated on the
    call's stream, so when it is replaced by a larger one, the caching allocator reuses the old
    memory only in that stream's order, after the calls already enqueued there.

    A call that is captured into a graph gets a buffer of its own instead, from the graph's memory: the graph may be
    replayed on any stream, beside calls on the stream that it was captured on and beside other graphs
    captured there, and after a larger call has replaced the kept buffer.
    """
    if _capturing(stream, handle):
        return _new(nbytes + 256, torch.uint8, device, stream), UNSHARED
    key = (device.index, handle)
    lock = workspace_lock(device, handle)
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes + 256:
        with lock:
            buf = _workspaces.get(key)
            if buf is None or buf.numel() < nbytes + 256:
                buf = _workspaces[key] = _new(max(nbytes, 256) + 256, torch.uint8, device, stream)
    return buf, lock


def given_workspace(workspace, device: torch.device):
    """(address, bytes) of a caller's workspace."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def workspace_of(device_index, handle: int):
    """The kept workspace of (device, stream) or None."""
    return _workspaces.get((device_index, handle))


def workspace_lock(device: torch.device, handle: int):
    """The lock of the kept workspace of (device, stream).

    A call enqueues several kernels that hand their results on through the workspace, and the interpreter lets
    other threads run meanwhile. The call holds this lock from its first kernel to its last (and, where it waits
    for its verdict, until it has read it), so that another thread's call on the same stream comes before or
    after all of them and never writes the workspace in between.
    """
    key = (device.index, handle)
    lock = _locks.get(key)
    return lock if lock is not None else _locks.setdefault(key, threading.RLock())


def status_word(device: torch.device, stream, handle: int) -> torch.Tensor:
    """The status word of this thread's single-token steps on the stream (None: the current one) of this handle.

    A step may read the word before it writes the pool (its slots' verdict, from a kernel before), so no step
    that can run, or be enqueued, at the same time may have the same one; a step that is captured into a graph
    has one of the graph's own, as a workspace would be. Every step writes the word before it reads it.
    """
    if _capturing(stream, handle):
        return _new(1, torch.int32, device, stream)
    key = (device.index, handle, threading.get_ident())
    word = _words.get(key)
    if word is None:
        word = _words[key] = _new(1, torch.int32, device, stream)
    return word


def aligned_ptr(buf: torch.Tensor) -> int:
    return (buf.data_ptr() + 255) & ~255
