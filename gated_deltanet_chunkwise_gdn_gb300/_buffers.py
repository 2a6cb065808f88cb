"""The workspaces and status words that the Python calls keep between them."""

from __future__ import annotations

import contextlib
import threading

import torch

_workspaces: dict = {}
_locks: dict = {}
_words: dict = {}

UNSHARED = contextlib.nullcontext()  # in the place of a lock, for a workspace that is one call's alone


def kept_workspace(device: torch.device, stream: torch.cuda.Stream, nbytes: int) -> torch.Tensor:
    """The kept workspace of (device, stream), with room for `nbytes` at a 256-byte boundary.

    One buffer per stream: calls on one stream are ordered, so they may share it, while calls
    on two streams of a device run concurrently and must not. The buffer is allocated on the
    call's stream, so when it is replaced by a larger one, the caching allocator reuses the old
    memory only in that stream's order, after the calls already enqueued there.
    """
    key = (device.index, stream.cuda_stream)
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes + 256:
        with workspace_lock(device, stream.cuda_stream):
            buf = _workspaces.get(key)
            if buf is None or buf.numel() < nbytes + 256:
                with torch.cuda.stream(stream):
                    buf = torch.empty(max(nbytes, 256) + 256, dtype=torch.uint8, device=device)
                _workspaces[key] = buf
    return buf


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


def status_word(device: torch.device, handle: int) -> torch.Tensor:
    """The status word of this thread's single-token steps on (device, stream).

    A step may read the word before it writes the pool (its slots' verdict, from a kernel before), so no step
    that can run, or be enqueued, at the same time may have the same one.
    """
    key = (device.index, handle, threading.get_ident())
    word = _words.get(key)
    if word is None:
        word = _words[key] = torch.zeros(64, dtype=torch.int32, device=device)
    return word


def aligned_ptr(buf: torch.Tensor) -> int:
    return (buf.data_ptr() + 255) & ~255
