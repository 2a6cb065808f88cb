"""The layers around the delta rule in a recurrent mixer block: the short causal convolution, the selective
state space scan and layer norm, for packed prompts, single tokens and training.

Argument marshalling for the C ABI of include/gdn.h, which states the formulas; every step runs in the
library's CUDA kernels. Packed batches, state pools, slots, streams and errors are as for
``gdn_extend_chunkwise``. Activations are bf16, fp16 or fp32 with dense rows; a row stride is allowed, so
they may be column slices of wider projections. Parameters and the scan's states are fp32.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._buffers import UNSHARED, aligned_ptr, current_device, given_workspace, require_current, status_word, workspace_for
from ._lib import GdnError

_DTYPE_CODE = {torch.bfloat16: _lib.GDN_BF16, torch.float16: _lib.GDN_FP16, torch.float32: _lib.GDN_FP32}


# ----------------------------------------------------------------------------- arguments


# A single-token step runs for a few microseconds on the GPU, so what the host spends per argument counts. The
# calls first ask in one expression whether every argument is as it should be, and only where that fails go
# over them one by one (_rows, _dense) for the fault, or for a rarer layout that is fine.


def _refuse(t, name, dtype, dev, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name, dtype, dev, shape) -> int:
    """Checks an activation of `shape` with dense rows; returns its row stride in elements."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev:
        st = t.stride()
        if len(shape) == 2:
            if st[1] == 1 and st[0] >= shape[1] and shape[0] > 1:
                return st[0]
            width, dense = shape[1], st[1] == 1 or shape[1] == 1
        else:
            width = shape[1] * shape[2]
            dense = (st[2] == 1 or shape[2] == 1) and (st[1] == shape[2] or shape[1] == 1)
        if dense and shape[0] <= 1:  # a single row has no stride of its own
            return width
        if dense and st[0] >= width:
            return st[0]
        raise ValueError(f"{name} must have dense rows that do not overlap")
    _refuse(t, name, dtype, dev, shape)


def _dense(t, name, dtype, dev, shape):
    """Checks a dense tensor; returns its address."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev:
        if t.is_contiguous():
            return t.data_ptr()
        raise ValueError(f"{name} must be contiguous")
    _refuse(t, name, dtype, dev, shape)


def _opt(t, name, dtype, dev, shape):
    return None if t is None else _dense(t, name, dtype, dev, shape)


def _activation(t, name, dims):
    """Device and dtype of the activation that the other arguments follow."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev, dtype = t.device, t.dtype
    if not t.is_cuda:
        raise ValueError(f"{name} is on {dev}: the kernels run on a CUDA device; move the inputs there first")
    if dtype not in _DTYPE_CODE:
        raise TypeError(f"{name} has dtype {dtype}, expected one of {tuple(_DTYPE_CODE)}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    return dev, dtype


_ACTIVATIONS = {"silu": 1, "swish": 1, None: 0, "identity": 0}


def _silu(activation) -> int:
    try:
        return _ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}") from None


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _stream(stream, dev):
    """(the given stream or None, handle of the stream to run on), where the inputs' device is the current one."""
    index = dev.index
    if current_device() != index:
        require_current(dev)
    if stream is None:
        return None, _raw_stream(index) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return stream, stream.cuda_stream


def _empty(shape, dtype, dev, stream):
    """A new tensor, made on the call's stream: the allocator reuses its memory in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _like(t, stream):
    """A new dense tensor shaped like t, whose rows are dense. (For such a tensor empty_like gives a dense one: it
    keeps strides only where they leave no gaps. It costs the host less than empty.)"""
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _state_grad(pool, n, nb, dev, stream):
    """A new fp32 gradient of a pool of n slots: zero outside the batch, which writes every slot where nb = n."""
    make = torch.empty if n == nb else torch.zeros
    if stream is None:
        return make(pool.shape, dtype=torch.float32, device=dev)
    with torch.cuda.stream(stream):
        return make(pool.shape, dtype=torch.float32, device=dev)


def _out(out, x, dtype, dev, stream):
    """The given output or a new one, shaped like the activation x and dense."""
    if out is None:
        return torch.empty_like(x) if stream is None else _like(x, stream)
    _dense(out, "out", dtype, dev, x.shape)
    return out


def _slots(cache_indices, dev):
    """(number of sequences, address) of the batch's slots."""
    if not isinstance(cache_indices, torch.Tensor) or cache_indices.dim() != 1:
        raise ValueError("cache_indices must be a 1-D tensor with one entry per sequence")
    shape = cache_indices.shape
    return shape[0], _dense(cache_indices, "cache_indices", torch.int64, dev, shape)


def _pool(pool, name, dtype, dev, inner):
    """(number of slots, address) of a state pool."""
    if not isinstance(pool, torch.Tensor) or pool.dim() != 3:
        raise ValueError(f"{name} must be [pool, {inner[0]}, {inner[1]}]")
    n = pool.shape[0]
    return n, _dense(pool, name, dtype, dev, (n, *inner))


def _workspace(need, what, workspace, stream, handle, dev, keep):
    """(pointer, bytes, owner, lock to hold while the call is enqueued) of the call's workspace: the caller's, the one
    kept for this stream, or a new one."""
    if need == 0:
        raise GdnError(2, f"{what}: unsupported sizes")
    if workspace is not None:
        return *given_workspace(workspace, dev), workspace, UNSHARED
    if keep:
        buf, lock = workspace_for(dev, stream, handle, need)
    else:
        buf, lock = _empty((need + 256,), torch.uint8, dev, stream), UNSHARED
    ptr = aligned_ptr(buf)
    return ptr, buf.numel() - (ptr - buf.data_ptr()), buf, lock


def _status_word(status, dev, stream, handle):
    """(a step's status word, its address): the caller's, or the one kept for this thread and stream."""
    if status is None:
        status = status_word(dev, stream, handle)
    elif not isinstance(status, torch.Tensor) or status.dtype != torch.int32 or status.device != dev or status.numel() < 1:
        raise ValueError("status must be an int32 tensor on the inputs' device")
    return status, status.data_ptr()


def _finish(st, what, check, word, handle):
    if st:
        _lib.check(st, what)
    if check:
        _lib.check(_lib.load().gdn_get_device_status(word, handle), f"{what} (device)")


# ----------------------------------------------------------------------------- short causal convolution


def _conv_args(x, weight, bias, conv_pool, cache_indices, activation):
    """(device, dtype, rows, channels, width, B, pool slots, the C call's arguments up to the slots)."""
    silu = _silu(activation)
    try:
        dtype, i = x.dtype, x.get_device()
        T, D = x.shape
        W = weight.shape[1]
        xs = x.stride()
        B, pool = cache_indices.numel(), conv_pool.shape[0]
        if (T > 0 and xs[1] == 1 and (xs[0] >= D or T == 1) and dtype in _DTYPE_CODE and weight.dtype is torch.float32
                and weight.shape == (D, W) and conv_pool.shape == (pool, W - 1, D) and conv_pool.dtype is dtype
                and cache_indices.dtype is torch.int64 and cache_indices.dim() == 1 and i >= 0
                and weight.get_device() == i and conv_pool.get_device() == i and cache_indices.get_device() == i
                and weight.is_contiguous() and conv_pool.is_contiguous() and cache_indices.is_contiguous()
                and (bias is None or bias.dtype is torch.float32 and bias.get_device() == i and bias.dim() == 1
                     and bias.numel() == D and bias.is_contiguous())):
            return (x.device, dtype, T, D, W, B, pool,
                    (x.data_ptr(), xs[0] if T > 1 else D, _DTYPE_CODE[dtype], weight.data_ptr(), None if bias is None else bias.data_ptr(),
                     conv_pool.data_ptr(), pool, cache_indices.data_ptr()), silu)
    except (AttributeError, ValueError, IndexError):
        pass
    dev, dtype = _activation(x, "x", 2)
    T, D = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight must be [{D}, width]")
    W = weight.shape[1]
    xs, wp = _rows(x, "x", dtype, dev, (T, D)), _dense(weight, "weight", torch.float32, dev, (D, W))
    bp = _opt(bias, "bias", torch.float32, dev, (D,))
    pool, pp = _pool(conv_pool, "conv_pool", dtype, dev, (W - 1, D))
    B, ip = _slots(cache_indices, dev)
    return dev, dtype, T, D, W, B, pool, (x.data_ptr(), xs, _DTYPE_CODE[dtype], wp, bp, pp, pool, ip), silu


def gdn_conv_extend(x, weight, bias, conv_pool, cache_indices, cu_seqlens, *, activation: Optional[str] = "silu",
                    out: torch.Tensor = None, workspace: torch.Tensor = None, check: bool = False,
                    stream=None) -> torch.Tensor:
    """Short causal convolution of a packed batch; returns ``out [T, D]`` in x's dtype.

    x ``[T, D]``; weight ``[D, W]`` fp32 with W = 2, 3 or 4 (the last tap meets the newest token); bias
    ``[D]`` fp32 or None; conv_pool ``[pool, W - 1, D]`` in x's dtype, each slot's last W - 1 inputs, oldest
    first, updated in place; cache_indices ``[B]``, cu_seqlens ``[B + 1]`` int64. ``activation`` is
    ``"silu"`` or None. ``check=True`` waits and raises on a bad slot or bad cu_seqlens. ``workspace``: memory for the
    call's plan (256-byte aligned; its first int32 becomes the call's status); by default a kept one of the stream,
    or the graph's own in a capture.
    """
    dev, dtype, T, D, W, B, pool, args, silu = _conv_args(x, weight, bias, conv_pool, cache_indices, activation)
    cp = _dense(cu_seqlens, "cu_seqlens", torch.int64, dev, (B + 1,))
    stream, handle = _stream(stream, dev)
    out = _out(out, x, dtype, dev, stream)
    L = _lib.load()
    ws, nbytes, _keep, lock = _workspace(L.gdn_conv_workspace_size(T, B, D, W), "gdn_conv_extend", workspace, stream, handle,
                                         dev, True)
    with lock:
        st = L.gdn_conv_extend(*args, cp, B, out.data_ptr(), T, D, W, silu, ws, nbytes, handle)
        _finish(st, "gdn_conv_extend", check, ws, handle)
    return out


def gdn_conv_step(x, weight, bias, conv_pool, cache_indices, *, activation: Optional[str] = "silu",
                  out: torch.Tensor = None, status: torch.Tensor = None, check: bool = False, stream=None) -> torch.Tensor:
    """:func:`gdn_conv_extend` with one token per sequence: x, out ``[B, D]``.

    ``status``: an int32 device tensor for the step's status word, which no step that may run at the same time
    shares; by default a kept one of the calling thread and stream, or the graph's own in a capture.
    """
    dev, dtype, B, D, W, n, _, args, silu = _conv_args(x, weight, bias, conv_pool, cache_indices, activation)
    if n != B:
        raise ValueError("cache_indices must have one entry per sequence")
    stream, handle = _stream(stream, dev)
    out = _out(out, x, dtype, dev, stream)
    _keep, word = _status_word(status, dev, stream, handle)
    st = _lib.load().gdn_conv_step(*args, B, out.data_ptr(), D, W, silu, word, handle)
    _finish(st, "gdn_conv_step", check, word, handle)
    return out


class GdnConvGrads(NamedTuple):
    """Gradients returned by :func:`gdn_conv_backward`."""
    dx: torch.Tensor             # [T, D], x's dtype
    dweight: torch.Tensor        # [D, W] fp32
    dbias: Optional[torch.Tensor]  # [D] fp32, None without a bias
    d_state_pool: torch.Tensor   # [pool, W - 1, D] fp32: zero except at the batch's slots


def gdn_conv_backward(x, weight, bias, conv_pool, cache_indices, cu_seqlens, d_out, d_state=None, *,
                      activation: Optional[str] = "silu", workspace: torch.Tensor = None, check: bool = False,
                      stream=None) -> GdnConvGrads:
    """Gradients of :func:`gdn_conv_extend` for ``L = <d_out, out> + <d_state, final slots>``.

    Inputs as for the forward call, with ``conv_pool`` as that call found it. d_out ``[T, D]`` in x's dtype;
    d_state ``[pool, W - 1, D]`` fp32 or None.
    """
    dev, dtype, T, D, W, B, pool, args, silu = _conv_args(x, weight, bias, conv_pool, cache_indices, activation)
    f32 = torch.float32
    cp = _dense(cu_seqlens, "cu_seqlens", torch.int64, dev, (B + 1,))
    ds = _rows(d_out, "d_out", dtype, dev, (T, D))
    dsp = _opt(d_state, "d_state", f32, dev, conv_pool.shape)
    stream, handle = _stream(stream, dev)
    g = GdnConvGrads(_like(x, stream), _like(weight, stream), None if bias is None else _like(bias, stream),
                     _state_grad(conv_pool, pool, B, dev, stream))
    L = _lib.load()
    ws, nbytes, _keep, lock = _workspace(L.gdn_conv_backward_workspace_size(T, B, D, W), "gdn_conv_backward", workspace, stream,
                                         handle, dev, True)
    with lock:
        st = L.gdn_conv_backward(*args, cp, B, d_out.data_ptr(), ds, dsp,
                                 g.dx.data_ptr(), g.dweight.data_ptr(), None if g.dbias is None else g.dbias.data_ptr(),
                                 g.d_state_pool.data_ptr(), T, D, W, silu, ws, nbytes, handle)
        _finish(st, "gdn_conv_backward", check, ws, handle)
    return g


# ----------------------------------------------------------------------------- selective scan


def _ssm_args(x, dt, A, B, C, D, z, dt_bias, state_pool, cache_indices):
    """(device, dtype, rows, channels, groups, states, batch, pool slots, the C call's arguments up to the slots)."""
    f32 = torch.float32
    try:
        rows, dtype, i = x.shape, x.dtype, x.get_device()
        T, Dm = rows
        inner = B.shape
        G, N = inner[1], inner[2]
        xs, ts, bs, cs = x.stride(), dt.stride(), B.stride(), C.stride()
        nb, pool, GN = cache_indices.numel(), state_pool.shape[0], G * N
        zs = (0, 1) if z is None else z.stride()
        if (T > 1 and Dm % G == 0 and i >= 0 and dtype in _DTYPE_CODE
                and xs[1] == 1 and ts[1] == 1 and zs[1] == 1 and bs[2] == 1 and cs[2] == 1 and bs[1] == N and cs[1] == N
                and xs[0] >= Dm and ts[0] >= Dm and bs[0] >= GN and cs[0] >= GN
                and dt.dtype is dtype and B.dtype is dtype and C.dtype is dtype and A.dtype is f32
                and dt.shape == rows and inner == (T, G, N) and C.shape == inner and A.shape == (Dm, N)
                and state_pool.shape == (pool, Dm, N) and state_pool.dtype is f32 and cache_indices.dtype is torch.int64
                and cache_indices.dim() == 1 and dt.get_device() == i and B.get_device() == i and C.get_device() == i
                and A.get_device() == i and state_pool.get_device() == i and cache_indices.get_device() == i
                and A.is_contiguous() and state_pool.is_contiguous() and cache_indices.is_contiguous()
                and (z is None or z.shape == rows and zs[0] >= Dm and z.dtype is dtype and z.get_device() == i)
                and (D is None or D.dtype is f32 and D.get_device() == i and D.dim() == 1 and D.numel() == Dm
                     and D.is_contiguous())
                and (dt_bias is None or dt_bias.dtype is f32 and dt_bias.get_device() == i and dt_bias.dim() == 1
                     and dt_bias.numel() == Dm and dt_bias.is_contiguous())):
            return (x.device, dtype, T, Dm, G, N, nb, pool,
                    (x.data_ptr(), xs[0], dt.data_ptr(), ts[0], _DTYPE_CODE[dtype], A.data_ptr(), B.data_ptr(), bs[0],
                     C.data_ptr(), cs[0], None if D is None else D.data_ptr(), None if z is None else z.data_ptr(), zs[0],
                     None if dt_bias is None else dt_bias.data_ptr(), state_pool.data_ptr(), pool, cache_indices.data_ptr()))
    except (AttributeError, ValueError, IndexError, ZeroDivisionError):
        pass
    dev, dtype = _activation(x, "x", 2)
    rows = x.shape
    T, Dm = rows
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError(f"A must be [{Dm}, states]")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError(f"B must be [{T}, groups, states]")
    N, G = A.shape[1], B.shape[1]
    if G <= 0 or Dm % G:
        raise ValueError(f"{Dm} channels are not a multiple of {G} groups")
    per, inner = (Dm,), (T, G, N)
    xs, ts = _rows(x, "x", dtype, dev, rows), _rows(dt, "dt", dtype, dev, rows)
    bs, cs = _rows(B, "B", dtype, dev, inner), _rows(C, "C", dtype, dev, inner)
    zs = 0 if z is None else _rows(z, "z", dtype, dev, rows)
    ap, dp, bp = _dense(A, "A", f32, dev, (Dm, N)), _opt(D, "D", f32, dev, per), _opt(dt_bias, "dt_bias", f32, dev, per)
    pool, pp = _pool(state_pool, "state_pool", f32, dev, (Dm, N))
    nb, ip = _slots(cache_indices, dev)
    return (dev, dtype, T, Dm, G, N, nb, pool,
            (x.data_ptr(), xs, dt.data_ptr(), ts, _DTYPE_CODE[dtype], ap, B.data_ptr(), bs, C.data_ptr(), cs, dp,
             None if z is None else z.data_ptr(), zs, bp, pp, pool, ip))


def gdn_ssm_extend(x, dt, A, B, C, D, z, dt_bias, state_pool, cache_indices, cu_seqlens, *, softplus: bool = True,
                   out: torch.Tensor = None, workspace: torch.Tensor = None, check: bool = False,
                   stream=None) -> torch.Tensor:
    """Selective state space scan of a packed batch; returns ``out [T, Dm]`` in x's dtype.

    x, dt ``[T, Dm]`` and the gate z ``[T, Dm]`` (or None); A ``[Dm, N]`` fp32 (N from 1 to 64); B, C
    ``[T, G, N]`` with Dm a multiple of G; D, dt_bias ``[Dm]`` fp32 or None; state_pool ``[pool, Dm, N]``
    fp32, updated in place; cache_indices ``[B]``, cu_seqlens ``[B + 1]`` int64. With ``softplus`` the step
    is softplus(dt + dt_bias), else dt + dt_bias. ``check=True`` waits and raises on a bad slot or bad
    cu_seqlens.
    """
    dev, dtype, T, Dm, G, N, nb, pool, args = _ssm_args(x, dt, A, B, C, D, z, dt_bias, state_pool, cache_indices)
    cp = _dense(cu_seqlens, "cu_seqlens", torch.int64, dev, (nb + 1,))
    stream, handle = _stream(stream, dev)
    out = _out(out, x, dtype, dev, stream)
    L = _lib.load()
    ws, nbytes, _keep, lock = _workspace(L.gdn_ssm_workspace_size(T, nb, Dm, G, N), "gdn_ssm_extend", workspace, stream, handle,
                                         dev, True)
    with lock:
        st = L.gdn_ssm_extend(*args, cp, nb, out.data_ptr(), T, Dm, G, N, 1 if softplus else 0, ws, nbytes, handle)
        _finish(st, "gdn_ssm_extend", check, ws, handle)
    return out


def gdn_ssm_step(x, dt, A, B, C, D, z, dt_bias, state_pool, cache_indices, *, softplus: bool = True,
                 out: torch.Tensor = None, status: torch.Tensor = None, check: bool = False, stream=None) -> torch.Tensor:
    """:func:`gdn_ssm_extend` with one token per sequence: x, dt, z, out ``[B, Dm]``, B, C ``[B, G, N]``.

    ``status`` as for :func:`gdn_conv_step`.
    """
    dev, dtype, nb, Dm, G, N, n, _, args = _ssm_args(x, dt, A, B, C, D, z, dt_bias, state_pool, cache_indices)
    if n != nb:
        raise ValueError("cache_indices must have one entry per sequence")
    stream, handle = _stream(stream, dev)
    out = _out(out, x, dtype, dev, stream)
    _keep, word = _status_word(status, dev, stream, handle)
    st = _lib.load().gdn_ssm_step(*args, nb, out.data_ptr(), Dm, G, N, 1 if softplus else 0, word, handle)
    _finish(st, "gdn_ssm_step", check, word, handle)
    return out


class GdnSsmGrads(NamedTuple):
    """Gradients returned by :func:`gdn_ssm_backward`; None where the input was None."""
    dx: torch.Tensor                  # [T, Dm], x's dtype
    ddt: torch.Tensor                 # [T, Dm], x's dtype
    dA: torch.Tensor                  # [Dm, N] fp32
    dB: torch.Tensor                  # [T, G, N], x's dtype
    dC: torch.Tensor                  # [T, G, N], x's dtype
    dD: Optional[torch.Tensor]        # [Dm] fp32
    dz: Optional[torch.Tensor]        # [T, Dm], x's dtype
    ddt_bias: Optional[torch.Tensor]  # [Dm] fp32
    d_state_pool: torch.Tensor        # [pool, Dm, N] fp32: zero except at the batch's slots


def gdn_ssm_backward(x, dt, A, B, C, D, z, dt_bias, state_pool, cache_indices, cu_seqlens, d_out, d_state=None, *,
                     softplus: bool = True, d_state_pool: torch.Tensor = None, workspace: torch.Tensor = None,
                     check: bool = False, stream=None) -> GdnSsmGrads:
    """Gradients of :func:`gdn_ssm_extend` for ``L = <d_out, out> + <d_state, final states>``.

    Inputs as for the forward call, with ``state_pool`` as that call found it. d_out ``[T, Dm]`` in x's dtype;
    d_state ``[pool, Dm, N]`` fp32 or None. ``d_state_pool``: a tensor to write the initial states' gradients
    into at the batch's slots (it may be ``d_state`` itself) instead of a new zero tensor.
    """
    dev, dtype, T, Dm, G, N, nb, pool, args = _ssm_args(x, dt, A, B, C, D, z, dt_bias, state_pool, cache_indices)
    f32 = torch.float32
    cp = _dense(cu_seqlens, "cu_seqlens", torch.int64, dev, (nb + 1,))
    ds = _rows(d_out, "d_out", dtype, dev, (T, Dm))
    dsp = _opt(d_state, "d_state", f32, dev, state_pool.shape)
    _opt(d_state_pool, "d_state_pool", f32, dev, state_pool.shape)
    stream, handle = _stream(stream, dev)
    g = GdnSsmGrads(_like(x, stream), _like(dt, stream), _like(A, stream), _like(B, stream), _like(C, stream),
                    None if D is None else _like(D, stream), None if z is None else _like(z, stream),
                    None if dt_bias is None else _like(dt_bias, stream),
                    _state_grad(state_pool, pool, nb, dev, stream) if d_state_pool is None else d_state_pool)
    L = _lib.load()
    ws, nbytes, _keep, _ = _workspace(L.gdn_ssm_backward_workspace_size(T, nb, Dm, G, N), "gdn_ssm_backward", workspace, stream,
                                      handle, dev, False)
    st = L.gdn_ssm_backward(*args, cp, nb, d_out.data_ptr(), ds, dsp,
                            *[None if t is None else t.data_ptr() for t in g], T, Dm, G, N, 1 if softplus else 0, ws, nbytes,
                            handle)
    _finish(st, "gdn_ssm_backward", check, ws, handle)
    return g


# ----------------------------------------------------------------------------- layer norm


def _norm_args(x, params):
    """(device, dtype, rows, columns, x's row stride, the fp32 [columns] parameters' addresses)."""
    f32 = torch.float32
    try:
        dtype, i = x.dtype, x.get_device()
        rows, n = x.shape
        xs = x.stride()
        if rows > 0 and xs[1] == 1 and (xs[0] >= n or rows == 1) and i >= 0 and dtype in _DTYPE_CODE:
            for t in params:
                if t is not None and not (t.dtype is f32 and t.get_device() == i and t.dim() == 1 and t.numel() == n
                                          and t.is_contiguous()):
                    break
            else:
                return (x.device, dtype, rows, n, xs[0] if rows > 1 else n,
                        [None if t is None else t.data_ptr() for t in params])
    except (AttributeError, ValueError, IndexError):
        pass
    dev, dtype = _activation(x, "x", 2)
    rows, n = x.shape
    xs = _rows(x, "x", dtype, dev, (rows, n))
    return dev, dtype, rows, n, xs, [_opt(t, name, f32, dev, (n,)) for name, t in zip(("weight", "bias"), params)]


def gdn_layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, out: torch.Tensor = None, return_stats: bool = False,
                   stream=None):
    """Layer norm of the rows of x ``[rows, n]``; returns ``out`` in x's dtype.

    weight, bias ``[n]`` fp32 or None. With ``return_stats`` returns ``(out, mean, rstd)``, the statistics
    ``[rows]`` fp32 that :func:`gdn_layer_norm_backward` takes.
    """
    dev, dtype, rows, n, xs, (wp, bp) = _norm_args(x, (weight, bias))
    stream, handle = _stream(stream, dev)
    out = _out(out, x, dtype, dev, stream)
    mean = _empty((rows,), torch.float32, dev, stream) if return_stats else None
    rstd = _like(mean, stream) if return_stats else None
    st = _lib.load().gdn_layer_norm(x.data_ptr(), xs, _DTYPE_CODE[dtype], wp, bp, out.data_ptr(),
                                    mean.data_ptr() if return_stats else None, rstd.data_ptr() if return_stats else None,
                                    rows, n, float(eps), handle)
    _lib.check(st, "gdn_layer_norm")
    return (out, mean, rstd) if return_stats else out


class GdnNormGrads(NamedTuple):
    """Gradients returned by :func:`gdn_layer_norm_backward`."""
    dx: torch.Tensor       # [rows, n], x's dtype
    dweight: torch.Tensor  # [n] fp32
    dbias: torch.Tensor    # [n] fp32


def gdn_layer_norm_backward(d_out, x, weight, mean, rstd, *, workspace: torch.Tensor = None, stream=None) -> GdnNormGrads:
    """Gradients of :func:`gdn_layer_norm` for the gradient ``d_out [rows, n]`` (x's dtype) of its output."""
    dev, dtype, rows, n, xs, (wp,) = _norm_args(x, (weight,))
    ds = _rows(d_out, "d_out", dtype, dev, (rows, n))
    f32 = torch.float32
    mp, rp = _dense(mean, "mean", f32, dev, (rows,)), _dense(rstd, "rstd", f32, dev, (rows,))
    stream, handle = _stream(stream, dev)
    if weight is None:
        dw, db = _empty((n,), f32, dev, stream), _empty((n,), f32, dev, stream)
    else:
        dw, db = _like(weight, stream), _like(weight, stream)
    g = GdnNormGrads(_like(x, stream), dw, db)
    L = _lib.load()
    # (Not the stream's kept workspace: that one's first word is the status of the last call that has one.)
    ws, nbytes, _keep, _ = _workspace(L.gdn_layer_norm_backward_workspace_size(rows, n), "gdn_layer_norm_backward", workspace,
                                      stream, handle, dev, False)
    st = L.gdn_layer_norm_backward(d_out.data_ptr(), ds, x.data_ptr(), xs, _DTYPE_CODE[dtype], wp, mp, rp, g.dx.data_ptr(),
                                   g.dweight.data_ptr(), g.dbias.data_ptr(), rows, n, ws, nbytes, handle)
    _lib.check(st, "gdn_layer_norm_backward")
    return g


# ----------------------------------------------------------------------------- autograd


# (The backward passes are kernels without gradients of their own: once_differentiable makes a second derivative an
# error, where it would otherwise be zero in silence.)

def _own_slots(state, x):
    return torch.arange(state.shape[0], dtype=torch.int64, device=x.device)


class CausalConv(torch.autograd.Function):
    """The convolution as an autograd function: ``apply(x, weight, bias, initial_state, cu_seqlens,
    activation="silu")`` with ``initial_state [B, W - 1, D]`` in x's dtype (one per sequence) returns
    ``(out, final_state)``; gradients flow to x, weight, bias and initial_state. Second derivatives are an error."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation="silu"):
        pool = initial_state.detach().clone(memory_format=torch.contiguous_format)
        out = gdn_conv_extend(x, weight, bias, pool, _own_slots(pool, x), cu_seqlens, activation=activation)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        return out, pool

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_final):
        x, weight, bias, state, cu = ctx.saved_tensors
        d_out = torch.zeros_like(x, memory_format=torch.contiguous_format) if d_out is None else d_out.to(x.dtype).contiguous()
        d_state = None if d_final is None else d_final.float().contiguous()
        g = gdn_conv_backward(x, weight, bias, state.detach().contiguous(), _own_slots(state, x), cu, d_out, d_state,
                              activation=ctx.activation)
        return g.dx, g.dweight, g.dbias, g.d_state_pool.to(state.dtype), None, None


class SelectiveScan(torch.autograd.Function):
    """The scan as an autograd function: ``apply(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens,
    softplus=True)`` with ``initial_state [B, Dm, N]`` fp32 (one per sequence) returns ``(out,
    final_state)``; gradients flow to every tensor but cu_seqlens. Second derivatives are an error."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, softplus=True):
        pool = initial_state.detach().clone(memory_format=torch.contiguous_format)
        out = gdn_ssm_extend(x, dt, A, B, C, D, z, dt_bias, pool, _own_slots(pool, x), cu_seqlens, softplus=softplus)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens)
        ctx.softplus = softplus
        return out, pool

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_final):
        x, dt, A, B, C, D, z, dt_bias, state, cu = ctx.saved_tensors
        d_out = torch.zeros_like(x, memory_format=torch.contiguous_format) if d_out is None else d_out.to(x.dtype).contiguous()
        d_state = None if d_final is None else d_final.float().contiguous()
        g = gdn_ssm_backward(x, dt, A, B, C, D, z, dt_bias, state.detach().contiguous(), _own_slots(state, x), cu, d_out,
                             d_state, softplus=ctx.softplus)
        return g.dx, g.ddt, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddt_bias, g.d_state_pool, None, None


class LayerNorm(torch.autograd.Function):
    """Layer norm as an autograd function: ``apply(x, weight, bias, eps=1e-5)``; gradients flow to x, weight
    and bias. Second derivatives are an error."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps=1e-5):
        out, mean, rstd = gdn_layer_norm(x, weight, bias, eps=eps, return_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        x, weight, mean, rstd = ctx.saved_tensors
        g = gdn_layer_norm_backward(d_out.to(x.dtype).contiguous(), x, weight, mean, rstd)
        return g.dx, None if weight is None else g.dweight, g.dbias if ctx.has_bias else None, None
