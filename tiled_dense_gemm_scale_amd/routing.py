"""Routed experts on the fused product: the rows of a batch sorted by group
(group_rows), every group's product with its own weights (gemm_grouped), the
rows copied into group order (gather_rows) and summed back with their weights
(combine_rows and its gradient), and the whole layer (expert_mlp).

Every function enqueues on `stream` (default: the current stream of the
inputs' device); what it allocates itself is allocated for that stream.  As
with every call of this package autograd records nothing: outputs carry no
gradient, whatever the inputs require.  combine_rows and combine_rows_backward
are the gradients of gather_rows and combine_rows; the grouped product has none
here.
"""
from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch

from . import _native
from ._native import group_workspace_bytes

__all__ = ["group_rows", "group_workspace_bytes", "gather_rows", "combine_rows", "combine_rows_backward",
           "gemm_grouped", "expert_mlp"]


@contextlib.contextmanager
def _environment(device: torch.device, stream):
    """`device` current, and `stream` (None: the current one, a torch stream,
    or a hipStream_t as an integer) as the stream that allocations belong to.
    Yields the stream's handle."""
    with torch.cuda.device(device):
        if stream is None:
            yield int(torch.cuda.current_stream(device).cuda_stream)
        elif not hasattr(stream, "cuda_stream") and int(stream) == 0:
            with torch.cuda.stream(torch.cuda.default_stream(device)):
                yield 0
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)
            with torch.cuda.stream(s):
                yield int(s.cuda_stream)


# A launch takes 3 us of host time, less than the context managers and stream
# objects around it would; so the usual call, on its device's current stream,
# reads the stream's handle as torch's own generated code does.
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def enqueue(index: int, stream, go):
    """go(stream handle) with device `index` current and allocations made for
    that stream; what it returns."""
    if stream is None and _current_stream is not None and _current_device() == index:
        return go(_current_stream(index))
    with _environment(torch.device("cuda", index), stream) as s:
        return go(s)


def check(name: str, t: torch.Tensor, dtypes, shape, index: Optional[int]) -> None:
    """Refuses (TypeError, ValueError) a `t` that is not a contiguous tensor
    of one of `dtypes`, of `shape` (None: any length in that place), on device
    `index` (None: any)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d).replace('torch.', '') for d in dtypes)}")
    if t.dim() != len(shape) or any(want is not None and int(got) != want for got, want in zip(t.shape, shape)):
        want = tuple("*" if s is None else s for s in shape)
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def need(name: str, t: torch.Tensor, dtype, shape, index: int) -> int:
    """`t`'s address once it is what check() lets pass; the usual case first."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    check(name, t, dtype, tuple(shape), index)
    return t.data_ptr()


def matrix(name: str, t, dtype, rank: int, index: Optional[int] = None) -> int:
    """need() for a tensor of `rank` dimensions of any length (index None: on
    any device)."""
    try:
        at = t.get_device()
        if t.dtype is dtype and t.dim() == rank and at >= 0 and (index is None or at == index) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    check(name, t, dtype, (None,) * rank, index)
    return t.data_ptr()


def output(name: str, t: Optional[torch.Tensor], dtype, shape, like: torch.Tensor) -> torch.Tensor:
    """`t` after need(), or a new tensor on `like`'s device."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    need(name, t, dtype, shape, like.get_device())
    return t


def workspace_of(workspace: torch.Tensor, index: int) -> Tuple[int, int]:
    """The workspace's address and bytes."""
    return matrix("workspace", workspace, torch.uint8, 1, index), workspace.numel()


def group_rows(ids: torch.Tensor, groups: int, offsets: Optional[torch.Tensor] = None,
               rows: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The slots of ids (T, k) or (T,), int32 or int64, sorted by group and by
    slot within a group; ids outside [0, groups) are dropped.  Returns int32
    tensors: offsets (groups + 1,), where the sorted rows of each group start;
    rows (T k,), the token of each sorted row, -1 behind the last group;
    positions (like ids), the sorted row of each slot, -1 for a dropped one.
    groups is 1..1024.  workspace: group_workspace_bytes(T k, groups) bytes of
    any content, allocated here when not given."""
    if not isinstance(ids, torch.Tensor) or ids.dim() not in (1, 2):
        raise ValueError("ids must be a tensor of shape (tokens, k) or (tokens,)")
    if ids.dtype not in (torch.int32, torch.int64) or ids.get_device() < 0 or not ids.is_contiguous():
        check("ids", ids, (torch.int32, torch.int64), ids.shape, None)
    shape, dev, groups = ids.shape, ids.get_device(), int(groups)
    T, k = shape[0], shape[1] if len(shape) == 2 else 1
    n = T * k

    def go(s):
        if workspace is not None:
            wptr, wbytes = workspace_of(workspace, dev)
        else:
            wbytes = group_workspace_bytes(n, groups)
            ws = torch.empty(wbytes, dtype=torch.uint8, device=ids.device) if wbytes else None
            wptr = ws.data_ptr() if wbytes else 0
        o = output("offsets", offsets, torch.int32, (max(groups, 0) + 1,), ids)
        r = output("rows", rows, torch.int32, (n,), ids)
        p = output("positions", positions, torch.int32, shape, ids)
        _native.check(_native.group_rows(T, k, groups, ids.data_ptr(), ids.element_size(), o.data_ptr(), r.data_ptr(),
                                         p.data_ptr(), wptr, wbytes, s))
        return o, r, p

    return enqueue(dev, stream, go)


def gather_rows(x: torch.Tensor, rows: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[p] = x[rows[p]] for x (T, H) fp16 and rows (P,) int32; zeros where
    rows[p] is outside [0, T).  Its gradient is combine_rows(dout, positions)
    without weights.  Returns out (P, H)."""
    matrix("x", x, torch.float16, 2)
    matrix("rows", rows, torch.int32, 1, x.get_device())
    (T, H), P = x.shape, rows.shape[0]

    def go(s):
        y = output("out", out, torch.float16, (P, H), x)
        _native.check(_native.gather_rows(P, T, H, x.data_ptr(), rows.data_ptr(), y.data_ptr(), s))
        return y

    return enqueue(x.get_device(), stream, go)


def _positions(positions: torch.Tensor, index: int) -> Tuple[int, int]:
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
        raise ValueError("positions must be a tensor of shape (tokens, k) or (tokens,)")
    need("positions", positions, torch.int32, positions.shape, index)
    return positions.shape[0], positions.shape[1] if positions.dim() == 2 else 1


def combine_rows(y: torch.Tensor, positions: torch.Tensor, weights: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[positions[t, j]] for y (P, H) fp16,
    positions (T, k) or (T,) int32 and weights like positions, float32 (None:
    ones); fp32 sums in order of j, rounded once to fp16.  Positions outside
    [0, P) have no term.  Returns out (T, H)."""
    matrix("y", y, torch.float16, 2)
    (P, H), dev = y.shape, y.get_device()
    T, k = _positions(positions, dev)
    wptr = need("weights", weights, torch.float32, positions.shape, dev) if weights is not None else 0

    def go(s):
        o = output("out", out, torch.float16, (T, H), y)
        _native.check(_native.combine_rows(T, k, P, H, y.data_ptr(), positions.data_ptr(), wptr, o.data_ptr(), s))
        return o

    return enqueue(dev, stream, go)


def combine_rows_backward(dout: torch.Tensor, y: Optional[torch.Tensor], positions: torch.Tensor,
                          weights: Optional[torch.Tensor], rows: torch.Tensor, dy: Optional[torch.Tensor] = None,
                          dweights: Optional[torch.Tensor] = None, stream=None
                          ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gradient of combine_rows: dy (P, H) fp16 with
    dy[positions[t, j]] = weights[t, j] * dout[t], zeros in the rows p that no
    choice names (rows[p] outside [0, T)), and dweights (like positions,
    float32) with <dout[t], y[positions[t, j]]>, 0 for a dropped choice.
    rows (P,) and positions are group_rows's; positions inside [0, P) must be
    distinct.  Without weights, y may be None and dweights is None."""
    matrix("dout", dout, torch.float16, 2)
    (T, H), dev = dout.shape, dout.get_device()
    tokens, k = _positions(positions, dev)
    if tokens != T:
        raise ValueError(f"positions must have {T} tokens as dout does, got {tokens}")
    matrix("rows", rows, torch.int32, 1, dev)
    P, wptr, yptr = rows.shape[0], 0, 0
    if weights is not None:
        wptr = need("weights", weights, torch.float32, positions.shape, dev)
        if y is None:
            raise ValueError("y is needed for the weights' gradient")
    elif dweights is not None:
        raise ValueError("dweights without weights")
    if y is not None:
        yptr = need("y", y, torch.float16, (P, H), dev)

    def go(s):
        gy = output("dy", dy, torch.float16, (P, H), dout)
        gw = output("dweights", dweights, torch.float32, positions.shape, dout) if weights is not None else None
        _native.check(_native.combine_rows_backward(T, k, P, H, dout.data_ptr(), yptr, positions.data_ptr(), wptr,
                                                    rows.data_ptr(), gy.data_ptr(),
                                                    gw.data_ptr() if gw is not None else 0, s))
        return gy, gw

    return enqueue(dev, stream, go)


ACTIVATIONS = {"relu": _native.GSR_ACT_RELU, "gelu": _native.GSR_ACT_GELU, "none": _native.GSR_ACT_NONE}


def gemm_grouped(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, alpha: float = 1.0, activation: str = "relu",
                 c: Optional[torch.Tensor] = None, stream=None, config_id: int = -1) -> torch.Tensor:
    """c[r] = act(alpha * a[rows[r]] @ b[e] + bias[e]) for the rows
    offsets[e] <= r < offsets[e + 1] of every group e: a (T, K) fp16 with rows
    (P,) int32 (an index outside [0, T) is a row of zeros), or a (P, K) without;
    b (E, K, N) fp16, bias (E, N) fp16 or None, offsets (E + 1,) int32 on the
    device (group_rows's), act "relu", "gelu" (tanh form) or "none".  Rows of
    c outside every group stay as they were; a c allocated here holds
    anything there.  Returns c (P, N)."""
    matrix("a", a, torch.float16, 2)
    (T, K), dev = a.shape, a.get_device()
    matrix("b", b, torch.float16, 3, dev)
    if b.shape[1] != K:
        raise ValueError(f"b must have shape (*, {K}, *), got {tuple(b.shape)}")
    E, N = b.shape[0], b.shape[2]
    optr = need("offsets", offsets, torch.int32, (E + 1,), dev)
    P, rptr = T, 0
    if rows is not None:
        matrix("rows", rows, torch.int32, 1, dev)
        P, rptr = rows.shape[0], rows.data_ptr()
    bias_ptr = need("bias", bias, torch.float16, (E, N), dev) if bias is not None else 0
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")

    def go(s):
        o = output("c", c, torch.float16, (P, N), a)
        _native.check(_native.gemm_grouped_scale_bias_act(P, N, K, E, a.data_ptr(), T, rptr, b.data_ptr(), bias_ptr,
                                                          o.data_ptr(), optr, alpha, ACTIVATIONS[activation], s,
                                                          config_id))
        return o

    return enqueue(dev, stream, go)


def expert_mlp(x: torch.Tensor, ids: torch.Tensor, weights: Optional[torch.Tensor], up: torch.Tensor,
               down: torch.Tensor, bias_up: Optional[torch.Tensor] = None, bias_down: Optional[torch.Tensor] = None,
               activation: str = "gelu", stream=None) -> torch.Tensor:
    """A layer of routed experts: out[t] = sum_j weights[t, j] *
    (act(x[t] @ up[e] + bias_up[e]) @ down[e] + bias_down[e]) with
    e = ids[t, j]; choices whose id names no expert are left out.  x (T, H),
    ids (T, k) int32 or int64, weights (T, k) float32 or None (ones), up
    (E, H, F), down (E, F, H).  The rows are sorted once; the products fetch
    x's rows where they are.  Returns out (T, H) fp16."""
    offsets, rows, positions = group_rows(ids, int(up.shape[0]), stream=stream)
    hidden = gemm_grouped(x, up, offsets, rows=rows, bias=bias_up, activation=activation, stream=stream)
    y = gemm_grouped(hidden, down, offsets, bias=bias_down, activation="none", stream=stream)
    return combine_rows(y, positions, weights, stream=stream)
