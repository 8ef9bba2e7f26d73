"""Routed experts on the fused product: the rows of a batch sorted by group
(group_rows), every group's product with its own weights (gemm_grouped), the
rows copied into group order (gather_rows) and summed back with their weights
(combine_rows and its gradient), and the whole layer (expert_mlp).

Every function enqueues on `stream` (default: the current stream of the
inputs' device); what it allocates itself is allocated for that stream.
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
def on_stream(device: torch.device, stream):
    """The launch environment: `device` current, and `stream` (None: the
    current one, a torch stream, or a hipStream_t as an integer) as the stream
    that allocations belong to.  Yields the stream's handle."""
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


def check(name: str, t: torch.Tensor, dtypes, shape, device: Optional[torch.device]) -> torch.Tensor:
    """`t` as a contiguous tensor of one of `dtypes`, of `shape` (None: any
    length in that place) and on `device`; raises TypeError or ValueError."""
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
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def check_workspace(workspace: torch.Tensor, device: torch.device) -> Tuple[int, int]:
    check("workspace", workspace, torch.uint8, (None,), device)
    return workspace.data_ptr(), workspace.numel()


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
    check("ids", ids, (torch.int32, torch.int64), tuple(ids.shape), None)
    groups = int(groups)
    T, k = int(ids.shape[0]), int(ids.shape[1]) if ids.dim() == 2 else 1
    dev, n = ids.device, T * k
    with on_stream(dev, stream) as s:
        need = group_workspace_bytes(n, groups)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        wptr, wbytes = check_workspace(workspace, dev)
        new = dict(dtype=torch.int32, device=dev)
        offsets = torch.empty(groups + 1, **new) if offsets is None else offsets
        rows = torch.empty(n, **new) if rows is None else rows
        positions = torch.empty(ids.shape, **new) if positions is None else positions
        check("offsets", offsets, torch.int32, (groups + 1,), dev)
        check("rows", rows, torch.int32, (n,), dev)
        check("positions", positions, torch.int32, tuple(ids.shape), dev)
        st = _native.group_rows(T, k, groups, ids.data_ptr(), ids.element_size(), offsets.data_ptr(), rows.data_ptr(),
                                positions.data_ptr(), wptr, wbytes, s)
    _native.check(st)
    return offsets, rows, positions


def gather_rows(x: torch.Tensor, rows: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[p] = x[rows[p]] for x (T, H) fp16 and rows (P,) int32; zeros where
    rows[p] is outside [0, T).  Its gradient is combine_rows(dout, positions)
    without weights.  Returns out (P, H)."""
    check("x", x, torch.float16, (None, None), None)
    T, H = int(x.shape[0]), int(x.shape[1])
    check("rows", rows, torch.int32, (None,), x.device)
    P = int(rows.shape[0])
    with on_stream(x.device, stream) as s:
        out = torch.empty((P, H), dtype=torch.float16, device=x.device) if out is None else out
        check("out", out, torch.float16, (P, H), x.device)
        st = _native.gather_rows(P, T, H, x.data_ptr(), rows.data_ptr(), out.data_ptr(), s)
    _native.check(st)
    return out


def _positions(positions: torch.Tensor, device: torch.device) -> Tuple[int, int]:
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
        raise ValueError("positions must be a tensor of shape (tokens, k) or (tokens,)")
    check("positions", positions, torch.int32, tuple(positions.shape), device)
    return int(positions.shape[0]), int(positions.shape[1]) if positions.dim() == 2 else 1


def combine_rows(y: torch.Tensor, positions: torch.Tensor, weights: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[positions[t, j]] for y (P, H) fp16,
    positions (T, k) or (T,) int32 and weights like positions, float32 (None:
    ones); fp32 sums in order of j, rounded once to fp16.  Positions outside
    [0, P) have no term.  Returns out (T, H)."""
    check("y", y, torch.float16, (None, None), None)
    P, H = int(y.shape[0]), int(y.shape[1])
    T, k = _positions(positions, y.device)
    if weights is not None:
        check("weights", weights, torch.float32, tuple(positions.shape), y.device)
    with on_stream(y.device, stream) as s:
        out = torch.empty((T, H), dtype=torch.float16, device=y.device) if out is None else out
        check("out", out, torch.float16, (T, H), y.device)
        st = _native.combine_rows(T, k, P, H, y.data_ptr(), positions.data_ptr(),
                                  weights.data_ptr() if weights is not None else 0, out.data_ptr(), s)
    _native.check(st)
    return out


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
    check("dout", dout, torch.float16, (None, None), None)
    T, H, dev = int(dout.shape[0]), int(dout.shape[1]), dout.device
    tokens, k = _positions(positions, dev)
    if tokens != T:
        raise ValueError(f"positions must have {T} tokens as dout does, got {tokens}")
    check("rows", rows, torch.int32, (None,), dev)
    P = int(rows.shape[0])
    if weights is not None:
        check("weights", weights, torch.float32, tuple(positions.shape), dev)
        if y is None:
            raise ValueError("y is needed for the weights' gradient")
    elif dweights is not None:
        raise ValueError("dweights without weights")
    if y is not None:
        check("y", y, torch.float16, (P, H), dev)
    with on_stream(dev, stream) as s:
        dy = torch.empty((P, H), dtype=torch.float16, device=dev) if dy is None else dy
        check("dy", dy, torch.float16, (P, H), dev)
        if weights is not None:
            dweights = torch.empty(positions.shape, dtype=torch.float32, device=dev) if dweights is None else dweights
            check("dweights", dweights, torch.float32, tuple(positions.shape), dev)
        st = _native.combine_rows_backward(
            T, k, P, H, dout.data_ptr(), y.data_ptr() if y is not None else 0, positions.data_ptr(),
            weights.data_ptr() if weights is not None else 0, rows.data_ptr(), dy.data_ptr(),
            dweights.data_ptr() if weights is not None else 0, s)
    _native.check(st)
    return dy, dweights


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
    check("a", a, torch.float16, (None, None), None)
    dev, T, K = a.device, int(a.shape[0]), int(a.shape[1])
    check("b", b, torch.float16, (None, K, None), dev)
    E, N = int(b.shape[0]), int(b.shape[2])
    check("offsets", offsets, torch.int32, (E + 1,), dev)
    if rows is not None:
        check("rows", rows, torch.int32, (None,), dev)
    P = T if rows is None else int(rows.shape[0])
    if bias is not None:
        check("bias", bias, torch.float16, (E, N), dev)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    with on_stream(dev, stream) as s:
        c = torch.empty((P, N), dtype=torch.float16, device=dev) if c is None else c
        check("c", c, torch.float16, (P, N), dev)
        st = _native.gemm_grouped_scale_bias_act(
            P, N, K, E, a.data_ptr(), T, rows.data_ptr() if rows is not None else 0, b.data_ptr(),
            bias.data_ptr() if bias is not None else 0, c.data_ptr(), offsets.data_ptr(), alpha,
            ACTIVATIONS[activation], s, config_id)
    _native.check(st)
    return c


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
