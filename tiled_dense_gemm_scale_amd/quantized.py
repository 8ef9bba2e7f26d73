"""Weights in 4 bits with a scale for every column and group of rows: made from
fp16 weights (quantize_w4), given back (dequantize_w4), and multiplied
(gemm_w4), for serving a few rows at a time.  Autograd records nothing, and
there is no gradient here."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _native
from ._native import w4_workspace_bytes
from .routing import ACTIVATIONS, enqueue, matrix, need, output, workspace_of

__all__ = ["W4", "quantize_w4", "dequantize_w4", "gemm_w4", "w4_workspace_bytes"]


class W4(NamedTuple):
    """A (K, N) matrix in 4 bits, or E of them: the weight of row r and column
    n is (q - zeros[r // group, n]) * scales[r // group, n].

    codes   int32 (ceil(K / 8), N) or (E, ceil(K / 8), N): bits 4i .. 4i + 3 of
            word (r, n) are the code q (0..15) of row 8 r + i
    scales  float16 (ceil(K / group), N) or (E, ceil(K / group), N)
    zeros   uint8 like scales, or None: 8 everywhere
    k       K
    group   a power of two from 32 on
    """
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: Optional[torch.Tensor]
    k: int
    group: int


def check_w4(name: str, w: W4, index: Optional[int], lead: tuple):
    """Refuses a `w` that is not a W4 of `lead` (E,) or () matrices on device
    `index` (None: any).  Returns K, N and the addresses of codes, scales and
    zeros."""
    if not isinstance(w, W4):
        raise TypeError(f"{name} must be a W4")
    k, group = int(w.k), int(w.group)
    if group < 32 or group & (group - 1):
        raise ValueError(f"{name}.group must be a power of two from 32 on, got {group}")
    if k < 0:
        raise ValueError(f"{name}.k must not be negative")
    codes = matrix(name + ".codes", w.codes, torch.int32, 2 + len(lead), index)
    at, shape = w.codes.get_device(), tuple(w.codes.shape)
    N = shape[-1]
    if shape[-2] != (k + 7) // 8 or shape[:-2] != lead:
        raise ValueError(f"{name}.codes must have shape {lead + ((k + 7) // 8, '*')}, got {shape}")
    like = lead + (-(-k // group), N)
    scales = need(name + ".scales", w.scales, torch.float16, like, at)
    zeros = need(name + ".zeros", w.zeros, torch.uint8, like, at) if w.zeros is not None else 0
    return k, N, codes, scales, zeros


def quantize_w4(b: torch.Tensor, group: int = 128, zeros: bool = False, stream=None) -> W4:
    """b (K, N) or (E, K, N) fp16 in 4 bits, groups of `group` rows.  Without
    zero points the scale is fp16(max|b| / 7) and q = clamp(rint(b / scale), -8,
    7) + 8; with them lo = min(b, 0), hi = max(b, 0), the scale is
    fp16((hi - lo) / 15), the zero point clamp(rint(-lo / scale), 0, 15) and
    q = clamp(rint(b / scale) + zero, 0, 15).  A group with an infinity or a NaN
    gets the scale NaN."""
    if not isinstance(b, torch.Tensor) or b.dim() not in (2, 3):
        raise ValueError("b must be a tensor of shape (K, N) or (E, K, N)")
    matrix("b", b, torch.float16, b.dim())
    group = int(group)
    if group < 32 or group & (group - 1):
        raise ValueError(f"group must be a power of two from 32 on, got {group}")
    lead, (K, N) = tuple(b.shape[:-2]), b.shape[-2:]

    def go(s):
        codes = torch.empty(lead + ((K + 7) // 8, N), dtype=torch.int32, device=b.device)
        scales = torch.empty(lead + (-(-K // group), N), dtype=torch.float16, device=b.device)
        z = torch.empty(scales.shape, dtype=torch.uint8, device=b.device) if zeros else None
        _native.check(_native.quantize_w4(lead[0] if lead else 1, K, N, group, b.data_ptr(), codes.data_ptr(),
                                          scales.data_ptr(), z.data_ptr() if zeros else 0, s))
        return W4(codes, scales, z, K, group)

    return enqueue(b.get_device(), stream, go)


def dequantize_w4(w: W4, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The weights' values, rounded once to fp16: (K, N) or (E, K, N)."""
    if not isinstance(w, W4):
        raise TypeError("w must be a W4")
    lead = tuple(w.codes.shape[:-2]) if isinstance(w.codes, torch.Tensor) and w.codes.dim() == 3 else ()
    K, N, codes, scales, zeros = check_w4("w", w, None, lead)

    def go(s):
        o = output("out", out, torch.float16, lead + (K, N), w.codes)
        _native.check(_native.dequantize_w4(lead[0] if lead else 1, K, N, w.group, codes, scales, zeros, o.data_ptr(), s))
        return o

    return enqueue(w.codes.get_device(), stream, go)


def gemm_w4(a: torch.Tensor, w: W4, workspace: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
            alpha: float = 1.0, activation: str = "relu", c: Optional[torch.Tensor] = None, stream=None,
            round_weights: bool = True) -> torch.Tensor:
    """c = act(alpha * a @ w + bias) for a (M, K) fp16, w a W4 of one (K, N)
    matrix, bias (N,) fp16 or None, act "relu", "gelu" (tanh form) or "none".
    Products are summed in fp32 and scaled group by group; the weights are not
    rounded, but where many rows make it faster (more than 16, commonly from 200
    on) they are written to the workspace as dequantize_w4 gives them, each rounded
    once to fp16, and multiplied by the dense kernels (but for the columns whose
    weights could pass fp16's range, which stay as they are).  round_weights False:
    never.  workspace: new_workspace(w4_workspace_bytes(M, N, K)), one per call that
    may run at the same time; with less, or None, neither that is done nor K split
    across workgroups.  Returns c (M, N)."""
    matrix("a", a, torch.float16, 2)
    (M, K), dev = a.shape, a.get_device()
    k, N, codes, scales, zeros = check_w4("w", w, dev, ())
    if k != K:
        raise ValueError(f"w must have {K} rows as a has columns, got {k}")
    bias_ptr = need("bias", bias, torch.float16, (N,), dev) if bias is not None else 0
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    wptr, wbytes = workspace_of(workspace, dev) if workspace is not None else (0, 0)
    values = 512 + 2 * K * N  # what the weights' values take
    if not round_weights and wbytes >= values and w4_workspace_bytes(M, N, K) == values:
        wbytes = values - 1

    def go(s):
        o = output("c", c, torch.float16, (M, N), a)
        _native.check(_native.gemm_w4_scale_bias_act(M, N, K, a.data_ptr(), w.group, codes, scales, zeros, bias_ptr,
                                                     o.data_ptr(), alpha, ACTIVATIONS[activation], wptr, wbytes, s))
        return o

    return enqueue(dev, stream, go)
