"""A whole layer of routed experts for a few tokens in two launches, with the
experts in fp16 or in 4 bits.  For serving: autograd records nothing, and there
is no gradient here.  expert_mlp takes any number of tokens, of experts in fp16
without a gate (and without SiLU); for more than 64 tokens 4-bit experts are
dequantize_w4's values, and a gate is a second gemm_grouped and the caller's own
product of the two."""
from __future__ import annotations

from typing import Optional, Union

import torch

from . import _native
from ._native import expert_few_workspace_bytes
from .quantized import W4, check_w4
from .routing import ACTIVATIONS as _PRODUCT_ACTIVATIONS
from .routing import enqueue, matrix, need, output, workspace_of

__all__ = ["expert_mlp_few", "expert_few_workspace_bytes"]

ACTIVATIONS = dict(_PRODUCT_ACTIVATIONS, silu=_native.GSR_ACT_SILU)


def _weights(name, w, bias, experts, rows, index):
    """The matrices (experts, rows, any) of `w` and their bias as a C struct,
    and their columns (experts None: any number, returned too)."""
    if isinstance(w, W4):
        if not isinstance(w.codes, torch.Tensor) or w.codes.dim() != 3:
            raise ValueError(f"{name}.codes must have three dimensions")
        E = w.codes.shape[0] if experts is None else experts
        K, N, data, scales, zeros = check_w4(name, w, index, (E,))
        group = w.group
    else:
        data, scales, zeros, group = matrix(name, w, torch.float16, 3, index), 0, 0, 0
        E, K, N = w.shape
    if K != rows or (experts is not None and E != experts):
        raise ValueError(f"{name} must have shape ({'*' if experts is None else experts}, {rows}, *), got ({E}, {K}, {N})")
    b = need("bias_" + name, bias, torch.float16, (E, N), index) if bias is not None else 0
    return _native.GsrWeights(data or None, scales or None, zeros or None, b or None, group), E, N


def expert_mlp_few(x: torch.Tensor, ids: torch.Tensor, weights: Optional[torch.Tensor], up: Union[torch.Tensor, W4],
                   down: Union[torch.Tensor, W4], workspace: torch.Tensor, gate: Union[torch.Tensor, W4, None] = None,
                   bias_up: Optional[torch.Tensor] = None, bias_gate: Optional[torch.Tensor] = None,
                   bias_down: Optional[torch.Tensor] = None, activation: str = "gelu",
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * (h @ down[e] + bias_down[e]) with
    e = ids[t, j] and h = act(x[t] @ up[e] + bias_up[e]), or with a gate
    h = act(x[t] @ gate[e] + bias_gate[e]) * (x[t] @ up[e] + bias_up[e]); choices
    whose id names no expert are left out.  x (T, H) fp16 with T <= 64, ids (T, k)
    int32 or int64 with T k <= 1024, weights (T, k) float32 or None (ones); up and
    gate (E, H, F) and down (E, F, O) fp16, or all of them W4 of those sizes, up
    and gate of one group; biases (E, F), (E, F) and (E, O) fp16 or None; act
    "relu", "gelu" (tanh form), "silu" or "none".  Sums are fp32; h is kept to
    within 2^-22 of itself or 2^-35, whichever is more, and becomes an infinity past
    fp16's range.  workspace: new_workspace(expert_few_workspace_bytes(T, k, E, F, O)), one
    per call that may run at the same time.  Returns out (T, O)."""
    matrix("x", x, torch.float16, 2)
    (T, H), dev = x.shape, x.get_device()
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be a tensor of shape ({T}, k)")
    iptr = matrix("ids", ids, ids.dtype if ids.dtype in (torch.int32, torch.int64) else torch.int32, 2, dev)
    k = ids.shape[1]
    wptr = need("weights", weights, torch.float32, ids.shape, dev) if weights is not None else 0
    u, E, F = _weights("up", up, bias_up, None, H, dev)
    g = None
    if gate is not None:
        g, _, Fg = _weights("gate", gate, bias_gate, E, H, dev)
        if Fg != F:
            raise ValueError(f"gate must have {F} columns as up has, got {Fg}")
    elif bias_gate is not None:
        raise ValueError("bias_gate without a gate")
    d, _, O = _weights("down", down, bias_down, E, F, dev)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    ws, wbytes = workspace_of(workspace, dev)

    def go(s):
        o = output("out", out, torch.float16, (T, O), x)
        _native.check(_native.expert_mlp_few(T, k, E, H, F, O, x.data_ptr(), iptr, ids.element_size(), wptr, u, g, d,
                                             ACTIVATIONS[activation], o.data_ptr(), ws, wbytes, s))
        return o

    return enqueue(dev, stream, go)
