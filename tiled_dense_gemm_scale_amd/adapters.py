"""The fused product with low-rank adapters: a batch whose rows belong to
requests with adapters of their own, against one shared weight matrix.  For
serving: autograd records nothing, and there is no gradient here."""
from __future__ import annotations

from typing import Optional

import torch

from . import _native
from ._native import adapter_workspace_bytes
from .routing import ACTIVATIONS, enqueue, matrix, need, output, workspace_of

__all__ = ["gemm_adapters", "adapter_workspace_bytes"]


def gemm_adapters(a: torch.Tensor, b: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor, ids: torch.Tensor,
                  workspace: torch.Tensor, scales: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  alpha: float = 1.0, activation: str = "relu", c: Optional[torch.Tensor] = None, stream=None,
                  config_id: int = -1, splits: int = 0) -> torch.Tensor:
    """c[m] = act(alpha * (a[m] @ b + scales[l] * (a[m] @ lora_a[l].T) @
    lora_b[l].T) + bias) with l = ids[m]; rows whose id is outside [0, L) take
    a[m] @ b alone.  a (M, K), b (K, N), lora_a (L, R, K), lora_b (L, N, R) and
    bias (N,) or None are fp16, ids (M,) int32, scales (L,) float32 or None
    (ones); R is at most 256.  workspace: new_workspace(
    adapter_workspace_bytes(M, N, K, R)), one per call that may run at the same
    time.  Returns c (M, N)."""
    matrix("a", a, torch.float16, 2)
    (M, K), dev = a.shape, a.get_device()
    matrix("b", b, torch.float16, 2, dev)
    matrix("lora_a", lora_a, torch.float16, 3, dev)
    if b.shape[0] != K or lora_a.shape[2] != K:
        raise ValueError(f"b and lora_a must have shapes ({K}, *) and (*, *, {K}), got {tuple(b.shape)} and {tuple(lora_a.shape)}")
    N = b.shape[1]
    L, R = lora_a.shape[0], lora_a.shape[1]
    lb = need("lora_b", lora_b, torch.float16, (L, N, R), dev)
    iptr = need("ids", ids, torch.int32, (M,), dev)
    sptr = need("scales", scales, torch.float32, (L,), dev) if scales is not None else 0
    bias_ptr = need("bias", bias, torch.float16, (N,), dev) if bias is not None else 0
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    wptr, wbytes = workspace_of(workspace, dev)

    def go(s):
        o = output("c", c, torch.float16, (M, N), a)
        _native.check(_native.gemm_adapters_scale_bias_act(
            M, N, K, a.data_ptr(), b.data_ptr(), bias_ptr, o.data_ptr(), L, R, lora_a.data_ptr(), lb, iptr, sptr, alpha,
            ACTIVATIONS[activation], wptr, wbytes, s, config_id, splits))
        return o

    return enqueue(dev, stream, go)
