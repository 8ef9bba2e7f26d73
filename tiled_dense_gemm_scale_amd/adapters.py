"""The fused product with low-rank adapters: a batch whose rows belong to
requests with adapters of their own, against one shared weight matrix."""
from __future__ import annotations

from typing import Optional

import torch

from . import _native
from ._native import adapter_workspace_bytes
from .routing import ACTIVATIONS, check, check_workspace, on_stream

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
    check("a", a, torch.float16, (None, None), None)
    dev, M, K = a.device, int(a.shape[0]), int(a.shape[1])
    check("b", b, torch.float16, (K, None), dev)
    N = int(b.shape[1])
    check("lora_a", lora_a, torch.float16, (None, None, K), dev)
    L, R = int(lora_a.shape[0]), int(lora_a.shape[1])
    check("lora_b", lora_b, torch.float16, (L, N, R), dev)
    check("ids", ids, torch.int32, (M,), dev)
    if scales is not None:
        check("scales", scales, torch.float32, (L,), dev)
    if bias is not None:
        check("bias", bias, torch.float16, (N,), dev)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    wptr, wbytes = check_workspace(workspace, dev)
    with on_stream(dev, stream) as s:
        c = torch.empty((M, N), dtype=torch.float16, device=dev) if c is None else c
        check("c", c, torch.float16, (M, N), dev)
        st = _native.gemm_adapters_scale_bias_act(
            M, N, K, a.data_ptr(), b.data_ptr(), bias.data_ptr() if bias is not None else 0, c.data_ptr(), L, R,
            lora_a.data_ptr(), lora_b.data_ptr(), ids.data_ptr(), scales.data_ptr() if scales is not None else 0, alpha,
            ACTIVATIONS[activation], wptr, wbytes, s, config_id, splits)
    _native.check(st)
    return c
