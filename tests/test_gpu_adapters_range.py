"""GPU tests of the product with low-rank adapters whose inner sums are far
from 1: alpha brings the outputs back into fp16's range."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CONFIGS = [-1, 21, 22, 28, 31, 32]


@pytest.fixture(scope="module")
def gsr(native):
    import tiled_dense_gemm_scale_amd as g

    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return g


@pytest.mark.parametrize("power", [-100, -60, -41, 100, 117, 124])
@pytest.mark.parametrize("shape", [(40, 64, 256, 3, 16), (150, 136, 264, 4, 72), (33, 101, 77, 3, 5)],
                         ids=lambda s: "x".join(map(str, s)))
def test_inner_sums_over_the_range_of_fp32(gsr, shape, power):
    """Scales of 2^power: powers of two, so the outputs keep the bound that they
    have at power 0.  |t| < 8 and |t Lb| < 8 at power 0 (checked), so at 2^124
    both stay below fp32's 2^128."""
    M, N, K, L, R = shape
    g = torch.Generator().manual_seed(M + R)
    n = lambda std, *s: (torch.randn(*s, generator=g) * std).half()
    a, b = n(1.0, M, K), torch.zeros(K, N, dtype=torch.float16)
    la, lb = n(K ** -0.5, L, R, K), n(R ** -0.5, L, N, R)
    ids = np.random.default_rng(M).integers(-1, L, M).astype(np.int32)
    factor = np.array([1.0, -0.5, 0.75, 0.3125])[:L]
    u = 2.0 ** -24
    want, slack = np.zeros((M, N)), np.full((M, N), 2.0 ** -25)
    for l in range(L):
        m = np.flatnonzero(ids == l)
        x, w, v = a.double().numpy()[m], la[l].double().numpy(), lb[l].double().numpy()
        t = factor[l] * (x @ w.T)
        want[m] = t @ v.T
        terr = (K + 40) * u * abs(factor[l]) * (np.abs(x) @ np.abs(w).T) + 2.0 ** -23 * np.abs(t).max(1, keepdims=True)
        off = (terr + (2 * R + 4) * u * np.abs(t)) @ np.abs(v).T + 4 * u * np.abs(want[m])
        slack[m] += off + 2.0 ** -11 * (np.abs(want[m]) + off)
        assert np.abs(t).max() < 8 and np.abs(want[m]).max() < 8 and (np.abs(t) @ np.abs(v).T).max() < 16
    scales = torch.tensor(factor * 2.0 ** power, dtype=torch.float32)
    ws = gsr.new_workspace(max(gsr.adapter_workspace_bytes(M, N, K, R), 512))
    for config in CONFIGS:
        print(f"[gpu] inner sums of 2^{power} {shape} config={config}", flush=True)
        c = gsr.gemm_adapters(a.to(DEV), b.to(DEV), la.to(DEV), lb.to(DEV), torch.from_numpy(ids).to(DEV), ws,
                              scales=scales.to(DEV), alpha=2.0 ** -power, activation="none", config_id=config)
        err = np.abs(c.cpu().double().numpy() - want)
        assert np.all(err <= slack), f"{np.count_nonzero(~(err <= slack))} values, worst {np.nanmax(err / slack)}"
