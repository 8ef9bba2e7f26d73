"""GPU tests of the product with 4-bit weights at the ends of its range: weights
past fp16, weights that fp16 rounds, and more rows than one launch has."""
import numpy as np
import pytest
import torch

import w4_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gsr(native):
    import tiled_dense_gemm_scale_amd as g

    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return g


def say(msg):
    print("[gpu] " + msg, flush=True)


def handle(gsr, q, s, z, K, group):
    return gsr.W4(ref.pack(q).to(DEV), torch.from_numpy(s).to(DEV), None if z is None else torch.from_numpy(z).to(DEV), K, group)


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("case", [(1025, 2048, 1024, 128), (1500, 1000, 4096, 64), (16000, 333, 1001, 32), (400000, 3, 64, 32)],
                         ids=lambda c: "x".join(map(str, c)))
def test_weights_past_fp16(gsr, case, zeros):
    """Many rows with the weights' values in the workspace: a column with a weight
    that fp16 does not hold has the formula's values all the same, and no other
    column's bits change; a scale that is not finite stays in its column."""
    M, N, K, group = case
    rng = np.random.default_rng(M + zeros)
    G = -(-K // group)
    q = rng.integers(0, 16, (K, N))
    s = ((0.5 + rng.random((G, N))) * 0.2).astype(np.float16)
    z = rng.integers(0, 16, (G, N)).astype(np.uint8) if zeros else None
    at = np.arange(N)
    s[0, at % 7 == 2], s[G - 1, at % 11 == 5] = 9360.0, -60000.0  # 7 x 9360 = 65520, the first past fp16
    s[G // 2, at % 13 == 4] = 8188.0                             # 8 x 8188 = 65504 stays
    if zeros:
        z[G - 1, at % 17 == 8], s[G - 1, at % 17 == 8] = 255, 300.0
    f = ref.values(q, s, z, group)
    past = (np.abs(f) >= 65520).any(0)
    assert past.any() and (N == 3 or not past.all())
    if N > 3:
        s[1, N - 2] = np.nan if zeros else np.inf
    odd = ~np.isfinite(s).all(0)
    w = handle(gsr, q, s, z, K, group)
    a, bias = torch.randn(M, K, device=DEV).half(), torch.randn(N, device=DEV).half()
    nbytes = gsr.w4_workspace_bytes(M, N, K)
    assert nbytes == 512 + 2 * K * N  # the values are written out
    alpha = 2.0 ** -9
    say(f"w4 past fp16 {case} zeros={zeros}: {int(past.sum())} of {N} columns")
    got = gsr.gemm_w4(a, w, gsr.new_workspace(nbytes), bias=bias, alpha=alpha, activation="none")
    dense = gsr.gemm_scale_bias_act(a, gsr.dequantize_w4(w), bias, alpha, "none")
    same = torch.from_numpy(~past & ~odd & (np.abs(f) <= 65504).all(0)).to(DEV)
    # a column whose codes could stand for a weight past fp16 may keep its weights too
    z64 = 8.0 if z is None else z.astype(np.float64)
    near = (np.abs(s.astype(np.float64)) * np.maximum(z64, 15.0 - z64) >= 65520).any(0)
    same &= torch.from_numpy(~near).to(DEV)
    assert torch.equal(got[:, same], dense[:, same])
    got = got.cpu().numpy().astype(np.float64)
    assert not np.isfinite(got[:, odd]).any()
    a64, b64 = a.cpu().numpy().astype(np.float64), bias.cpu().numpy().astype(np.float64)
    v, top = alpha * (a64 @ f) + b64, alpha * (np.abs(a64) @ np.abs(f)) + np.abs(b64)
    # half an fp16 step of each weight where the column's are rounded
    rounded = np.where(past, 0.0, alpha * (np.abs(a64) @ ref.half_step(f)))
    slack = ref.sum_slack(K + G + 2, top) + rounded
    bound = slack + ref.half_step(np.abs(v) + slack)
    cols = ~odd & (np.abs(v) + bound < 65504).all(0)
    assert past[cols].any()
    err = np.abs(got - v)[:, cols]
    assert (err <= bound[:, cols]).all(), f"{np.count_nonzero(~(err <= bound[:, cols]))} of {err.size}"


def unrounded_inputs(gsr, M, N, K, group, zeros):
    """Weights of 12 and 13 bits, (q - z) (1024 + c) / 1024 with odd q - z up to 7 and
    q constant in a column; a row of A takes one weight and gives back another, so
    the output is (q - z) (c1 - c2) / 1024 exactly."""
    rng = np.random.default_rng(M + N + K)
    G = -(-K // group)
    c = rng.integers(0, 128, (G, N))
    s = ((1024 + c) / 1024.0).astype(np.float16)
    zero = 8 if not zeros else 6
    q = np.broadcast_to(zero + rng.choice([-5, -3, 5, 7], N), (K, N))
    z = np.full((G, N), zero, np.uint8) if zeros else None
    a = np.zeros((M, K), np.float16)
    for m in range(M):
        k1, k2 = rng.choice(K, 2, replace=False)
        a[m, k1], a[m, k2] = 1.0, -1.0
    want = a.astype(np.float64) @ ref.values(q, s, z, group)
    assert np.array_equal(want, want.astype(np.float16))
    return torch.from_numpy(a).to(DEV), handle(gsr, q, s, z, K, group), want


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("case", [(2, 4096, 512, 128), (17, 1000, 1000, 32), (33, 514, 1024, 64), (64, 11008, 1024, 128),
                                  (100, 4096, 4096, 256), (130, 4096, 1030, 128), (150, 2048, 4093, 32)],
                         ids=lambda c: "x".join(map(str, c)))
def test_weights_of_a_few_rows_are_not_rounded(gsr, case, zeros):
    M, N, K, group = case
    a, w, want = unrounded_inputs(gsr, M, N, K, group, zeros)
    nbytes = gsr.w4_workspace_bytes(M, N, K)
    assert nbytes != 512 + 2 * K * N  # nothing is written out
    for ws in (gsr.new_workspace(nbytes), None):
        say(f"w4 unrounded {case} zeros={zeros} workspace={ws is not None}")
        got = gsr.gemm_w4(a, w, ws, activation="none").cpu().numpy()
        assert np.array_equal(got, want), f"{np.count_nonzero(got != want)} of {want.size} differ"


@pytest.mark.parametrize("case", [(1025, 2048, 1024, 128), (1500, 1000, 1000, 64), (4000, 333, 1001, 32)],
                         ids=lambda c: "x".join(map(str, c)))
def test_rounding_of_many_rows_is_the_callers_choice(gsr, case):
    """The same workspace with and without the weights rounded."""
    M, N, K, group = case
    a, w, want = unrounded_inputs(gsr, M, N, K, group, True)
    nbytes = 512 + 2 * K * N
    ws = gsr.new_workspace(max(nbytes, gsr.w4_workspace_bytes(M, N, K)))
    say(f"w4 choice of rounding {case}")
    got = gsr.gemm_w4(a, w, ws, activation="none", round_weights=False).cpu().numpy()
    assert np.array_equal(got, want), f"{np.count_nonzero(got != want)} of {want.size} differ"
    if gsr.w4_workspace_bytes(M, N, K) == nbytes:
        got = gsr.gemm_w4(a, w, ws, activation="none")
        assert torch.equal(got, gsr.gemm_scale_bias_act(a, gsr.dequantize_w4(w), activation="none"))
    # in a product whose rows are few nothing changes, its K split included
    b, v, few = unrounded_inputs(gsr, 5, 512, 4096, 128, True)
    ws = gsr.new_workspace(gsr.w4_workspace_bytes(5, 512, 4096))
    assert torch.equal(gsr.gemm_w4(b, v, ws, activation="none"), gsr.gemm_w4(b, v, ws, activation="none", round_weights=False))
    assert int(ws.count_nonzero()) > 0 and int(ws[:512].count_nonzero()) == 0  # parts met there


@pytest.mark.parametrize("N", [1, 70])
def test_more_rows_than_a_launch_has(gsr, N):
    """More tiles than the 2^23 workgroups of 512 threads that a launch can have,
    without a workspace: every row, and nothing behind the last."""
    K, group = 2, 32
    M = (2 ** 23 // -(-N // 64)) * 16 + 33
    q = np.arange(K * N).reshape(K, N) % 16
    s = np.full((1, N), 0.5, np.float16)
    w = handle(gsr, q, s, None, K, group)
    a = torch.randint(-2, 3, (M, K), device=DEV, dtype=torch.int8).half()
    f = torch.from_numpy(ref.values(q, s, None, group)).to(DEV).float()
    buf = torch.full((M * N + 64,), 9.0, dtype=torch.float16, device=DEV)
    say(f"w4 {M} rows of {N}")
    gsr.gemm_w4(a, w, activation="none", c=buf[:M * N].view(M, N))
    for m in range(0, M, 2 ** 24):
        part = a[m:m + 2 ** 24].float()
        want = (part[:, :1] * f[:1] + part[:, 1:] * f[1:]).half()
        assert torch.equal(buf[m * N:m * N + want.numel()].view(-1, N), want), m
    assert bool((buf[M * N:] == 9.0).all())
