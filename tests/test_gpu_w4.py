"""GPU tests of the 4-bit weights against their definitions in 64 bits on the
host: codes and scales exactly, values bit for bit, products of whole numbers
bit for bit and of normal values within the bound of their sums."""
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


def bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy()


def matrix(rng, K, N, kind):
    """fp16 values: normal ones of uneven columns, or hard ones."""
    b = rng.standard_normal((K, N)) * np.exp(rng.standard_normal(N))
    if kind == "offset":
        b = np.abs(b) + 0.5
    elif kind == "small":
        b = b * 2.0 ** -20
    elif kind == "large":
        b = np.clip(b * 4e4, -65504, 65504)
    elif kind == "ties":  # many values halfway between codes
        b = rng.integers(-15, 16, (K, N)) * 0.5 * 2.0 ** rng.integers(-4, 4, N)
    elif kind == "zero":
        b = b * (rng.random(N) < 0.5)
    return b.astype(np.float16)


QUANT = [(1, 1, 32), (8, 3, 32), (32, 64, 32), (33, 65, 32), (200, 130, 64), (128, 257, 128), (129, 8, 128), (515, 77, 256),
         (999, 1001, 32), (1000, 4, 1024), (4096, 132, 128), (7, 40, 128)]


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("kind", ["normal", "offset", "small", "large", "ties", "zero"])
@pytest.mark.parametrize("case", QUANT, ids=lambda c: "x".join(map(str, c)))
def test_quantize_and_back(gsr, case, kind, zeros):
    K, N, group = case
    b = matrix(np.random.default_rng(K * 7 + N), K, N, kind)
    say(f"quantize {case} {kind} zeros={zeros}")
    w = gsr.quantize_w4(torch.from_numpy(b).to(DEV), group, zeros=zeros)
    q, s, z = ref.quantize(b, group, zeros)
    assert np.array_equal(w.scales.cpu().numpy().view(np.uint16), s.view(np.uint16))
    assert (w.zeros is None) == (not zeros)
    if zeros:
        assert np.array_equal(w.zeros.cpu().numpy().astype(np.int64), z)
    assert np.array_equal(ref.unpack(w.codes, K), q)
    want = ref.values(q, s, z, group).astype(np.float16)
    assert np.array_equal(bits(gsr.dequantize_w4(w)), want.view(np.int16))


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
def test_quantize_stack_and_odd_addresses(gsr, zeros):
    """Several matrices, and one that starts on an odd element."""
    E, K, N, group = 3, 70, 37, 32
    b = matrix(np.random.default_rng(5), E * K, N, "normal").reshape(E, K, N)
    say("quantize stack")
    w = gsr.quantize_w4(torch.from_numpy(b).to(DEV), group, zeros=zeros)
    back = gsr.dequantize_w4(w)
    buf = torch.zeros(K * N + 1, dtype=torch.float16, device=DEV)
    for e in range(E):
        buf[1:].view(K, N).copy_(torch.from_numpy(b[e]))
        one = gsr.quantize_w4(buf[1:].view(K, N), group, zeros=zeros)
        assert torch.equal(one.codes, w.codes[e]) and torch.equal(one.scales, w.scales[e])
        out = torch.full((K * N + 2,), 3.0, dtype=torch.float16, device=DEV)
        gsr.dequantize_w4(one, out=out[1:-1].view(K, N))
        assert torch.equal(out[1:-1].view(K, N), back[e]) and out[0] == 3.0 and out[-1] == 3.0


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
def test_quantize_nonfinite(gsr, zeros):
    """A group with an infinity or NaN has the scale NaN, its neighbours their own."""
    K, N, group = 64, 6, 32
    b = matrix(np.random.default_rng(1), K, N, "normal")
    b[3, 1], b[40, 2], b[5, 4] = np.inf, np.nan, -np.inf
    say("quantize non-finite")
    w = gsr.quantize_w4(torch.from_numpy(b).to(DEV), group, zeros=zeros)
    s = w.scales.cpu().numpy()
    want = np.zeros((2, N), bool)
    want[0, 1] = want[1, 2] = want[0, 4] = True
    assert np.array_equal(np.isnan(s), want)
    back = gsr.dequantize_w4(w).cpu().numpy()
    assert np.array_equal(np.isnan(back), np.repeat(want, group, 0))


def test_quantize_nothing(gsr):
    say("quantize empty")
    for shape in ((0, 5), (5, 0), (0, 4, 4)):
        w = gsr.quantize_w4(torch.empty(*shape, dtype=torch.float16, device=DEV))
        assert tuple(gsr.dequantize_w4(w).shape) == shape


# ---- the product ---------------------------------------------------------------------

def weights(rng, K, N, group, zeros, whole):
    q = rng.integers(0, 16, (K, N))
    G = -(-K // group)
    s = 2.0 ** rng.integers(-2, 3, (G, N)) if whole else (0.5 + rng.random((G, N))) * 0.2
    z = rng.integers(0, 16, (G, N)).astype(np.uint8) if zeros else None
    return q, s.astype(np.float16), z


def handle(gsr, q, s, z, K, group):
    """codes past K hold other bits"""
    words = ref.pack(q)
    if K % 8:
        words[-1] |= torch.from_numpy(np.full(words.shape[-1], (0xffffffff << (4 * (K % 8))) & 0xffffffff, np.uint32).view(np.int32))
    return gsr.W4(words.to(DEV), torch.from_numpy(s).to(DEV), None if z is None else torch.from_numpy(z).to(DEV), K, group)


SHAPES = [(1, 1, 1, 32), (1, 64, 128, 32), (1, 4096, 4096, 128), (2, 3, 40, 32), (3, 100, 129, 64), (5, 67, 1000, 128),
          (7, 1001, 517, 32), (15, 256, 2048, 256), (16, 1000, 1024, 64), (17, 300, 4093, 32), (31, 64, 11008, 128),
          (33, 514, 777, 64), (48, 132, 600, 1024), (61, 1001, 1093, 32), (64, 257, 1025, 128), (65, 130, 300, 64),
          (130, 301, 517, 128), (257, 264, 512, 32), (513, 520, 640, 128)]


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "x".join(map(str, c)))
def test_product_of_whole_numbers(gsr, case, zeros):
    """Whole rows of A and scales that are powers of two: every sum is exact, so
    the outputs are the fp16 values nearest the formula's, with and without a
    workspace."""
    M, N, K, group = case
    rng = np.random.default_rng(M + N + K)
    q, s, z = weights(rng, K, N, group, zeros, True)
    a = rng.integers(-2, 3, (M, K)).astype(np.float16)
    bias = rng.integers(-50, 50, N).astype(np.float16)
    v = a.astype(np.float64) @ ref.values(q, s, z, group)
    assert np.abs(v).max() * 4 < 2 ** 24  # steps of 1/4
    w = handle(gsr, q, s, z, K, group)
    A, B = torch.from_numpy(a).to(DEV), torch.from_numpy(bias).to(DEV)
    ws = gsr.new_workspace(gsr.w4_workspace_bytes(M, N, K))
    for act, alpha, use in (("none", 0.5, None), ("relu", -0.25, B)):
        want = ref.act64(alpha * v + (0.0 if use is None else bias.astype(np.float64)), act)
        with np.errstate(over="ignore"):
            want = want.astype(np.float16) + np.float16(0)  # +0
        for work in (ws, None):
            say(f"w4 whole {case} zeros={zeros} {act} workspace={work is not None}")
            got = gsr.gemm_w4(A, w, work, bias=use, alpha=alpha, activation=act).cpu().numpy()
            assert np.array_equal(got, want), f"{np.count_nonzero(got != want)} of {want.size} differ"
    assert int(ws[:512].count_nonzero()) == 0


def test_narrow_products(gsr):
    """Every N and K up to 18 and around a block of columns, with and without zero
    points; nothing written behind the last row."""
    rng = np.random.default_rng(6)
    for N in list(range(1, 19)) + [63, 64, 65, 66, 68, 127, 129]:
        for M, K, zeros in ((5, 40, False), (21, 300, True), (3, N, True)):
            q, s, z = weights(rng, K, N, 32, zeros, True)
            a, bias = rng.integers(-2, 3, (M, K)).astype(np.float16), rng.integers(-50, 50, N).astype(np.float16)
            want = (a.astype(np.float64) @ ref.values(q, s, z, 32) + bias).astype(np.float16)
            buf = torch.full((M * N + 64,), 5.0, dtype=torch.float16, device=DEV)
            say(f"w4 narrow {M}x{N}x{K} zeros={zeros}")
            got = gsr.gemm_w4(torch.from_numpy(a).to(DEV), handle(gsr, q, s, z, K, 32), bias=torch.from_numpy(bias).to(DEV),
                              activation="none", c=buf[:M * N].view(M, N))
            assert np.array_equal(got.cpu().numpy(), want), (M, N, K)
            assert bool((buf[M * N:] == 5.0).all()), (M, N, K)


@pytest.mark.parametrize("act", ["relu", "gelu", "none"])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "x".join(map(str, c)))
def test_product(gsr, case, act):
    M, N, K, group = case
    rng = np.random.default_rng(M + 3 * N + K)
    q, s, z = weights(rng, K, N, group, M % 2 == 0, False)
    a, bias = rng.standard_normal((M, K)).astype(np.float16), rng.standard_normal(N).astype(np.float16)
    alpha = K ** -0.5
    f = ref.values(q, s, z, group)
    a64 = a.astype(np.float64)
    top = alpha * (np.abs(a64) @ np.abs(f)) + np.abs(bias.astype(np.float64))
    v = alpha * (a64 @ f) + bias.astype(np.float64)
    # many rows take weights rounded to fp16: half a step each
    rounded = alpha * (np.abs(a64) @ ref.half_step(f)) if M > 16 else 0.0
    slack = ref.act_slack(ref.sum_slack(K + -(-K // group) + 2, top) + rounded, v, act)
    want = ref.act64(v, act)
    say(f"w4 {case} {act}")
    ws = gsr.new_workspace(gsr.w4_workspace_bytes(M, N, K))
    got = gsr.gemm_w4(torch.from_numpy(a).to(DEV), handle(gsr, q, s, z, K, group), ws, bias=torch.from_numpy(bias).to(DEV),
                      alpha=alpha, activation=act).cpu().numpy().astype(np.float64)
    err, bound = np.abs(got - want), slack + ref.half_step(np.abs(want) + slack)
    say(f"w4 {case} {act}: worst {float((err / bound).max()):.3f} of its bound, "
        f"{float(err.max() / np.abs(want).max()):.1e} of the largest output")
    assert (err <= bound).all()


@pytest.mark.parametrize("case", [(1025, 2048, 1024, 128), (1500, 1000, 4096, 64), (16000, 333, 1001, 32)], ids=lambda c: "x".join(map(str, c)))
def test_product_of_many_rows(gsr, case):
    """Many rows: the bits of the dense product with the weights' values, and the
    formula's within one more rounding; a workspace too small for the values keeps
    the weights as they are."""
    M, N, K, group = case
    rng = np.random.default_rng(M)
    q, s, z = weights(rng, K, N, group, True, False)
    w = handle(gsr, q, s, z, K, group)
    a, bias = torch.randn(M, K, device=DEV).half(), torch.randn(N, device=DEV).half()
    nbytes = gsr.w4_workspace_bytes(M, N, K)
    assert nbytes == 512 + 2 * K * N
    say(f"w4 many rows {case}")
    got = gsr.gemm_w4(a, w, gsr.new_workspace(nbytes), bias=bias, alpha=0.5, activation="gelu")
    assert torch.equal(got, gsr.gemm_scale_bias_act(a, gsr.dequantize_w4(w), bias, 0.5, "gelu"))
    f, a64 = ref.values(q, s, z, group), a.cpu().numpy().astype(np.float64)
    b64 = bias.cpu().numpy().astype(np.float64)
    v, top = 0.5 * (a64 @ f) + b64, 0.5 * (np.abs(a64) @ np.abs(f)) + np.abs(b64)
    for work, rounded in ((gsr.new_workspace(nbytes), 0.5 * (np.abs(a64) @ ref.half_step(f))), (gsr.new_workspace(nbytes - 1), 0.0)):
        slack = ref.act_slack(ref.sum_slack(K + -(-K // group) + 2, top) + rounded, v, "gelu")
        want = ref.act64(v, "gelu")
        err = np.abs(gsr.gemm_w4(a, w, work, bias=bias, alpha=0.5, activation="gelu").cpu().numpy().astype(np.float64) - want)
        assert (err <= slack + ref.half_step(np.abs(want) + slack)).all()


@pytest.mark.parametrize("shape", [(1, 4096, 512, 128), (9, 130, 300, 64), (40, 77, 333, 32), (70, 77, 333, 32)],
                         ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_product_at_odd_addresses(gsr, shape, offset):
    """A, scales, bias and C on odd elements, zeros on odd bytes, codes on a word;
    values beside C left alone; the same bits as aligned."""
    M, N, K, group = shape
    rng = np.random.default_rng(M)
    q, s, z = weights(rng, K, N, group, True, False)
    w = handle(gsr, q, s, z, K, group)
    a, bias = torch.randn(M, K, device=DEV).half(), torch.randn(N, device=DEV).half()
    ws = gsr.new_workspace(gsr.w4_workspace_bytes(M, N, K))

    def moved(t):
        buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device=DEV)
        out = buf[offset:offset + t.numel()].view(t.shape)
        out.copy_(t)
        return out

    say(f"w4 addresses {shape} +{offset}")
    base = gsr.gemm_w4(a, w, ws, bias=bias, activation="none")
    cbuf = torch.full((M * N + 8,), 3.0, dtype=torch.float16, device=DEV)
    c = cbuf[offset:offset + M * N].view(M, N)
    gsr.gemm_w4(moved(a), gsr.W4(moved(w.codes), moved(w.scales), moved(w.zeros), K, group), ws, bias=moved(bias),
                activation="none", c=c)
    assert torch.equal(c, base)
    assert bool((cbuf[:offset] == 3.0).all()) and bool((cbuf[offset + M * N:] == 3.0).all())


@pytest.mark.parametrize("M", [1, 20, 50, 100])
def test_nonfinite_rows_and_scales(gsr, M):
    """An infinity or NaN of A reaches its row alone, as the formula says (an
    infinity times the weight 0 is NaN), and a scale that is not finite its
    column alone."""
    K, N, group = 300, 140, 64
    rng = np.random.default_rng(M)
    q, s, z = weights(rng, K, N, group, True, True)
    a = rng.integers(-2, 3, (M, K)).astype(np.float16)
    a[0, 17] = np.inf
    if M > 1:
        a[M - 1, 299], a[M // 2, 64] = -np.inf, np.nan
    s[1, 5], s[4, 139] = np.inf, np.nan
    f = ref.values(q, np.where(np.isfinite(s), s, 1.0).astype(np.float16), z, group)
    with np.errstate(invalid="ignore"):
        want = (a.astype(np.float64)[:, :, None] * f[None]).sum(1)
    say(f"w4 non-finite M={M}")
    ws = gsr.new_workspace(gsr.w4_workspace_bytes(M, N, K))
    got = gsr.gemm_w4(torch.from_numpy(a).to(DEV), handle(gsr, q, s, z, K, group), ws, alpha=0.125,
                      activation="none").cpu().numpy()
    cols = np.ones(N, bool)
    cols[[5, 139]] = False
    assert not np.isfinite(got[:, ~cols]).any()
    assert np.array_equal(got[:, cols], (0.125 * want).astype(np.float16)[:, cols], equal_nan=True)


def test_zero_points_of_all_sizes(gsr):
    """Zero points are 8-bit values: 0 to 255."""
    M, N, K, group = 4, 256, 64, 32
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (K, N))
    z = np.stack([np.arange(256), np.arange(256)[::-1]]).astype(np.uint8)
    s = np.full((2, N), 0.25, np.float16)
    a = rng.integers(-2, 3, (M, K)).astype(np.float16)
    say("w4 zero points")
    got = gsr.gemm_w4(torch.from_numpy(a).to(DEV), handle(gsr, q, s, z, K, group), activation="none").cpu().numpy()
    assert np.array_equal(got, (a.astype(np.float64) @ ref.values(q, s, z, group)).astype(np.float16))


def test_small_values_keep_their_bits(gsr):
    """Subnormal A and scales: whole multiples of 2^-24 on both sides."""
    M, N, K, group = 3, 64, 96, 32
    rng = np.random.default_rng(3)
    q, z = rng.integers(0, 16, (K, N)), None
    s = (rng.integers(1, 8, (3, N)) * 2.0 ** -24).astype(np.float16)
    a = (rng.integers(-8, 9, (M, K)) * 2.0 ** -24).astype(np.float16)
    say("w4 subnormal")
    alpha = 2.0 ** 40
    got = gsr.gemm_w4(torch.from_numpy(a).to(DEV), handle(gsr, q, s, z, K, group), alpha=alpha, activation="none").cpu().numpy()
    assert np.array_equal(got, (alpha * (a.astype(np.float64) @ ref.values(q, s, z, group))).astype(np.float16))


def test_empty_products(gsr):
    say("w4 empty")
    w = handle(gsr, np.zeros((0, 5), np.int64), np.zeros((0, 5), np.float16), None, 0, 32)
    bias = torch.tensor([-1.0, 2.0, 0.0, 3.0, -4.0], dtype=torch.float16, device=DEV)
    a = torch.empty(3, 0, dtype=torch.float16, device=DEV)
    assert gsr.gemm_w4(a, w, bias=bias).cpu().tolist() == [[0.0, 2.0, 0.0, 3.0, 0.0]] * 3
    q, s, z = weights(np.random.default_rng(0), 40, 5, 32, False, True)
    assert tuple(gsr.gemm_w4(torch.empty(0, 40, dtype=torch.float16, device=DEV), handle(gsr, q, s, z, 40, 32)).shape) == (0, 5)


def test_output_past_2_31_bytes(gsr):
    """C of more than 2^31 bytes, with the weights' values in the workspace (the
    rows then in runs below that) and without a workspace: whole numbers."""
    M, N, K, group = 70001, 16384, 64, 32
    rng = np.random.default_rng(2)
    q, s, z = weights(rng, K, N, group, True, True)
    w = handle(gsr, q, s, z, K, group)
    a = torch.randint(-2, 3, (M, K), device=DEV).half()
    f = torch.from_numpy(ref.values(q, s, z, group)).to(DEV).float()
    nbytes = gsr.w4_workspace_bytes(M, N, K)
    assert nbytes == 512 + 2 * K * N
    c = torch.empty(M, N, dtype=torch.float16, device=DEV)
    for ws in (gsr.new_workspace(nbytes), None):
        say(f"w4 large output workspace={ws is not None}")
        c.fill_(9.0)
        gsr.gemm_w4(a, w, ws, alpha=0.5, activation="none", c=c)
        for m in range(0, M, 10000):
            want = ((a[m:m + 10000].float() @ f) * 0.5).half()
            assert torch.equal(c[m:m + 10000], want), m


def test_captured_product_of_many_rows(gsr):
    """The weights' values and the dense product in a graph, replayed on new rows
    and new weights beside eager calls in the same workspace."""
    M, N, K, group = 1100, 2048, 1024, 128
    rng = np.random.default_rng(5)
    q, s, z = weights(rng, K, N, group, True, False)
    w = handle(gsr, q, s, z, K, group)
    ws = gsr.new_workspace(max(gsr.w4_workspace_bytes(M, N, K), gsr.w4_workspace_bytes(4, N, K)))
    a, c = torch.randn(M, K, device=DEV).half(), torch.empty(M, N, dtype=torch.float16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gsr.gemm_w4(a, w, ws, c=c, activation="gelu", alpha=0.1, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("w4 capture of many rows")
    with torch.cuda.graph(graph, stream=side):
        gsr.gemm_w4(a, w, ws, c=c, activation="gelu", alpha=0.1)
    for i in range(4):
        a.copy_(torch.randn(M, K, device=DEV).half())
        w.codes.random_(-2 ** 31, 2 ** 31 - 1)
        want = gsr.gemm_w4(a, w, ws, activation="gelu", alpha=0.1)
        gsr.gemm_w4(a[:4].contiguous(), w, ws)
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want), i
    assert int(ws[:512].count_nonzero()) == 0


def test_streams_graphs_and_shared_workspace(gsr):
    """A captured call replays with the eager bits on new inputs, beside eager
    calls of other shapes and of the split product in the same workspace."""
    M, N, K, group = 5, 512, 4096, 128
    rng = np.random.default_rng(9)
    q, s, z = weights(rng, K, N, group, True, False)
    w = handle(gsr, q, s, z, K, group)
    b = torch.randn(K, N, device=DEV).half()
    ws = gsr.new_workspace(max(gsr.w4_workspace_bytes(M, N, K), gsr.workspace_bytes(M, N, K), gsr.w4_workspace_bytes(1, 70, 2000)))
    a = torch.randn(M, K, device=DEV).half()
    c = torch.empty(M, N, dtype=torch.float16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gsr.gemm_w4(a, w, ws, c=c, activation="none", stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("w4 capture")
    with torch.cuda.graph(graph, stream=side):
        gsr.gemm_w4(a, w, ws, c=c, activation="none")
    q2, s2, z2 = weights(rng, 2000, 70, 32, False, False)
    w2 = handle(gsr, q2, s2, z2, 2000, 32)
    for i in range(4):
        a.copy_(torch.randn(M, K, device=DEV).half())
        want = gsr.gemm_w4(a, w, ws, activation="none")
        gsr.gemm_scale_bias_act_ws(a, b, ws)
        gsr.gemm_w4(a[:1, :2000].contiguous(), w2, ws)
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want), i
    assert int(ws[:512].count_nonzero()) == 0
