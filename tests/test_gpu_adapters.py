"""GPU tests of the product with low-rank adapters against its definition in
64 bits on the host."""
import math

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


def say(msg):
    print("[gpu] " + msg, flush=True)


def activate(v, act):
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "gelu":
        return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def reference(a, b, la, lb, ids, scales, bias, alpha, act):
    """c and, per value, the bound on what the fp32 sums, the split of the
    inner sum (2^-23 of its row's largest value) and one fp16 rounding may be
    off by."""
    u = 2.0 ** -24
    a64, b64, la64, lb64 = (t.double().numpy() for t in (a, b, la, lb))
    K, R = b64.shape[0], la64.shape[1]
    v, off = a64 @ b64, (K + 2) * u * (np.abs(a64) @ np.abs(b64))
    for l in range(len(la64)):
        m = np.flatnonzero(ids == l)
        s = float(scales[l]) if scales is not None else 1.0
        t, tmag = s * (a64[m] @ la64[l].T), abs(s) * (np.abs(a64[m]) @ np.abs(la64[l]).T)
        terr = (K + 40) * u * tmag + (2.0 ** -23 * np.abs(t).max(1, keepdims=True) if R else 0.0)
        v[m] += t @ lb64[l].T
        off[m] += (terr + (2 * R + 4) * u * np.abs(t)) @ np.abs(lb64[l]).T
    v, off = alpha * v, abs(alpha) * off + 2 * u * np.abs(alpha * v)
    if bias is not None:
        v, off = v + bias.double().numpy(), off + u * np.abs(bias.double().numpy())
    # GELU: slope below 1.13, and a few 2^-22 of its own arithmetic
    off = 1.13 * off + (2.0 ** -20 * np.abs(v) if act == "gelu" else 0.0)
    c = activate(v, act)
    return c, off + 2.0 ** -11 * (np.abs(c) + off) + 2.0 ** -25


def within(name, got, ref, slack):
    err = np.abs(got - ref)
    assert np.all(err <= slack), f"{name}: {np.count_nonzero(~(err <= slack))} values, worst {np.nanmax(err / slack)}"
    say(f"{name}: worst error {float(np.max(err / slack)):.3f} of its bound")


def ids_of(kind, M, L, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "mixed":
        return rng.integers(-1, L + 1, M).astype(np.int32)
    if kind == "runs":
        return ((np.arange(M) * (L + 1)) // max(M, 1) - 1).astype(np.int32)
    return np.full(M, {"one": L - 1, "none": -1}[kind], np.int32)


def workspace(gsr, M, N, K, R, extra=0):
    return gsr.new_workspace(max(gsr.adapter_workspace_bytes(M, N, K, R), 512) + extra)


def counters_zero(ws):
    torch.cuda.synchronize()
    return bool((ws[:512] == 0).all().item())


def run(gsr, ws, a, b, la, lb, ids, scales=None, bias=None, **kw):
    d = lambda t: t.to(DEV) if t is not None else None
    return gsr.gemm_adapters(d(a), d(b), d(la), d(lb), torch.from_numpy(ids).to(DEV), ws, scales=d(scales), bias=d(bias), **kw)


def integer_case(M, N, K, L, R, seed):
    g = torch.Generator().manual_seed(seed)
    i = lambda n, *s: torch.randint(-n, n + 1, s, generator=g).half()
    return i(3, M, K), i(3, K, N), i(2, L, R, K), i(2, L, N, R)


@pytest.mark.parametrize("kind", ["mixed", "runs", "one", "none"])
@pytest.mark.parametrize("R", [1, 8, 16, 40, 64, 130])
@pytest.mark.parametrize("config", CONFIGS)
def test_integer_inputs_bitwise(gsr, config, R, kind):
    """Small integers: both sums are exact in fp32 and the inner one in its two
    halves, so any order gives the same bits."""
    M, N, K, L = 150, 136, 72, 7
    a, b, la, lb = integer_case(M, N, K, L, R, seed=R)
    ids = ids_of(kind, M, L)
    ws = workspace(gsr, M, N, K, R)
    say(f"adapters integers config={config} R={R} {kind}")
    scales = torch.tensor([1.0, 2.0, 0.5, -1.0, 1.0, 0.0, 4.0])
    c = run(gsr, ws, a, b, la, lb, ids, scales, alpha=0.0625, activation="none", config_id=config)
    ref, _ = reference(a, b, la, lb, ids, scales, None, 0.0625, "none")
    assert torch.equal(c.cpu(), torch.from_numpy(ref).half())
    assert counters_zero(ws)


@pytest.mark.parametrize("act", ["relu", "gelu", "none"])
@pytest.mark.parametrize("shape", [(1, 64, 512, 2, 8), (1, 4096, 4096, 4, 64), (16, 1000, 2056, 32, 16), (37, 101, 77, 3, 5),
                                   (300, 264, 520, 9, 16), (513, 300, 130, 4, 33), (33, 8, 8, 1, 1), (70, 1, 65, 2, 128),
                                   (2100, 136, 128, 5, 256)], ids=lambda s: "x".join(map(str, s)))
def test_normal_inputs(gsr, shape, act):
    """Every path (16-byte units or value by value for each operand) and rank
    class against the definition, rows of one batch mixed over adapters."""
    M, N, K, L, R = shape
    g = torch.Generator().manual_seed(M + N)
    n = lambda std, *s: (torch.randn(*s, generator=g) * std).half()
    a, b, la, lb = n(1.0, M, K), n(K ** -0.5, K, N), n(K ** -0.5, L, R, K), n(R ** -0.5, L, N, R)
    bias = n(1.0, N) if act != "none" else None
    scales = torch.rand(L, generator=g) * 2 if act != "relu" else None
    ids = ids_of("mixed", M, L, seed=N)
    ids[0] = 0
    ref, slack = reference(a, b, la, lb, ids, scales, bias, -0.75, act)
    ws = workspace(gsr, M, N, K, R)
    for config in CONFIGS:
        say(f"adapters normal {shape} {act} config={config}")
        c = run(gsr, ws, a, b, la, lb, ids, scales, bias, alpha=-0.75, activation=act, config_id=config)
        within(f"config {config}", c.cpu().double().numpy(), ref, slack)
        assert counters_zero(ws)


@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
@pytest.mark.parametrize("shape", [(65, 72, 10240, 5, 24), (100, 40, 9221, 3, 17), (400, 24, 9224, 2, 16), (1100, 24, 9224, 2, 16),
                                   (50, 40, 333, 5, 7), (90, 40, 333, 5, 7), (70, 33, 4097, 3, 5)],
                         ids=lambda s: "x".join(map(str, s)))
def test_inner_sums_of_long_and_odd_rows(gsr, shape, kind):
    """The inner sums in parts of K above 64 rows, and rows of odd length, where
    rows and adapters start at any 2-byte address: small sparse integers, whose
    sums are exact: |t| <= 6 (K / 16 + 3) < 2^12 is kept whole in its two
    halves, and |c| <= 9 * 643 + 24 * 2 * 2^12 < 2^18 in fp32."""
    M, N, K, L, R = shape
    a, b, la, lb = integer_case(M, N, K, L, R, seed=K)
    keep = (torch.arange(K) % 16 == 0) | (torch.arange(K) >= K - 3)  # at most K / 16 + 3 values of K count
    a, b, la = a * keep, b * keep[:, None], la * keep
    for shift in (0, 1):  # every operand also from an address that is no multiple of 4
        d = lambda t: torch.cat([torch.zeros(shift, dtype=t.dtype), t.flatten()]).to(DEV)[shift:].view(t.shape)
        ids = ids_of(kind, M, L)
        ws = workspace(gsr, M, N, K, R)
        say(f"adapters long rows {shape} {kind} shift={shift}")
        c = gsr.gemm_adapters(d(a), d(b), d(la), d(lb), torch.from_numpy(ids).to(DEV), ws, alpha=2.0 ** -7, activation="none")
        ref, _ = reference(a, b, la, lb, ids, None, None, 2.0 ** -7, "none")
        assert torch.equal(c.cpu(), torch.from_numpy(ref).half())
        assert counters_zero(ws)


@pytest.mark.parametrize("size", [1e-6, 1.0, 2000.0])
def test_inner_sums_of_any_size(gsr, size):
    """Inner sums above fp16's range and below its normal numbers keep their value."""
    M, N, K, L, R = 40, 64, 256, 3, 16
    g = torch.Generator().manual_seed(3)
    n = lambda std, *s: (torch.randn(*s, generator=g) * std).half()
    a, b = n(min(size, 30.0), M, K), torch.zeros(K, N, dtype=torch.float16)
    la, lb = n(max(min(size, 2000.0), 1e-3), L, R, K), n(1e-3 if size > 1 else 1.0, L, N, R)
    scales = torch.tensor([1.0, 10.0, 0.1])
    if size < 1:
        scales = scales * 1e3
    ids = ids_of("mixed", M, L)
    alpha = 1e-3 if size > 1 else 1.0
    ref, slack = reference(a, b, la, lb, ids, scales, None, alpha, "none")
    ws = workspace(gsr, M, N, K, R)
    for config in CONFIGS:
        say(f"adapters inner size {size} config={config}")
        c = run(gsr, ws, a, b, la, lb, ids, scales, alpha=alpha, activation="none", config_id=config)
        within(f"size {size}", c.cpu().double().numpy(), ref, slack)


def test_other_adapters_do_not_reach_a_row(gsr):
    """NaN and infinities in an adapter nobody or somebody else uses, and
    garbage in the workspace, leave a row's bits alone."""
    M, N, K, L, R = 90, 128, 64, 4, 16
    a, b, la, lb = integer_case(M, N, K, L, R, seed=2)
    ids = ids_of("mixed", M, L, seed=5)
    ref, _ = reference(a, b, la, lb, ids, None, None, 0.0625, "none")
    la[1, 3, 5], lb[1, :, 2], lb[2, 7] = float("nan"), float("inf"), float("nan")
    want = torch.from_numpy(ref).half()
    good = torch.from_numpy((ids != 1) & (ids != 2))
    for config in CONFIGS:
        ws = workspace(gsr, M, N, K, R)
        ws[512:] = 0xFF  # NaN patterns
        say(f"adapters NaN config={config}")
        c = run(gsr, ws, a, b, la, lb, ids, alpha=0.0625, activation="none", config_id=config).cpu()
        assert torch.equal(c[good], want[good])
        assert bool(torch.isnan(c[torch.from_numpy(ids == 1)]).all())
        two = c[torch.from_numpy(ids == 2)]
        assert bool(torch.isnan(two[:, 7]).all()) and torch.equal(two[:, :7], want[torch.from_numpy(ids == 2)][:, :7])


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 16])
@pytest.mark.parametrize("config", [21, 22])
def test_forced_splits(gsr, config, splits):
    M, N, K, L, R = 20, 200, 2048, 5, 24
    a, b, la, lb = integer_case(M, N, K, L, R, seed=splits)
    a, b = a.clamp(-1, 1), b.clamp(-1, 1)
    la = la.clamp(-1, 1)
    ids = ids_of("mixed", M, L, seed=splits)
    ref, _ = reference(a, b, la, lb, ids, None, None, 0.03125, "none")
    ws = workspace(gsr, M, N, K, R, extra=4 << 20)
    say(f"adapters forced split {splits} config={config}")
    for _ in range(3):
        c = run(gsr, ws, a, b, la, lb, ids, alpha=0.03125, activation="none", config_id=config, splits=splits)
        assert torch.equal(c.cpu(), torch.from_numpy(ref).half())
        assert counters_zero(ws)


@pytest.mark.parametrize("shape", [(1, 4096, 4096, 4, 64), (5, 200, 1032, 3, 16), (16, 1000, 2056, 16, 16),
                                   (17, 136, 5000, 2, 40), (33, 512, 4096, 5, 16), (64, 264, 520, 8, 8),
                                   (64, 72, 136, 2, 256)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("config", [21, 22])
def test_inner_sums_that_are_not_there_yet(gsr, native, config, shape):
    """The one-kernel form: a tile's workgroup that does not find the inner sums
    (looks = 0: it never does; 1: hardly) makes them itself, with the same
    bits, and the counters end at zero either way, call after call."""
    M, N, K, L, R = shape
    g = torch.Generator().manual_seed(M + K)
    n = lambda std, *s: (torch.randn(*s, generator=g) * std).half().to(DEV)
    a, b, la, lb = n(1.0, M, K), n(K ** -0.5, K, N), n(K ** -0.5, L, R, K), n(R ** -0.5, L, N, R)
    bias, scales = n(1.0, N), torch.rand(L, generator=g).to(DEV) + 0.5
    ids_host = ids_of("mixed", M, L, seed=K)
    ids_host[0] = L - 1
    ws = workspace(gsr, M, N, K, R, extra=4 << 20)
    stream = torch.cuda.current_stream().cuda_stream
    for splits in (0, 1, 3):
        bits = {}
        for ids_host in (ids_host, np.full(M, -1, np.int32)):
            ids = torch.from_numpy(ids_host).to(DEV)
            for looks in (-1, 0, 1, 0, -1):
                c = torch.full((M, N), float("nan"), dtype=torch.float16, device=DEV)
                say(f"adapters config={config} {shape} splits={splits} looks={looks}")
                assert native.gemm_adapters_scale_bias_act(
                    M, N, K, a.data_ptr(), b.data_ptr(), bias.data_ptr(), c.data_ptr(), L, R, la.data_ptr(), lb.data_ptr(),
                    ids.data_ptr(), scales.data_ptr(), -0.75, 1, ws.data_ptr(), ws.numel(), stream, config, splits, looks) == 0
                assert counters_zero(ws)
                key = int(ids_host.max())
                assert torch.equal(bits.setdefault(key, c).view(torch.int16), c.view(torch.int16))
            ref, slack = reference(a.cpu(), b.cpu(), la.cpu(), lb.cpu(), ids_host, scales.cpu(), bias.cpu(), -0.75, "gelu")
            within(f"splits {splits}", bits[key].cpu().double().numpy(), ref, slack)


def test_one_workspace_for_all_entry_points(gsr):
    """Products with and without adapters in turn on one workspace."""
    shapes = [(1, 4096, 4096), (64, 4096, 4096), (16, 1000, 2056), (300, 264, 520)]
    ws = gsr.new_workspace(max(max(gsr.workspace_bytes(*s), gsr.adapter_workspace_bytes(*s, 64)) for s in shapes))
    for i, (M, N, K) in enumerate(shapes + shapes):
        a, b, la, lb = integer_case(M, N, K, 3, 8, seed=i)
        a, b, la, lb = (t.clamp(-1, 1) for t in (a, b, la, lb))
        ids = ids_of("mixed", M, 3, seed=i)
        say(f"adapters and plain on one workspace {M}x{N}x{K}")
        ref, _ = reference(a, b, la, lb, ids, None, None, 0.125, "relu")
        c = run(gsr, ws, a, b, la, lb, ids, alpha=0.125, activation="relu")
        assert torch.equal(c.cpu(), torch.from_numpy(ref).half())
        plain = gsr.gemm_scale_relu_ws(a.to(DEV), b.to(DEV), 0.125, ws)
        assert torch.equal(plain.cpu(), torch.from_numpy(np.maximum(0.125 * (a.double().numpy() @ b.double().numpy()), 0)).half())
        assert counters_zero(ws)


def test_no_adapters_is_the_product(gsr):
    M, N, K = 33, 72, 264
    g = torch.Generator().manual_seed(1)
    a, b = torch.randn(M, K, generator=g).half().to(DEV), torch.randn(K, N, generator=g).half().to(DEV)
    ids, ws = torch.zeros(M, dtype=torch.int32, device=DEV), gsr.new_workspace(16)
    want = gsr.gemm_scale_bias_act(a, b, None, 0.5, "gelu")
    say("adapters: none in memory, rank 0")
    for L, R in ((0, 16), (3, 0)):
        c = gsr.gemm_adapters(a, b, torch.empty(L, R, K, dtype=torch.float16, device=DEV),
                              torch.empty(L, N, R, dtype=torch.float16, device=DEV), ids, ws, alpha=0.5, activation="gelu")
        assert torch.equal(c.view(torch.int16), want.view(torch.int16))
    # rows without one, among rows with: the bits of the product with the same configuration
    la, lb = torch.randn(2, 8, K, generator=g).half().to(DEV), torch.randn(2, N, 8, generator=g).half().to(DEV)
    ids[::2] = -1
    ws = workspace(gsr, M, N, K, 8)
    for config in CONFIGS[1:]:
        c = gsr.gemm_adapters(a, b, la, lb, ids, ws, alpha=0.5, activation="gelu", config_id=config)
        want = gsr.gemm_scale_bias_act(a, b, None, 0.5, "gelu", config_id=config)
        assert torch.equal(c[::2].view(torch.int16), want[::2].view(torch.int16))
        assert not torch.equal(c[1::2], want[1::2])


@pytest.mark.parametrize("which", ["a", "b", "la", "lb", "c"])
def test_less_aligned_operands(gsr, which):
    M, N, K, L, R = 45, 72, 136, 3, 16
    a, b, la, lb = integer_case(M, N, K, L, R, seed=4)
    ids = ids_of("mixed", M, L)
    want = torch.from_numpy(reference(a, b, la, lb, ids, None, None, 0.0625, "none")[0]).half()
    ws = workspace(gsr, M, N, K, R)
    for off in (1, 2, 4):
        def place(name, t):
            o = off if name == which else 0
            buf = torch.full((t.numel() + 8,), 3.0, dtype=torch.float16, device=DEV)
            v = buf[o:o + t.numel()].view(t.shape)
            v.copy_(t)
            return v, buf, o

        say(f"adapters {which} at +{2 * off} bytes")
        c, cbuf, o = place("c", torch.zeros(M, N))
        gsr.gemm_adapters(place("a", a)[0], place("b", b)[0], place("la", la)[0], place("lb", lb)[0],
                          torch.from_numpy(ids).to(DEV), ws, alpha=0.0625, activation="none", c=c)
        assert torch.equal(c.cpu(), want)
        host = cbuf.cpu()
        assert bool((host[:o] == 3.0).all()) and bool((host[o + M * N:] == 3.0).all())


def test_adapters_past_32_bit_offsets(gsr):
    """All adapters together above 2^31 bytes: the last one's values."""
    M, N, K, L, R = 5, 4096, 4096, 1100, 256  # La and Lb of 2.3 GB each
    la = torch.zeros(L, R, K, dtype=torch.float16, device=DEV)
    lb = torch.zeros(L, N, R, dtype=torch.float16, device=DEV)
    la[L - 1, R - 1, :4], lb[L - 1, :, R - 1] = 1.0, 2.0
    la[0, 0, :4], lb[0, :, 0] = 1.0, 3.0
    a = torch.ones(M, K, dtype=torch.float16, device=DEV)
    b = torch.zeros(K, N, dtype=torch.float16, device=DEV)
    ids = torch.tensor([L - 1, 0, -1, L, L - 1], dtype=torch.int32, device=DEV)
    say("adapters past 32-bit offsets")
    c = gsr.gemm_adapters(a, b, la, lb, ids, workspace(gsr, M, N, K, R), activation="none")
    assert bool((c == torch.tensor([8.0, 12.0, 0.0, 0.0, 8.0], device=DEV)[:, None]).all())


def test_streams_and_capture(gsr):
    """Two calls at once on two streams with a workspace each, then captured
    and replayed with new adapters and ids in the same buffers, eager work
    between the replays."""
    M, N, K, L, R = 16, 4096, 4096, 8, 16
    g = torch.Generator().manual_seed(6)
    n = lambda std, *s: (torch.randn(*s, generator=g) * std).half().to(DEV)
    a, b = [n(1.0, M, K) for _ in range(2)], n(K ** -0.5, K, N)
    la, lb = [n(K ** -0.5, L, R, K) for _ in range(2)], [n(R ** -0.5, L, N, R) for _ in range(2)]
    ids = [torch.from_numpy(ids_of("mixed", M, L, seed=s)).to(DEV) for s in (1, 2)]
    ws = [workspace(gsr, M, N, K, R) for _ in range(2)]
    torch.cuda.synchronize()
    say("adapters eager")
    want = [gsr.gemm_adapters(a[i], b, la[i], lb[i], ids[i], ws[0]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    say("adapters on two streams")
    for _ in range(10):
        got = [gsr.gemm_adapters(a[i], b, la[i], lb[i], ids[i], ws[i], stream=streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    hold = [t.clone() for t in (a[0], la[0], lb[0], ids[0])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = gsr.gemm_adapters(hold[0], b, hold[1], hold[2], hold[3], ws[0])
    for i in (0, 1, 0, 1):
        for t, new in zip(hold, (a[i], la[i], lb[i], ids[i])):
            t.copy_(new)
        say(f"adapters replayed, inputs {i}")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want[i]) and counters_zero(ws[0])
        assert torch.equal(gsr.gemm_adapters(a[1], b, la[1], lb[1], ids[1], ws[1]), want[1])
        torch.cuda.synchronize()


def test_refusals_on_the_device(gsr):
    M, N, K, L, R = 4, 16, 32, 2, 8
    h = dict(dtype=torch.float16, device=DEV)
    a, b, la, lb = torch.zeros(M, K, **h), torch.zeros(K, N, **h), torch.zeros(L, R, K, **h), torch.zeros(L, N, R, **h)
    ids, ws = torch.zeros(M, dtype=torch.int32, device=DEV), workspace(gsr, M, N, K, R)
    for bad in (lambda: gsr.gemm_adapters(a, b, la[:, :, :8].contiguous(), lb, ids, ws),
                lambda: gsr.gemm_adapters(a, b, la, lb[:1], ids, ws), lambda: gsr.gemm_adapters(a, b, la, lb, ids[:2], ws),
                lambda: gsr.gemm_adapters(a, b, la, lb.transpose(1, 2), ids, ws),
                lambda: gsr.gemm_adapters(a, b, la, lb, ids, ws, scales=torch.ones(3, device=DEV)),
                lambda: gsr.gemm_adapters(a, b, la, lb, ids, ws, activation="tanh")):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: gsr.gemm_adapters(a, b, la, lb, ids, ws[:512]), 1),
                        (lambda: gsr.gemm_adapters(a, b, la, lb, ids, ws, config_id=16), 6),
                        (lambda: gsr.gemm_adapters(a, b, la, lb, ids, ws, config_id=28, splits=2), 6),
                        (lambda: gsr.gemm_adapters(a, b, la, lb, ids, ws, splits=17), 1)):
        with pytest.raises(gsr.GsrError) as e:
            bad()
        assert e.value.status == status


@pytest.mark.parametrize("L,R", [(0, 16), (3, 0)])
def test_no_adapters_keep_the_split(gsr, L, R):
    """Without adapters a decode call splits K as the call with a workspace does."""
    M, N, K = 16, 4096, 11008
    g = torch.Generator().manual_seed(12)
    a, b = torch.randn(M, K, generator=g).half().to(DEV), (torch.randn(K, N, generator=g) * K ** -0.5).half().to(DEV)
    h = dict(dtype=torch.float16, device=DEV)
    ids = torch.zeros(M, dtype=torch.int32, device=DEV)
    ws = gsr.new_workspace(gsr.adapter_workspace_bytes(M, N, K, R))
    say(f"adapters: {L} of rank {R}, split")
    want = gsr.gemm_scale_bias_act_ws(a, b, gsr.new_workspace(gsr.workspace_bytes(M, N, K)), None, 0.5, "gelu")
    assert not torch.equal(want, gsr.gemm_scale_bias_act(a, b, None, 0.5, "gelu"))  # it is a split's sum
    for _ in range(2):
        c = gsr.gemm_adapters(a, b, torch.empty(L, R, K, **h), torch.empty(L, N, R, **h), ids, ws, alpha=0.5, activation="gelu")
        assert torch.equal(c.view(torch.int16), want.view(torch.int16))
        assert counters_zero(ws)
