"""GPU tests of the grouped products and of the routed layer against their
definitions in 64 bits on the host, and against the dense call bit for bit."""
import math

import numpy as np
import pytest
import torch

from tiled_dense_gemm_scale_amd import workloads as W

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


def offsets_of(sizes, extra=0):
    o = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return o, int(o[-1]) + extra


def reference(a, b, offsets, rows, bias, alpha, act, P, a_err=None):
    """c and, per value, the bound on what fp32 sums (K + 2 additions of
    2^-24, relative to the sum of magnitudes) and one fp16 rounding may be off
    by.  a_err: a bound on a's own error."""
    a64, b64 = a.double().numpy(), b.double().numpy()
    E, K, N = b64.shape
    c, slack = np.zeros((P, N)), np.zeros((P, N))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if rows is None:
            x = a64[lo:hi]
        else:
            r = rows[lo:hi]
            x = np.where(((r >= 0) & (r < len(a64)))[:, None], a64[np.clip(r, 0, len(a64) - 1)], 0.0)
        v, mag = alpha * (x @ b64[e]), abs(alpha) * (np.abs(x) @ np.abs(b64[e]))
        if bias is not None:
            v, mag = v + bias[e].double().numpy(), mag + np.abs(bias[e].double().numpy())
        off = (K + 2) * 2.0 ** -24 * mag
        if a_err is not None:
            off = off + abs(alpha) * (a_err[lo:hi] @ np.abs(b64[e]))
        # GELU: slope below 1.13, and a few 2^-22 of its own arithmetic
        off = 1.13 * off + (2.0 ** -20 * np.abs(v) if act == "gelu" else 0.0)
        c[lo:hi] = activate(v, act)
        slack[lo:hi] = off + 2.0 ** -11 * (np.abs(c[lo:hi]) + off) + 2.0 ** -25
    return c, slack


def within(name, got, ref, slack):
    err = np.abs(got - ref)
    assert np.all(err <= slack), f"{name}: {np.count_nonzero(~(err <= slack))} values, worst {np.nanmax(err / slack)}"
    say(f"{name}: worst error {float(np.max(err / slack)) if err.size else 0.0:.3f} of its bound")


# group sizes with empty ones, single rows, and both sides of the tile heights
SIZES = {"few": [0, 1, 33, 0, 7], "edges": [31, 32, 33, 64, 65, 0, 127, 129], "one": [0, 0, 300], "tall": [257, 511, 1],
         "none": [0, 0, 0, 0]}


@pytest.mark.parametrize("gather", [True, False], ids=["gather", "inplace"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("config", CONFIGS)
def test_integer_inputs_bitwise(gsr, config, sizes, gather):
    """Small integers: every fp32 sum is exact, so any order gives the same
    bits.  Rows behind the last group keep their values."""
    E, K, N = len(SIZES[sizes]), 200, 136
    offsets, P = offsets_of(SIZES[sizes], extra=5)
    g = torch.Generator().manual_seed(P + K)
    T = 61 if gather else P
    a = torch.randint(-4, 5, (T, K), generator=g).half()
    b = torch.randint(-4, 5, (E, K, N), generator=g).half()
    bias = torch.randint(-4, 5, (E, N), generator=g).half()
    rows = torch.randint(-2, T + 2, (P,), generator=g).int() if gather else None
    c = torch.full((P, N), 9.0, dtype=torch.float16, device=DEV)
    say(f"grouped integers config={config} {sizes} gather={gather}")
    gsr.gemm_grouped(a.to(DEV), b.to(DEV), torch.from_numpy(offsets).to(DEV),
                     rows=rows.to(DEV) if gather else None, bias=bias.to(DEV), alpha=0.5, activation="relu", c=c,
                     config_id=config)
    ref, _ = reference(a, b, offsets, rows.numpy() if gather else None, bias, 0.5, "relu", P)
    want = torch.from_numpy(ref).half()  # multiples of 1/2 below 2^11: exact
    got = c.cpu()
    assert torch.equal(got[:offsets[-1]], want[:offsets[-1]])
    assert bool((got[offsets[-1]:] == 9.0).all())


@pytest.mark.parametrize("act", ["relu", "gelu", "none"])
@pytest.mark.parametrize("shape", [(3, 64, 64), (5, 1000, 264), (4, 77, 101), (2, 8, 8), (3, 130, 1), (6, 1, 40),
                                   (2, 516, 300), (9, 2056, 72)], ids=lambda s: "x".join(map(str, s)))
def test_normal_inputs(gsr, shape, act):
    """Every path (16-byte units, the element-wise kernel's 8, 4 and 2 bytes)
    against the definition."""
    E, K, N = shape
    rng = np.random.default_rng(K + N)
    sizes = rng.integers(0, 90, E)
    sizes[rng.integers(0, E)] = 0
    offsets, P = offsets_of(sizes, extra=2)
    g = torch.Generator().manual_seed(K)
    T = 50
    a, b = torch.randn(T, K, generator=g).half(), (torch.randn(E, K, N, generator=g) * K ** -0.5).half()
    bias = torch.randn(E, N, generator=g).half() if act != "none" else None
    rows = torch.randint(0, T, (P,), generator=g).int()
    for config in CONFIGS:
        say(f"grouped normal {shape} {act} config={config}")
        c = gsr.gemm_grouped(a.to(DEV), b.to(DEV), torch.from_numpy(offsets).to(DEV), rows=rows.to(DEV),
                             bias=bias.to(DEV) if bias is not None else None, alpha=-0.75, activation=act,
                             config_id=config)
        ref, slack = reference(a, b, offsets, rows.numpy(), bias, -0.75, act, P)
        n = int(offsets[-1])
        within(f"config {config}", c.cpu().double().numpy()[:n], ref[:n], slack[:n])


def test_many_groups(gsr):
    """More groups than a wave has lanes, most of them empty."""
    E, K, N = 200, 64, 64
    sizes = np.zeros(E, int)
    sizes[[0, 63, 64, 65, 127, 128, 150, 199]] = [3, 40, 1, 70, 2, 33, 5, 9]
    offsets, P = offsets_of(sizes)
    g = torch.Generator().manual_seed(5)
    a, b = torch.randint(-4, 5, (P, K), generator=g).half(), torch.randint(-4, 5, (E, K, N), generator=g).half()
    ref, _ = reference(a, b, offsets, None, None, 1.0, "none", P)
    for config in CONFIGS:
        say(f"grouped 200 groups config={config}")
        c = gsr.gemm_grouped(a.to(DEV), b.to(DEV), torch.from_numpy(offsets).to(DEV), activation="none",
                             config_id=config)
        assert torch.equal(c.cpu(), torch.from_numpy(ref).half())


@pytest.mark.parametrize("config", [21, 22, 28, 31, 32])
def test_same_bits_as_the_dense_call(gsr, config):
    E, K, N = 3, 1032, 528
    offsets, P = offsets_of([70, 0, 300])
    g = torch.Generator().manual_seed(8)
    a, b = torch.randn(P, K, generator=g).half().to(DEV), torch.randn(E, K, N, generator=g).half().to(DEV)
    bias = torch.randn(E, N, generator=g).half().to(DEV)
    say(f"grouped against dense config={config}")
    c = gsr.gemm_grouped(a, b, torch.from_numpy(offsets).to(DEV), bias=bias, alpha=0.1, activation="gelu",
                         config_id=config)
    for e in (0, 2):
        lo, hi = offsets[e], offsets[e + 1]
        want = gsr.gemm_scale_bias_act(a[lo:hi], b[e], bias[e], 0.1, "gelu", config_id=config)
        assert torch.equal(c[lo:hi].view(torch.int16), want.view(torch.int16))


def test_infinities_stay_in_their_rows(gsr):
    """NaN and infinity in one group's weights, or in rows of x that no index
    names, reach that group's rows only."""
    E, K, N = 3, 128, 128
    offsets, P = offsets_of([20, 30, 40])
    g = torch.Generator().manual_seed(9)
    a, b = torch.randint(-3, 4, (64, K), generator=g).half(), torch.randint(-3, 4, (E, K, N), generator=g).half()
    rows = torch.randint(0, 60, (P,), generator=g).int()
    ref, _ = reference(a, b, offsets, rows.numpy(), None, 1.0, "none", P)
    b[1, 5] = float("nan")
    b[1, 7] = float("inf")
    a[60:] = float("nan")
    for config in CONFIGS:
        say(f"grouped infinities config={config}")
        c = gsr.gemm_grouped(a.to(DEV), b.to(DEV), torch.from_numpy(offsets).to(DEV), rows=rows.to(DEV),
                             activation="none", config_id=config).cpu()
        want = torch.from_numpy(ref).half()
        assert torch.equal(c[:20], want[:20]) and torch.equal(c[50:], want[50:])
        assert bool(torch.isnan(c[20:50]).all())


@pytest.mark.parametrize("act", ["relu", "gelu", "none"])
def test_no_inner_dimension(gsr, act):
    offsets, P = offsets_of([3, 0, 2], extra=1)
    bias = torch.tensor([[-1.0, 0.5], [7.0, 7.0], [2.0, -3.0]]).half()
    c = torch.full((P, 2), 9.0, dtype=torch.float16, device=DEV)
    say(f"grouped K=0 {act}")
    gsr.gemm_grouped(torch.empty(P, 0, dtype=torch.float16, device=DEV), torch.empty(3, 0, 2, dtype=torch.float16, device=DEV),
                     torch.from_numpy(offsets).to(DEV), bias=bias.to(DEV), activation=act, c=c)
    want = torch.cat([bias[0].expand(3, 2), bias[2].expand(2, 2)]).double().numpy()
    got = c.cpu()
    assert np.allclose(got[:5].double().numpy(), activate(want, act), rtol=2.0 ** -11, atol=2.0 ** -20)
    assert bool((got[5] == 9.0).all())


@pytest.mark.parametrize("off", [1, 2, 4], ids=lambda o: f"+{2 * o}B")
def test_less_aligned_c_and_a(gsr, off):
    E, K, N = 2, 72, 88
    offsets, P = offsets_of([37, 20])
    g = torch.Generator().manual_seed(10)
    a, b = torch.randint(-4, 5, (P, K), generator=g).half(), torch.randint(-4, 5, (E, K, N), generator=g).half()
    ref, _ = reference(a, b, offsets, None, None, 1.0, "none", P)
    for which in ("c", "a", "b"):
        say(f"grouped {which} at +{2 * off} bytes")
        cb = torch.full((P * N + 8,), 3.0, dtype=torch.float16, device=DEV)
        o = off if which == "c" else 0
        c = cb[o:o + P * N].view(P, N)

        def place(t, on):
            buf = torch.zeros(t.numel() + 8, dtype=torch.float16, device=DEV)
            v = buf[on:on + t.numel()].view(t.shape)
            v.copy_(t)
            return v

        gsr.gemm_grouped(place(a, off if which == "a" else 0), place(b, off if which == "b" else 0),
                         torch.from_numpy(offsets).to(DEV), activation="none", c=c)
        assert torch.equal(c.cpu(), torch.from_numpy(ref).half())
        host = cb.cpu()
        assert bool((host[:o] == 3.0).all()) and bool((host[o + P * N:] == 3.0).all())


@pytest.mark.parametrize("config", [-1, 21, 22, 28, 31, 32])
@pytest.mark.parametrize("kind", ["overlapping", "decreasing", "outside", "far"])
def test_offsets_out_of_order(gsr, config, kind):
    """Offsets that no sort gives: the call ends and nothing outside the P rows
    of c is written."""
    P, E, K, N = 70, 130, 64, 72
    offsets = {"overlapping": [0, P] * 66, "decreasing": list(range(E, -1, -1)), "outside": [-5, 10 ** 6] * 66,
               "far": [-2 ** 31, 2 ** 31 - 1] * 66}[kind][:E + 1]
    a, b = torch.zeros(P, K, dtype=torch.float16, device=DEV), torch.zeros(E, K, N, dtype=torch.float16, device=DEV)
    c = torch.full((P + 300, N), 9.0, dtype=torch.float16, device=DEV)
    say(f"grouped offsets {kind} config={config}")
    gsr.gemm_grouped(a, b, torch.tensor(offsets, dtype=torch.int32, device=DEV), c=c[150:150 + P], activation="none",
                     config_id=config)
    torch.cuda.synchronize()
    assert bool((c[:150] == 9.0).all()) and bool((c[150 + P:] == 9.0).all())


def test_past_32_bit_offsets(gsr):
    """B and C of more than 2^31 bytes: the last group's weights, the last rows."""
    E, K, N = 40, 4096, 8192  # 2.7 GB
    b = torch.zeros(E, K, N, dtype=torch.float16, device=DEV)
    b[E - 1] = 1.0
    b[E - 2] = 2.0
    P = 140000  # 140000 x 8192 x 2 = 2.3 GB
    sizes = np.zeros(E, int)
    sizes[0], sizes[E - 2], sizes[E - 1] = P - 300, 100, 200
    offsets, _ = offsets_of(sizes)
    a = torch.zeros(3, K, dtype=torch.float16, device=DEV)
    a[1, :7], a[2, -5:] = 1.0, 1.0
    rows = (torch.arange(P, device=DEV) % 3).int()
    c = torch.full((P, N), 9.0, dtype=torch.float16, device=DEV)
    say("grouped past 32-bit offsets")
    gsr.gemm_grouped(a, b, torch.from_numpy(offsets).to(DEV), rows=rows, activation="none", c=c)
    want = torch.tensor([0.0, 7.0, 5.0], device=DEV)[rows[P - 300:].long()]
    want[:100] *= 2.0
    assert bool((c[P - 300:].float() == want[:, None]).all())
    assert bool((c[:P - 300] == 0.0).all())


def routed(T, k, E, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k].contiguous()
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    return ids, torch.softmax(torch.randn(T, k, generator=g), 1)


def layer_inputs(T, k, E, H, F, seed):
    g = torch.Generator().manual_seed(seed + 100)
    ids, w = routed(T, k, E, seed)
    return dict(x=torch.randn(T, H, generator=g).half(), ids=ids, weights=w,
                up=(torch.randn(E, H, F, generator=g) * H ** -0.5).half(),
                down=(torch.randn(E, F, H, generator=g) * F ** -0.5).half(),
                bias_up=torch.randn(E, F, generator=g).half(), bias_down=torch.randn(E, H, generator=g).half())


@pytest.mark.parametrize("shape", [(1, 2, 4, 64, 128), (37, 2, 8, 128, 264), (300, 3, 5, 101, 77), (513, 2, 4, 256, 512)],
                         ids=lambda s: "x".join(map(str, s)))
def test_expert_mlp(gsr, shape):
    """The whole layer (sort, two grouped products, weighted sum) as a model
    runs it, its roundings carried through as bounds."""
    T, k, E, H, F = shape
    i = layer_inputs(T, k, E, H, F, seed=T)
    say(f"expert_mlp {shape}")
    out = gsr.expert_mlp(**{n: t.to(DEV) for n, t in i.items()}, activation="gelu")
    offsets, rows, positions = (t.cpu().numpy() for t in gsr.group_rows(i["ids"].to(DEV), E))
    n = int(offsets[-1])
    h, hs = reference(i["x"], i["up"], offsets, rows, i["bias_up"], 1.0, "gelu", T * k)
    y, ys = reference(torch.from_numpy(h), i["down"], offsets, None, i["bias_down"], 1.0, "none", T * k, a_err=hs)
    ref, slack, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        ok = positions[:, j] >= 0
        w = i["weights"][ok, j].double().numpy()[:, None]
        ref[ok] += w * y[positions[ok, j]]
        slack[ok] += w * ys[positions[ok, j]]
        mag[ok] += w * np.abs(y[positions[ok, j]])
    slack += (k + 1) * 2.0 ** -24 * mag
    slack += 2.0 ** -11 * (np.abs(ref) + slack) + 2.0 ** -25
    assert n == int((i["ids"] >= 0).sum())
    within("layer", out.cpu().double().numpy(), ref, slack)


def test_expert_mlp_on_streams_and_captured(gsr):
    """Two layers at once on two streams, then a captured layer replayed with
    new inputs, eager work between the replays: the bits of the eager call."""
    T, k, E, H, F = 70, 2, 6, 128, 256
    a, b = ({n: t.to(DEV) for n, t in layer_inputs(T, k, E, H, F, seed=s).items()} for s in (1, 2))
    torch.cuda.synchronize()
    say("expert_mlp on two streams")
    want_a, want_b = gsr.expert_mlp(**a), gsr.expert_mlp(**b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got_a, got_b = gsr.expert_mlp(**a, stream=s1), gsr.expert_mlp(**b, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(got_a, want_a) and torch.equal(got_b, want_b)
    say("expert_mlp captured")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gsr.expert_mlp(**a)
    for new in (b, a, b):
        if new is not a:
            saved = {n: t.clone() for n, t in a.items()}
            for n in a:
                a[n].copy_(b[n])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_b if new is not a else want_a)
        if new is not a:
            for n in a:
                a[n].copy_(saved[n])
        _ = (a["x"].float() * 2).sum()
        torch.cuda.synchronize()


def test_python_refusals_on_the_device(gsr):
    a = torch.zeros(4, 8, dtype=torch.float16, device=DEV)
    b = torch.zeros(2, 8, 16, dtype=torch.float16, device=DEV)
    o = torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad in (lambda: gsr.gemm_grouped(a, b, o[:2]), lambda: gsr.gemm_grouped(a[:, :4].contiguous(), b, o),
                lambda: gsr.gemm_grouped(a, b.transpose(1, 2), o), lambda: gsr.gemm_grouped(a, b, o, bias=b[0]),
                lambda: gsr.gemm_grouped(a, b, o, activation="tanh"),
                lambda: gsr.gemm_grouped(a, b, o, c=torch.zeros(5, 16, dtype=torch.float16, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gsr.GsrError):
        gsr.gemm_grouped(a, b, o, config_id=16)
    with pytest.raises(gsr.GsrError):
        gsr.gemm_grouped(a, b, o, alpha=math.inf)


@pytest.mark.parametrize("K,N,shift", [(1032, 528, 1), (1032, 528, 2)] +
                         [(K, N, s) for K, N in ((517, 301), (2051, 77), (514, 130)) for s in (0, 1, 2)])
@pytest.mark.parametrize("config", [21, 22, 28, 31, 32])
def test_same_bits_as_the_dense_call_off_the_vector_path(gsr, config, K, N, shift):
    """As above for odd sizes and addresses: one chain of sums over K."""
    offsets, P = offsets_of([70, 0, 300])
    g = torch.Generator().manual_seed(K)
    d = lambda t: torch.cat([torch.zeros(shift, dtype=t.dtype), t.flatten()]).to(DEV)[shift:].view(t.shape)
    a, b = d(torch.randn(P, K, generator=g).half()), d(torch.randn(3, K, N, generator=g).half())
    bias = d(torch.randn(3, N, generator=g).half())
    say(f"grouped against dense {K}x{N} config={config} shift={shift}")
    c = gsr.gemm_grouped(a, b, torch.from_numpy(offsets).to(DEV), bias=bias, alpha=0.1, activation="gelu", config_id=config)
    for e in (0, 2):
        lo, hi = offsets[e], offsets[e + 1]
        want = gsr.gemm_scale_bias_act(a[lo:hi], b[e], bias[e], 0.1, "gelu", config_id=config)
        assert torch.equal(c[lo:hi].view(torch.int16), want.view(torch.int16))
