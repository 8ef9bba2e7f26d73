"""GPU tests of the few-token layer of routed experts against its definition in
64 bits on the host: whole numbers bit for bit, normal values within the bound
of their sums."""
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


def choices(rng, T, k, E, drop, distinct=True):
    if distinct and k <= E:
        ids = np.argsort(rng.random((T, E)) * (0.2 + rng.random(E)), axis=1)[:, :k]
    else:
        ids = rng.integers(0, E, (T, k))
    lost = rng.random((T, k)) < drop
    return np.where(lost, np.where(rng.random((T, k)) < 0.5, -1, E), ids)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def experts(gsr, rng, E, K, N, form, group, whole):
    """The handle and the values in 64 bits."""
    if form == "fp16":
        w = rng.integers(-1, 2, (E, K, N)) if whole else rng.standard_normal((E, K, N)) * max(K, 1) ** -0.5
        w = w.astype(np.float16)
        return dev(w), w.astype(np.float64)
    G = -(-K // group)
    q = rng.integers(7, 10, (E, K, N)) if whole else rng.integers(0, 16, (E, K, N))
    z = None if form == "w4" else rng.integers(6, 11, (E, G, N)).astype(np.uint8)
    s = np.ones((E, G, N)) if whole else (0.5 + rng.random((E, G, N))) * 0.2 * max(K, 1) ** -0.5
    s = s.astype(np.float16)
    f = np.stack([ref.values(q[e], s[e], None if z is None else z[e], group) for e in range(E)]) if E else np.zeros((0, K, N))
    return gsr.W4(ref.pack(q).to(DEV), dev(s), dev(z), K, group), f


def case_inputs(gsr, case, form, whole, gated, bias, seed=0, distinct=True):
    T, k, E, H, F, O, drop, group = case
    rng = np.random.default_rng(seed + T + k + E + H + F)
    x = (rng.integers(-1, 2, (T, H)) * (rng.random((T, H)) < 0.5) if whole else rng.standard_normal((T, H))).astype(np.float16)
    ids = choices(rng, T, k, E, drop, distinct)
    w = (2.0 ** rng.integers(-1, 2, (T, k)) if whole else rng.random((T, k))).astype(np.float32)
    hs, fs, biases = {}, {}, {}
    for name, K, N in (("up", H, F), ("gate", H, F), ("down", F, O)):
        if name == "gate" and not gated:
            hs[name] = fs[name] = biases[name] = None
            continue
        hs[name], fs[name] = experts(gsr, rng, E, K, N, form, group, whole)
        b = rng.integers(-3, 4, (E, N)) if whole else rng.standard_normal((E, N))
        biases[name] = b.astype(np.float16) if bias else None
    return x, ids, w, hs, fs, biases


def call(gsr, x, ids, w, hs, biases, act, ws, wide=False, **more):
    return gsr.expert_mlp_few(dev(x), dev(ids.astype(np.int64 if wide else np.int32)), dev(w), hs["up"], hs["down"], ws,
                              gate=hs["gate"], bias_up=dev(biases["up"]), bias_gate=dev(biases["gate"]),
                              bias_down=dev(biases["down"]), activation=act, **more)


def workspace(gsr, case):
    T, k, E, H, F, O, drop, group = case
    return gsr.new_workspace(gsr.expert_few_workspace_bytes(T, k, E, F, O))


# tokens, choices, experts, H, F, O, share dropped, group
CASES = [(1, 1, 1, 1, 1, 1, 0.0, 32), (1, 2, 8, 256, 512, 256, 0.0, 128), (1, 8, 64, 128, 64, 128, 0.0, 32),
         (2, 3, 5, 33, 70, 9, 0.0, 32), (3, 2, 4, 7, 5, 3, 0.0, 32), (4, 2, 8, 130, 129, 131, 0.3, 64),
         (7, 3, 10, 101, 517, 203, 0.25, 64), (16, 8, 24, 64, 96, 64, 0.1, 32), (16, 2, 2, 200, 300, 72, 0.0, 128),
         (17, 4, 6, 96, 130, 100, 0.1, 32), (31, 2, 1000, 40, 32, 48, 0.0, 32), (33, 5, 9, 65, 64, 33, 0.2, 64),
         (64, 2, 3, 128, 192, 64, 0.0, 128), (64, 16, 40, 36, 40, 44, 0.1, 32), (64, 4, 4, 72, 1100, 20, 0.0, 256),
         (5, 2, 4, 300, 2100, 140, 0.0, 128)]
FORMS = ["fp16", "w4", "w4z"]


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_whole_numbers(gsr, case, form, gated):
    """Sums of small whole numbers are exact, the hidden values below 2048 too:
    the outputs are the fp16 values nearest the formula's."""
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, True, gated, True)
    x[:, 24:] = 0  # keeps the hidden values small
    b64 = {n: None if b is None else b.astype(np.float64) for n, b in biases.items()}
    out, _, hidden = ref.layer(x.astype(np.float64), ids, w, fs["up"], fs["gate"], fs["down"], b64, "none")
    if hidden:
        assert max(np.abs(h).max() for h in hidden) <= 2048
    say(f"few whole {case} {form} gated={gated}")
    ws = workspace(gsr, case)
    with np.errstate(over="ignore"):
        want = out.astype(np.float16)
    for i in range(2):
        got = call(gsr, x, ids, w, hs, biases, "none", ws, wide=i == 1).cpu().numpy()
        assert np.array_equal(got, want), f"{np.count_nonzero(got != want)} of {want.size} differ"
    assert int(ws[:512].count_nonzero()) == 0


@pytest.mark.parametrize("act,gated", [("gelu", False), ("relu", False), ("silu", True), ("none", True), ("gelu", True)])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_layer(gsr, case, form, act, gated):
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, False, gated, act == "relu" or (gated and act == "gelu"), seed=1)
    b64 = {n: None if b is None else b.astype(np.float64) for n, b in biases.items()}
    out, slack, _ = ref.layer(x.astype(np.float64), ids, w, fs["up"], fs["gate"], fs["down"], b64, act)
    say(f"few {case} {form} {act} gated={gated}")
    got = call(gsr, x, ids, w, hs, biases, act, workspace(gsr, case)).cpu().numpy().astype(np.float64)
    err = np.abs(got - out)
    say(f"few {case} {form} {act}: worst {float((err / slack).max()):.3f} of its bound, "
        f"{float(err.max() / max(np.abs(out).max(), 1e-30)):.1e} of the largest output")
    assert (err <= slack).all()


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("form", FORMS)
def test_narrow_widths(gsr, form, gated):
    """Every width of F and O up to 18, columns of fewer than a lane's among them:
    the formula's values, and nothing written behind the last row."""
    for n in range(1, 19):
        for case in ((9, 2, 3, 40, n, 33, 0.2, 32), (9, 2, 3, 40, 24, n, 0.2, 32), (9, 2, 3, n, n, n, 0.2, 32)):
            x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, True, gated, True)
            b64 = {m: None if b is None else b.astype(np.float64) for m, b in biases.items()}
            out, _, _ = ref.layer(x.astype(np.float64), ids, w, fs["up"], fs["gate"], fs["down"], b64, "none")
            buf = torch.full((9 * case[5] + 64,), 5.0, dtype=torch.float16, device=DEV)
            say(f"few narrow {case} {form} gated={gated}")
            got = call(gsr, x, ids, w, hs, biases, "none", workspace(gsr, case), out=buf[:9 * case[5]].view(9, case[5]))
            with np.errstate(over="ignore"):
                assert np.array_equal(got.cpu().numpy(), out.astype(np.float16)), case
            assert bool((buf[9 * case[5]:] == 5.0).all()), case


@pytest.mark.parametrize("form", FORMS)
def test_named_twice(gsr, form):
    """A token that names an expert more than once has a term for each, and an
    expert may so have more rows than there are tokens."""
    case = (13, 6, 3, 40, 72, 50, 0.1, 32)
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, True, False, True, distinct=False)
    ids[:, 1] = ids[:, 0] = 1
    b64 = {n: None if b is None else b.astype(np.float64) for n, b in biases.items()}
    out, _, hidden = ref.layer(x.astype(np.float64), ids, w, fs["up"], None, fs["down"], b64, "none")
    say(f"few twice {form}")
    got = call(gsr, x, ids, w, hs, biases, "none", workspace(gsr, case)).cpu().numpy()
    assert np.array_equal(got, out.astype(np.float16))


@pytest.mark.parametrize("form", FORMS)
def test_many_slots_of_one_expert(gsr, form):
    """1024 slots that all name the same expert."""
    case = (64, 16, 5, 33, 40, 70, 0.0, 32)
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, True, True, False)
    ids[:] = 3
    x[:, 24:] = 0
    out, _, _ = ref.layer(x.astype(np.float64), ids, w, fs["up"], fs["gate"], fs["down"], {}, "none")
    say(f"few one expert {form}")
    got = call(gsr, x, ids, w, hs, biases, "none", workspace(gsr, case)).cpu().numpy()
    assert np.array_equal(got, out.astype(np.float16))


@pytest.mark.parametrize("form", FORMS)
def test_no_choice_left(gsr, form):
    """Tokens without a choice are rows of zeros, all of them too; no weights
    means ones; no choices at all, no experts, no hidden columns."""
    case = (6, 2, 4, 40, 50, 33, 0.0, 32)
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, True, False, True)
    b64 = {n: None if b is None else b.astype(np.float64) for n, b in biases.items()}
    ids[2] = (-1, 4)
    ws = workspace(gsr, case)
    say(f"few none {form}")
    out, _, _ = ref.layer(x.astype(np.float64), ids, None, fs["up"], None, fs["down"], b64, "relu")
    got = call(gsr, x, ids, None, hs, biases, "relu", ws).cpu().numpy()
    assert np.array_equal(got, out.astype(np.float16)) and not got[2].any()
    full = torch.full((6, 33), 7.0, dtype=torch.float16, device=DEV)
    ids[:] = -1
    assert not call(gsr, x, ids, w, hs, biases, "relu", ws, out=full).any()
    full.fill_(7.0)
    assert not call(gsr, x, ids[:, :0], w[:, :0], hs, biases, "relu", ws, out=full).any()
    assert tuple(call(gsr, x[:0], ids[:0], w[:0], hs, biases, "relu", ws).shape) == (0, 33)
    for changed in ((6, 2, 4, 40, 0, 33, 0.0, 32), (6, 2, 4, 0, 50, 33, 0.0, 32)):
        x, ids, w, hs, fs, biases = case_inputs(gsr, changed, form, True, False, True)
        b64 = {n: b.astype(np.float64) for n, b in biases.items() if b is not None}
        out, _, _ = ref.layer(x.astype(np.float64), ids, w, fs["up"], None, fs["down"], b64, "relu")
        say(f"few none {form} {changed}")
        assert np.array_equal(call(gsr, x, ids, w, hs, biases, "relu", ws).cpu().numpy(), out.astype(np.float16))


@pytest.mark.parametrize("form", FORMS)
def test_values_stay_in_their_rows(gsr, form):
    """Infinities and NaN of one token, of an expert's bias and (fp16) of an
    expert that nobody names reach no other token."""
    case = (9, 2, 6, 70, 90, 130, 0.0, 32)
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, False, True, True)
    ids[:] = np.stack([np.arange(9) % 4, 4 * np.ones(9)], 1)
    base = call(gsr, x, ids, w, hs, biases, "silu", workspace(gsr, case)).cpu().numpy()
    x[3, 5], x[3, 60] = np.inf, np.nan
    biases["down"][2] = np.nan
    if form == "fp16":
        for n in ("up", "gate", "down"):
            hs[n][5] = float("nan")
    else:
        for n in ("up", "gate", "down"):
            hs[n].scales[5] = float("inf")
    say(f"few non-finite {form}")
    got = call(gsr, x, ids, w, hs, biases, "silu", workspace(gsr, case)).cpu().numpy()
    bad = np.array([t == 3 or t % 4 == 2 for t in range(9)])
    assert np.array_equal(got[~bad], base[~bad])
    assert np.isnan(got[3]).all() and np.isnan(got[2]).all() and np.isnan(got[6]).all()


def test_infinite_weight_keeps_its_sign(gsr):
    """An infinity in the matrix makes an infinity of its own column, whatever
    lies in the last rows of ragged sizes."""
    T, k, E, H, F, O = 2, 1, 2, 37, 45, 29
    rng = np.random.default_rng(0)
    x = np.abs(rng.standard_normal((T, H))).astype(np.float16)
    up = np.abs(rng.standard_normal((E, H, F))).astype(np.float16) * np.float16(0.1)
    down = np.abs(rng.standard_normal((E, F, O))).astype(np.float16) * np.float16(0.1)
    down[0, F - 1, O - 1], down[0, 3, 0] = np.inf, -np.inf
    down[1] = np.inf
    ids = np.zeros((T, k), np.int32)
    say("few infinite weight")
    got = gsr.expert_mlp_few(dev(x), dev(ids), None, dev(up), dev(down),
                             gsr.new_workspace(gsr.expert_few_workspace_bytes(T, k, E, F, O)), activation="relu").cpu().numpy()
    assert (got[:, O - 1] == np.inf).all() and (got[:, 0] == -np.inf).all() and np.isfinite(got[:, 1:O - 1]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shift", [1, 2])
def test_odd_addresses(gsr, form, shift):
    case = (6, 2, 4, 64, 72, 80, 0.1, 32)
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, False, True, True)
    base = call(gsr, x, ids, w, hs, biases, "silu", workspace(gsr, case))

    def moved(t):
        buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device=DEV)
        out = buf[shift:shift + t.numel()].view(t.shape)
        out.copy_(t)
        return out

    def moved_w(h):
        return moved(h) if form == "fp16" else gsr.W4(moved(h.codes), moved(h.scales), None if h.zeros is None else moved(h.zeros),
                                                      h.k, h.group)

    obuf = torch.full((6 * 80 + 8,), 3.0, dtype=torch.float16, device=DEV)
    o = obuf[shift:shift + 480].view(6, 80)
    say(f"few addresses {form} +{shift}")
    gsr.expert_mlp_few(moved(dev(x)), moved(dev(ids.astype(np.int32))), moved(dev(w)), moved_w(hs["up"]), moved_w(hs["down"]),
                       workspace(gsr, case), gate=moved_w(hs["gate"]), bias_up=moved(dev(biases["up"])),
                       bias_gate=moved(dev(biases["gate"])), bias_down=moved(dev(biases["down"])), activation="silu", out=o)
    assert torch.equal(o, base)
    assert bool((obuf[:shift] == 3.0).all()) and bool((obuf[shift + 480:] == 3.0).all())


@pytest.mark.parametrize("form", ["fp16", "w4z"])
def test_captured_layer_beside_other_calls(gsr, form):
    """A captured layer replays with the eager bits for new tokens and routings,
    with eager calls of other sizes in the same workspace between the replays."""
    case, other = (8, 2, 8, 256, 1100, 300, 0.1, 64), (3, 2, 8, 64, 70, 9000, 0.0, 32)
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, False, True, True)
    o = case_inputs(gsr, other, "fp16", False, False, False)
    nbytes = max(gsr.expert_few_workspace_bytes(c[0], c[1], c[2], c[4], c[5]) for c in (case, other))
    ws, side = gsr.new_workspace(nbytes), torch.cuda.Stream()
    X, I, W = dev(x), dev(ids.astype(np.int64)), dev(w)
    B = {n: dev(b) for n, b in biases.items()}
    out = torch.empty(8, 300, dtype=torch.float16, device=DEV)

    def layer(to=None, stream=None):
        return gsr.expert_mlp_few(X, I, W, hs["up"], hs["down"], ws, gate=hs["gate"], bias_up=B["up"], bias_gate=B["gate"],
                                  bias_down=B["down"], activation="silu", out=to, stream=stream)

    side.wait_stream(torch.cuda.current_stream())
    layer(out, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    say(f"few capture {form}")
    with torch.cuda.graph(graph, stream=side):
        layer(out)
    rng = np.random.default_rng(3)
    for i in range(4):
        X.copy_(torch.randn(8, 256, device=DEV).half())
        I.copy_(dev(choices(rng, 8, 2, 8, 0.2)))
        want = layer()
        call(gsr, o[0], o[1], o[2], o[3], o[5], "gelu", ws)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    assert int(ws[:512].count_nonzero()) == 0


def test_agrees_with_the_layer_for_many_tokens(gsr):
    """The same layer through group_rows and the grouped products, and a decode
    step as a program makes it: experts brought into 4 bits, a projection in 4
    bits, the layer; every piece against its fp16 values."""
    T, k, E, H, F = 24, 2, 8, 256, 512
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(T, H, generator=g, device=DEV).half()
    score, ids = torch.softmax(torch.randn(T, E, generator=g, device=DEV), 1).topk(k)
    score = score.contiguous()
    up, down = (torch.randn(E, i, o, generator=g, device=DEV).half() * i ** -0.5 for i, o in ((H, F), (F, H)))
    proj = (torch.randn(H, H, generator=g, device=DEV) * H ** -0.5).half()
    ws = gsr.new_workspace(gsr.expert_few_workspace_bytes(T, k, E, F, H))
    say("few beside expert_mlp")
    a, b = gsr.expert_mlp_few(x, ids, score, up, down, ws), gsr.expert_mlp(x, ids, score, up, down)
    # the other one rounds h to fp16 (half a step, 2^-11, whose share of the output
    # adds up over F), and both the output (half a step each)
    assert float((a - b).float().norm() / b.float().norm()) < 2.0 ** -10
    wu, wd, wp = gsr.quantize_w4(up), gsr.quantize_w4(down, 64, zeros=True), gsr.quantize_w4(proj, 32)
    y = gsr.gemm_w4(x, wp, ws, activation="none")
    z = gsr.expert_mlp_few(y, ids, score, wu, wd, ws)
    y2 = gsr.gemm_scale_bias_act(x, gsr.dequantize_w4(wp), activation="none")
    z2 = gsr.expert_mlp_few(y2, ids, score, gsr.dequantize_w4(wu), gsr.dequantize_w4(wd), ws)
    # dequantized weights are rounded to fp16 (2^-11 each), which a product of
    # independent roundings keeps; three products and the rounding of y and h
    assert float((y - y2).float().norm() / y2.float().norm()) < 2.0 ** -10
    assert float((z - z2).float().norm() / z2.float().norm()) < 2.0 ** -8


def test_hidden_values_past_fp16(gsr):
    """An h that fp16 does not hold becomes an infinity, of its own token's slot
    alone; one just below stays, its rounding's rest with it."""
    H, F, O = 8, 40, 24
    x = torch.zeros(3, H, dtype=torch.float16, device=DEV)
    x[0, 0], x[1, 0], x[2, 0] = 60000.0, 64000.0, -64000.0
    up = torch.zeros(1, H, F, dtype=torch.float16, device=DEV)
    up[0, 0, 0], up[0, 0, 1] = 1.0009765625, 1.0
    down = torch.zeros(1, F, O, dtype=torch.float16, device=DEV)
    down[0, 0], down[0, 1] = 2.0 ** -4, -(2.0 ** -4)
    ids = torch.zeros(3, 1, dtype=torch.int32, device=DEV)
    up[0, 0, 2] = 1.125  # 67500, 72000, -72000
    ws = gsr.new_workspace(gsr.expert_few_workspace_bytes(3, 1, 1, F, O))
    say("few past fp16")
    got = gsr.expert_mlp_few(x, ids, None, up, down, ws, activation="none").cpu().numpy()
    # the row of the overflowed h is zero in down: infinity times zero
    assert np.isnan(got).all()
    up[0, 0, 2] = 0.0
    got = gsr.expert_mlp_few(x, ids, None, up, down, ws, activation="none").cpu().numpy()
    # h0 - h1 = x 2^-10, a multiple of h's last bit only with the second half
    want = np.array([60000.0, 64000.0, -64000.0]) * 2.0 ** -14
    assert np.array_equal(got, np.repeat(want.astype(np.float16)[:, None], O, 1))


@pytest.mark.parametrize("form", ["fp16", "w4z"])
def test_two_layers_at_once(gsr, form):
    """Calls on two streams with a workspace each, many times over."""
    case, other = (16, 4, 12, 264, 1100, 520, 0.1, 64), (3, 2, 8, 64, 700, 300, 0.0, 32)
    calls = []
    for c in (case, other):
        x, ids, w, hs, fs, biases = case_inputs(gsr, c, form, False, True, True, seed=4)
        T, k, E, H, F, O, drop, group = c
        X, I, W, B = dev(x), dev(ids.astype(np.int64)), dev(w), {n: dev(b) for n, b in biases.items()}
        ws, out, s = workspace(gsr, c), torch.empty(T, O, dtype=torch.float16, device=DEV), torch.cuda.Stream()
        calls.append((lambda X=X, I=I, W=W, hs=hs, B=B, ws=ws, out=out, s=s: gsr.expert_mlp_few(
            X, I, W, hs["up"], hs["down"], ws, gate=hs["gate"], bias_up=B["up"], bias_gate=B["gate"], bias_down=B["down"],
            activation="silu", out=out, stream=s), out, s))
    say(f"few two streams {form}")
    wants = []
    for go, out, s in calls:
        go()
        torch.cuda.synchronize()
        wants.append(out.clone())
    for _ in range(5):
        for go, out, s in calls:
            with torch.cuda.stream(s):
                out.fill_(9.0)
        for _ in range(20):
            for go, out, s in calls:
                go()
        torch.cuda.synchronize()
        for (go, out, s), want in zip(calls, wants):
            assert torch.equal(out, want)


def test_every_expert_and_slot(gsr):
    """1024 slots of 1024 experts, and one token of 1024 choices."""
    for case in ((64, 16, 1024, 24, 33, 40, 0.0, 32), (1, 1024, 1024, 24, 40, 33, 0.0, 32)):
        x, ids, w, hs, fs, biases = case_inputs(gsr, case, "w4z", True, False, False)
        w[:] = 2.0 ** -3 if case[0] == 1 else w  # keeps the output in fp16's whole numbers
        out, _, _ = ref.layer(x.astype(np.float64), ids, w, fs["up"], None, fs["down"], {}, "none")
        say(f"few every expert {case}")
        got = call(gsr, x, ids, w, hs, biases, "none", workspace(gsr, case)).cpu().numpy()
        with np.errstate(over="ignore"):
            assert np.array_equal(got, out.astype(np.float16))


def test_matrices_past_32_bits(gsr):
    """A stack of more than 2^33 values: quantized, given back and multiplied, its
    matrices' bits are those of the same matrices by themselves."""
    E, K, N, O = 700, 4096, 4096, 64
    b = torch.empty(E, K, N, dtype=torch.float16, device=DEV).normal_()
    down = torch.empty(E, N, O, dtype=torch.float16, device=DEV).normal_()
    say("few past 32 bits: quantize")
    w, wd = gsr.quantize_w4(b, 64, zeros=True), gsr.quantize_w4(down, 32)
    back = gsr.dequantize_w4(w)
    pick = [333, 699]
    few, fewd = b[pick].contiguous(), down[pick].contiguous()
    v, vd = gsr.quantize_w4(few, 64, zeros=True), gsr.quantize_w4(fewd, 32)
    for i, e in enumerate(pick):
        assert torch.equal(w.codes[e], v.codes[i]) and torch.equal(w.scales[e], v.scales[i]) and torch.equal(w.zeros[e], v.zeros[i])
        assert torch.equal(back[e], gsr.dequantize_w4(gsr.W4(v.codes[i], v.scales[i], v.zeros[i], K, 64)))
    x = torch.randn(1, K, device=DEV).half() * K ** -0.5
    ids, near = torch.tensor([pick], dtype=torch.int32, device=DEV), torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    ws = gsr.new_workspace(gsr.expert_few_workspace_bytes(1, 2, E, N, O))
    for big, bigd, small, smalld in ((b, down, few, fewd), (w, wd, v, vd)):
        say("few past 32 bits: layer")
        got = gsr.expert_mlp_few(x, ids, None, big, bigd, ws, gate=big, activation="silu")
        want = gsr.expert_mlp_few(x, near, None, small, smalld, ws, gate=small, activation="silu")
        assert torch.equal(got, want) and bool(torch.isfinite(got).all()) and bool(got.count_nonzero())
