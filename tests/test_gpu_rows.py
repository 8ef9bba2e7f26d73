"""GPU tests of the row operators against their definitions in 64 bits on the
host: the sort exactly, the copies bit for bit, the sums within the rounding of
their types (half a step of the output, 2^-24 per fp32 addition)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gsr(native):
    import tiled_dense_gemm_scale_amd as g

    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return g


def say(msg):
    print("[gpu] " + msg, flush=True)


def plan_of(ids, groups):
    """offsets, rows, positions by the definition (numpy, slot by slot order)."""
    flat, k = np.asarray(ids).reshape(-1), ids.shape[1] if ids.ndim == 2 else 1
    offsets, rows = [0], np.full(flat.size, -1, np.int32)
    positions = np.full(flat.size, -1, np.int32)
    for e in range(groups):
        slots = np.flatnonzero(flat == e)
        rows[offsets[-1]:offsets[-1] + slots.size] = slots // k
        positions[slots] = np.arange(offsets[-1], offsets[-1] + slots.size)
        offsets.append(offsets[-1] + slots.size)
    return np.array(offsets, np.int32), rows, positions.reshape(ids.shape)


def routing(T, k, groups, drop=0.0, seed=0):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, groups)) * (0.2 + rng.random(groups)), axis=1)[:, :k]
    ids = np.where(rng.random((T, k)) < drop, -1, ids)
    weights = rng.random((T, k)).astype(np.float32)
    return ids, torch.from_numpy(weights / np.maximum(weights.sum(1, keepdims=True), 1e-3))


GROUPS = [(1, 1, 1), (1, 8, 64), (32, 2, 8), (63, 1, 5), (65, 3, 7), (1000, 1, 1024), (1025, 4, 63), (4096, 2, 8),
          (8193, 1, 1000), (2731, 3, 16), (16384, 8, 64), (100001, 1, 3), (40000, 7, 129)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("case", GROUPS, ids=lambda c: "x".join(map(str, c)))
def test_group_rows(gsr, case, dtype):
    T, k, E = case
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(-2, E + 2, (T, k))  # some dropped, on both sides
    if dtype == torch.int64:
        ids = np.where(rng.random((T, k)) < 0.05, (1 << 32) + rng.integers(0, E, (T, k)), ids)
    say(f"group {case} {dtype}")
    got = gsr.group_rows(torch.from_numpy(ids).to(dtype).to(DEV), E)
    for name, g, want in zip(("offsets", "rows", "positions"), got, plan_of(ids, E)):
        assert np.array_equal(g.cpu().numpy(), want), name


@pytest.mark.parametrize("case", [(300001, 2, 1024), (1100001, 2, 5)], ids=lambda c: "x".join(map(str, c)))
def test_group_rows_many(gsr, case):
    """Larger blocks for many groups, and runs too long to keep in registers
    (more than 256 blocks of 8192 slots)."""
    T, k, E = case
    ids = np.random.default_rng(E).integers(-1, E, (T, k), dtype=np.int32)
    say(f"group many {case}")
    for g, want in zip(gsr.group_rows(torch.from_numpy(ids).to(DEV), E), plan_of(ids, E)):
        assert np.array_equal(g.cpu().numpy(), want)


@pytest.mark.parametrize("fill", ["one", "none", "last"])
@pytest.mark.parametrize("n", [64, 5000, 20000])
def test_group_rows_lopsided(gsr, fill, n):
    """Every slot in one group, in none, or in the last."""
    E = 37
    ids = np.full((n, 1), {"one": 5, "none": E, "last": E - 1}[fill])
    say(f"group all in {fill} n={n}")
    got = gsr.group_rows(torch.from_numpy(ids).int().to(DEV), E)
    for g, want in zip(got, plan_of(ids, E)):
        assert np.array_equal(g.cpu().numpy(), want)


def test_group_rows_empty_and_flat(gsr):
    say("group of no slots")
    o, r, p = gsr.group_rows(torch.empty(0, 4, dtype=torch.int32, device=DEV), 6)
    assert o.cpu().tolist() == [0] * 7 and r.numel() == 0 and tuple(p.shape) == (0, 4)
    ids = torch.tensor([2, 0, 2, 1, -1, 0], dtype=torch.int32, device=DEV)
    o, r, p = gsr.group_rows(ids, 3)
    assert o.cpu().tolist() == [0, 2, 3, 5] and r.cpu().tolist() == [1, 5, 3, 0, 2, -1]
    assert p.cpu().tolist() == [3, 0, 4, 2, -1, 1]


WIDTHS = [1, 2, 7, 8, 36, 64, 513, 1001, 4096, 8200]


@pytest.mark.parametrize("offset", [0, 1, 2, 4], ids=lambda o: f"+{2 * o}B")
@pytest.mark.parametrize("H", WIDTHS)
def test_gather_rows(gsr, H, offset):
    """Every unit of the copy: bit patterns of any kind, indices out of range
    and repeated, values beside the output left alone."""
    T, P = 37, 101
    rng = np.random.default_rng(H)
    xb = rng.integers(0, 1 << 16, (T, H)).astype(np.uint16)
    rows = rng.integers(-2, T + 3, P).astype(np.int32)
    buf = torch.empty(T * H + 8, dtype=torch.float16, device=DEV)
    x = buf[offset:offset + T * H].view(T, H)
    x.copy_(torch.from_numpy(xb.view(np.int16)).view(torch.float16))
    obuf = torch.full((P * H + 8,), 3.0, dtype=torch.float16, device=DEV)
    out = obuf[offset:offset + P * H].view(P, H)
    say(f"gather H={H} offset={offset}")
    gsr.gather_rows(x, torch.from_numpy(rows).to(DEV), out=out)
    got = out.cpu().view(torch.int16).numpy().view(np.uint16)
    ok = (rows >= 0) & (rows < T)
    want = np.where(ok[:, None], xb[np.clip(rows, 0, T - 1)], 0)
    assert np.array_equal(got, want)
    host = obuf.cpu()
    assert bool((host[:offset] == 3.0).all()) and bool((host[offset + P * H:] == 3.0).all())


def within(name, got, ref, slack):
    """|got - ref| <= slack elementwise; prints the worst share of it."""
    err = np.abs(got - ref)
    worst = float(np.max(err / slack)) if err.size else 0.0
    say(f"{name}: worst error {worst:.3f} of its bound")
    assert np.all(err <= slack), name


HALF16 = 2.0 ** -11  # half a step of fp16, relative; 2^-25 below its normal range
CASES = [(1, 1, 4, 64, 0.0), (1, 8, 64, 4096, 0.0), (16, 8, 64, 4096, 0.3), (129, 2, 8, 1001, 0.1), (33, 5, 9, 36, 0.2),
         (257, 3, 16, 513, 0.0), (40, 2, 8, 8200, 0.05), (7, 17, 40, 7, 0.1), (300, 1, 4, 1, 0.5), (64, 2, 4, 256, 1.0)]


def combine_inputs(case, seed=0):
    T, k, E, H, drop = case
    ids, w = routing(T, k, E, drop, seed)
    offsets, rows, positions = plan_of(ids, E)
    g = torch.Generator().manual_seed(seed + 1)
    y = torch.randn(T * k, H, generator=g).half()
    y[int(offsets[-1]):] = float("nan")  # rows that no choice names
    dout = torch.randn(T, H, generator=g).half()
    return rows, positions, w, y, dout


@pytest.mark.parametrize("weighted", [True, False], ids=["w", "ones"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_combine_rows(gsr, case, weighted):
    T, k, E, H, drop = case
    rows, positions, w, y, _ = combine_inputs(case)
    w = w if weighted else None
    say(f"combine {case} weighted={weighted}")
    out = gsr.combine_rows(y.to(DEV), torch.from_numpy(positions).to(DEV), w.to(DEV) if weighted else None)
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    y64 = y.double().numpy()
    for j in range(k):
        ok = positions[:, j] >= 0
        term = y64[positions[ok, j]] * (w[ok, j].double().numpy()[:, None] if weighted else 1.0)
        ref[ok] += term
        mag[ok] += np.abs(term)
    # k products and additions in fp32, then one rounding to fp16
    acc = (k + 1) * 2.0 ** -24 * mag
    within("combine", out.cpu().double().numpy(), ref, acc + HALF16 * (np.abs(ref) + acc) + 2.0 ** -25)


@pytest.mark.parametrize("weighted", [True, False], ids=["w", "ones"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_combine_rows_backward(gsr, case, weighted):
    T, k, E, H, drop = case
    rows, positions, w, y, dout = combine_inputs(case, seed=3)
    dy0 = torch.full((T * k, H), float("nan"), dtype=torch.float16, device=DEV)
    say(f"combine backward {case} weighted={weighted}")
    dy, dw = gsr.combine_rows_backward(dout.to(DEV), y.to(DEV) if weighted else None,
                                       torch.from_numpy(positions).to(DEV), w.to(DEV) if weighted else None,
                                       torch.from_numpy(rows).to(DEV), dy=dy0)
    assert dy.data_ptr() == dy0.data_ptr()
    ref, refw, magw = np.zeros((T * k, H)), np.zeros((T, k)), np.zeros((T, k))
    d64, y64, w64 = dout.double().numpy(), y.double().numpy(), w.double().numpy() if weighted else np.ones((T, k))
    for j in range(k):
        ok = positions[:, j] >= 0
        ref[positions[ok, j]] = w64[ok, j][:, None] * d64[ok]
        prod = d64[ok] * y64[positions[ok, j]]
        refw[ok, j], magw[ok, j] = prod.sum(1), np.abs(prod).sum(1)
    # one fp32 product, one rounding to fp16
    within("dy", dy.cpu().double().numpy(), ref, (HALF16 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -25)
    if not weighted:
        assert dw is None
        return
    # a lane adds at most 8 ceil(H / 512) products, then six additions over the lanes
    terms = 8 * -(-H // 512) + 6
    within("dweights", dw.cpu().double().numpy(), refw, terms * 2.0 ** -24 * magw + 1e-37)


@pytest.mark.parametrize("case", [(50, 3, 500), (50, 5, 1000), (50, 3, 2056), (50, 2, 4104), (50, 3, 4104), (50, 1, 8192),
                                  (70000, 8, 64), (8400, 4, 1000), (4100, 4, 2056), (4100, 2, 4104), (2100, 4, 4096),
                                  (8400, 1, 4096), (1400, 6, 4097)], ids=lambda c: "x".join(map(str, c)))
def test_combine_rows_backward_by_length(gsr, case):
    """Every form that the length of a row, the choices and the size of y
    (above and below 64 MiB) select, against the formula in 64 bits on the
    device."""
    T, k, H = case
    g = torch.Generator().manual_seed(T + H)
    ids = torch.randint(-1, 8, (T, k), generator=g).to(DEV)
    offsets, rows, positions = gsr.group_rows(ids, 8)
    w = torch.randn(T, k, generator=g).to(DEV)
    dg = torch.Generator(device=DEV).manual_seed(H)
    y = torch.randn(T * k, H, device=DEV, generator=dg).half()
    y[int(offsets[-1]):] = float("nan")
    dout = torch.randn(T, H, device=DEV, generator=dg).half()
    say(f"combine backward by length {case}")
    dy, dw = gsr.combine_rows_backward(dout, y, positions, w, rows,
                                       dy=torch.full((T * k, H), float("nan"), dtype=torch.float16, device=DEV))
    assert bool((dy[int(offsets[-1]):] == 0).all())
    for j in range(k):
        at, ok = positions[:, j].long(), positions[:, j] >= 0
        d, q = dout[ok].double(), at[ok]
        ref = w[ok, j].double()[:, None] * d
        assert bool(((dy[q].double() - ref).abs() <= (HALF16 + 2.0 ** -23) * ref.abs() + 2.0 ** -25).all())
        prod = d * y[q].double()
        # a lane adds at most 8 ceil(H / 512) products, then six additions over the lanes
        slack = (8 * -(-H // 512) + 6) * 2.0 ** -24 * prod.abs().sum(1) + 1e-37
        assert bool(((dw[ok, j].double() - prod.sum(1)).abs() <= slack).all())
        assert bool((dw[~ok, j] == 0).all())


def test_combine_gradient_by_differences(gsr):
    """<dout, combine(y + h v) - combine(y - h v)> / 2h against <dy, v> (and the
    same for the weights): the operator is linear in each, so the difference
    is exact up to the roundings of the two fp16 outputs."""
    T, k, E, H = 50, 3, 8, 200
    rows, positions, w, y, dout = combine_inputs((T, k, E, H, 0.1), seed=7)
    y = torch.nan_to_num(y)
    pos, wd = torch.from_numpy(positions).to(DEV), w.to(DEV)
    g = torch.Generator().manual_seed(11)
    say("combine gradient by differences")
    dy, dw = gsr.combine_rows_backward(dout.to(DEV), y.to(DEV), pos, wd, torch.from_numpy(rows).to(DEV))
    v = torch.randint(-1, 2, y.shape, generator=g).half()
    up, down = (gsr.combine_rows((y + s * v).to(DEV), pos, wd).cpu().double() for s in (1.0, -1.0))
    yup, ydown = (y + v).double(), (y - v).double()
    step = (yup - ydown) / 2  # what the fp16 inputs really moved by
    got = float((dout.double() * (up - down) / 2).sum())
    want = float((dy.cpu().double() * step).sum())
    # each output is off by half a step of fp16, each dy value too
    slack = float((dout.double().abs() * (up.abs() + down.abs()) / 2).sum() + (dy.cpu().double() * step).abs().sum()) * 2.0 ** -10
    assert abs(got - want) <= slack, (got, want, slack)
    vw = torch.randint(-1, 2, w.shape, generator=g).float() * 0.25
    up, down = (gsr.combine_rows(y.to(DEV), pos, (w + s * vw).to(DEV)).cpu().double() for s in (1.0, -1.0))
    got = float((dout.double() * (up - down) / 2).sum())
    want = float((dw.cpu().double() * ((w + vw).double() - (w - vw).double()) / 2).sum())
    slack = float((dout.double().abs() * (up.abs() + down.abs()) / 2).sum()) * 2.0 ** -10 + 1e-3
    assert abs(got - want) <= slack, (got, want, slack)


def test_rows_past_32_bit_offsets(gsr):
    """A table of more than 2^31 bytes (and 2^31 values): rows near its end."""
    T, H = 70000, 32768
    x = torch.zeros(T, H, dtype=torch.float16, device=DEV)
    marks = torch.tensor([0, 1, 32767, 65536, T - 1], device=DEV)
    x[marks] = (marks % 1000).half()[:, None] + 1.0
    say("rows past 32-bit offsets")
    rows = torch.tensor([T - 1, 0, 65536, 32767, T, 1], dtype=torch.int32, device=DEV)
    out = gsr.gather_rows(x, rows)
    assert [float(v) for v in out[:, 0]] == [float((T - 1) % 1000 + 1), 1.0, 537.0, 768.0, 0.0, 2.0]
    assert bool((out == out[:, :1]).all())
    both = gsr.combine_rows(x, rows.reshape(3, 2))
    assert [float(v) for v in both[:, -1]] == [float((T - 1) % 1000 + 2), 1305.0, 2.0]
    dy, dw = gsr.combine_rows_backward(both, x, rows.reshape(3, 2)[:, :1].contiguous(),
                                       torch.ones(3, 1, device=DEV), torch.full((T,), 0, dtype=torch.int32, device=DEV),
                                       dy=x.clone())
    assert torch.equal(dy[T - 1], both[0]) and torch.equal(dy[65536], both[1]) and float(dy[1, 0]) == 2.0


def test_rows_on_another_stream_and_captured(gsr):
    """The plan, the copy, the sum and its gradient on a side stream, then
    captured into a graph and replayed with new inputs in the same buffers,
    eager work between the replays."""
    T, k, E, H = 300, 2, 16, 520
    s = torch.cuda.Stream()
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    x = torch.empty(T, H, dtype=torch.float16, device=DEV)
    w = torch.empty(T, k, device=DEV)
    ws = gsr.new_workspace(gsr.group_workspace_bytes(T * k, E))

    def fill(seed):
        a, b = routing(T, k, E, 0.1, seed)
        ids.copy_(torch.from_numpy(a).int())
        w.copy_(b)
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).half())
        torch.cuda.synchronize()
        return a

    def chain(stream=None):
        o, r, p = gsr.group_rows(ids, E, workspace=ws, stream=stream)
        xs = gsr.gather_rows(x, r, stream=stream)
        out = gsr.combine_rows(xs, p, w, stream=stream)
        dy, dw = gsr.combine_rows_backward(out, xs, p, w, r, stream=stream)
        return o, r, p, xs, out, dy, dw

    fill(1)
    say("row operators on a side stream")
    side = chain(stream=s)
    torch.cuda.synchronize()
    here = chain()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(side, here))
    raw = chain(stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(raw, here))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = chain()
    for seed in (2, 3, 4):
        a = fill(seed)
        say(f"row operators replayed, inputs {seed}")
        g.replay()
        torch.cuda.synchronize()
        want = chain()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(held, want))
        assert np.array_equal(held[2].cpu().numpy(), plan_of(a, E)[2])


def test_python_refusals_on_the_device(gsr):
    i32 = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    h = torch.zeros(8, 16, dtype=torch.float16, device=DEV)
    r = torch.zeros(8, dtype=torch.int32, device=DEV)
    for bad in (lambda: gsr.group_rows(i32, 4, rows=r[:7]), lambda: gsr.group_rows(i32.t(), 4),
                lambda: gsr.gather_rows(h.t(), r), lambda: gsr.gather_rows(h, r, out=h[:4]),
                lambda: gsr.combine_rows(h, i32, torch.zeros(4, 3, device=DEV)),
                lambda: gsr.combine_rows(h, i32.t()),
                lambda: gsr.combine_rows_backward(h, h, i32, None, r),
                lambda: gsr.combine_rows_backward(h[:4], None, i32, torch.zeros(4, 2, device=DEV), r),
                lambda: gsr.combine_rows_backward(h[:4], h, i32, None, r, dweights=torch.zeros(4, 2, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gsr.gather_rows(h, r, out=h), lambda: gsr.group_rows(i32, 0), lambda: gsr.group_rows(i32, 1025)):
        with pytest.raises(gsr.GsrError):
            bad()


def test_group_rows_of_the_largest_count(gsr):
    """2^31 - 1 slots, whose last block ends at 2^31: every slot in its place."""
    n, E, period = 2 ** 31 - 1, 7, 8  # slot i has id i mod 8; 7 is dropped
    ids = torch.arange(n, dtype=torch.int32, device=DEV)
    ids.remainder_(period)
    offsets = torch.full((E + 1,), -7, dtype=torch.int32, device=DEV)
    rows, positions = (torch.full((n,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    say(f"group of {n} slots")
    gsr.group_rows(ids, E, offsets=offsets, rows=rows, positions=positions)
    torch.cuda.synchronize()
    counts = [(n - e + period - 1) // period for e in range(E)]
    starts = [sum(counts[:e]) for e in range(E + 1)]
    assert offsets.tolist() == starts
    say("group of the largest count: positions")
    base = torch.tensor(starts[:E] + [0], device=DEV)
    step = 1 << 27
    for lo in range(0, n, step):
        i = torch.arange(lo, min(lo + step, n), device=DEV)
        want = torch.where(i % period < E, base[i % period] + i // period, -1)
        assert torch.equal(positions[lo:lo + step].long(), want)
    say("group of the largest count: rows")
    for e in range(E):
        for lo in range(0, counts[e], step):
            i = torch.arange(lo, min(lo + step, counts[e]), device=DEV)
            assert torch.equal(rows[starts[e] + lo:starts[e] + lo + i.numel()].long(), i * period + e)
    for lo in range(starts[E], n, step):
        assert bool((rows[lo:lo + step] == -1).all())
    del ids, rows, positions
    torch.cuda.empty_cache()


def test_more_rows_than_a_grid_has_threads(gsr):
    """Rows x 256 threads past 2^32: 2^24 + 3 rows of 129 odd values for gather and
    combine, 2^26 + 5 tokens of one value for the gradient."""
    n, H, T = (1 << 24) + 3, 129, 1000
    x = torch.randint(-50, 50, (T, H), device=DEV).half()
    rows = torch.arange(n, device=DEV).remainder_(T + 1).int()  # T itself is no row
    padded = torch.cat([x, torch.zeros(1, H, dtype=torch.float16, device=DEV)])
    for name, go in (("gather", lambda: gsr.gather_rows(x, rows)), ("combine", lambda: gsr.combine_rows(x, rows))):
        say(f"{name} of {n} rows of {H}")
        out = go()
        for lo in range(0, n, 1 << 22):
            assert torch.equal(out[lo:lo + (1 << 22)], padded[rows[lo:lo + (1 << 22)].long()])
        del out
    n = (1 << 26) + 5
    say(f"gradient of {n} tokens")
    dout = torch.arange(n, device=DEV).remainder_(2000).half()[:, None]
    positions = torch.arange(n, device=DEV).flip(0).int()[:, None]
    w = torch.full((n, 1), 0.5, device=DEV)
    y = torch.full((n, 1), 2.0, dtype=torch.float16, device=DEV)
    rows = positions.flatten().clone()
    rows[7] = -1  # token n - 8's row, which then no choice names
    positions[n - 8] = -1
    dy, dw = gsr.combine_rows_backward(dout, y, positions, w, rows)
    want = 0.5 * dout.flip(0)
    want[7] = 0
    assert torch.equal(dy, want)
    want = 2.0 * dout.float()
    want[n - 8] = 0
    assert torch.equal(dw, want)
