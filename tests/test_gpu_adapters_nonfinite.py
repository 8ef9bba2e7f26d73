"""GPU tests of the product with low-rank adapters where a factor is an
infinity or a NaN: every output is what the formula makes of it in 64 bits, on
every tile, and finite ones keep their value."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CONFIGS = [-1, 21, 22, 28, 31, 32]
INF = float("inf")


@pytest.fixture(scope="module")
def gsr(native):
    import tiled_dense_gemm_scale_amd as g

    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return g


def say(msg):
    print("[gpu] " + msg, flush=True)


def products(x, y):
    """x @ y.T in 64 bits, product by product (0 * infinity is NaN, infinities
    of two signs add up to NaN)."""
    with np.errstate(invalid="ignore"):
        return np.stack([(x * row[None, :]).sum(1) for row in y], 1)


def formula(a, b, la, lb, ids, scales):
    """alpha 1, no bias, no activation: c, the inner sums, and per value the
    bound on what the fp32 sums, the split of the inner sum (2^-23 of its row's
    largest value) and one fp16 rounding may be off by."""
    u = 2.0 ** -24
    a64, b64, la64, lb64 = (t.double().numpy() for t in (a, b, la, lb))
    K, R = b64.shape[0], la64.shape[1]
    mag = lambda x: np.where(np.isfinite(x), np.abs(x), 0.0)
    v, t = products(a64, b64.T), np.zeros((len(a64), R))
    off = (K + 2) * u * products(mag(a64), mag(b64).T)
    with np.errstate(invalid="ignore"):
        for m, l in enumerate(ids):
            if 0 <= l < len(la64):
                t[m] = scales[l] * products(a64[m:m + 1], la64[l])[0]
                v[m] += products(t[m:m + 1], lb64[l])[0]
                tmag = abs(scales[l]) * products(mag(a64[m:m + 1]), mag(la64[l]))[0]
                terr = (K + 40) * u * tmag + 2.0 ** -23 * mag(t[m]).max()
                off[m] += products((terr + (2 * R + 4) * u * mag(t[m]))[None], mag(lb64[l]))[0]
    slack = off + 2.0 ** -11 * (mag(v) + off) + 2.0 ** -25
    # finite sums from 65520 on are rounded to fp16's infinity; none is in doubt
    past = np.isfinite(v) & (np.abs(v) >= 65520)
    assert not (np.isfinite(v) & (np.abs(np.abs(v) - 65520) <= off)).any()
    return np.where(past, np.copysign(np.inf, v), v), t, slack


def agree(got, want, slack):
    """Infinities and NaN in the same places, finite values within `slack`."""
    got = got.double().numpy()
    for name, kind in (("+inf", np.isposinf), ("-inf", np.isneginf), ("NaN", np.isnan)):
        assert np.array_equal(kind(got), kind(want)), f"{name}: {np.count_nonzero(kind(got) != kind(want))} values differ"
    fin = np.isfinite(want)
    assert np.all(np.abs(got[fin] - want[fin]) <= slack[fin])


def inputs(shape, seed):
    M, N, K, L, R = shape
    g = torch.Generator().manual_seed(seed)
    n = lambda std, *s: (torch.randn(*s, generator=g) * std).half()
    ids = np.random.default_rng(seed).integers(-1, L + 1, M).astype(np.int32)
    ids[:L] = np.arange(L)[:M]
    return n(1.0, M, K), n(K ** -0.5, K, N), n(K ** -0.5, L, R, K), n(R ** -0.5, L, N, R), ids


def calls(gsr, native, a, b, la, lb, ids, scales, act):
    """The call by every configuration, split over K, and with inner sums that
    the tiles make themselves; garbage in the workspace."""
    (M, K), N, (L, R) = a.shape, b.shape[1], la.shape[:2]
    d = [t.to(DEV) for t in (a, b, la, lb, torch.from_numpy(ids), torch.tensor(scales, dtype=torch.float32))]
    for config in CONFIGS:
        for splits, looks in [(0, -1)] + ([(3, -1), (1, 0)] if config in (21, 22) else []):
            ws = gsr.new_workspace(gsr.adapter_workspace_bytes(M, N, K, R) + (4 << 20))
            ws[512:] = 0xFF  # NaN patterns
            c = torch.full((M, N), 9.0, dtype=torch.float16, device=DEV)
            say(f"{M}x{N}x{K} of {L} rank {R} config={config} splits={splits} looks={looks}")
            native.check(native.gemm_adapters_scale_bias_act(
                M, N, K, d[0].data_ptr(), d[1].data_ptr(), 0, c.data_ptr(), L, R, d[2].data_ptr(), d[3].data_ptr(),
                d[4].data_ptr(), d[5].data_ptr(), 1.0, {"relu": 0, "none": 2}[act], ws.data_ptr(), ws.numel(),
                torch.cuda.current_stream().cuda_stream, config, splits, looks))
            yield c.cpu()
            assert bool((ws[:512] == 0).all())


SHAPES = [(1, 64, 512, 1, 8), (16, 200, 1032, 4, 16), (40, 136, 264, 3, 40), (150, 264, 520, 5, 24), (300, 264, 136, 3, 16),
          (33, 101, 77, 3, 5), (200, 301, 130, 4, 17)]


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("exact", [True, False], ids=["integers", "normal"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_infinite_lb(gsr, native, shape, exact, act):
    """Infinities of either sign and NaN in Lb meet inner sums that are exact in
    fp16 (zeros among them) and such whose two halves have one sign or two."""
    M, N, K, L, R = shape
    a, b, la, lb, ids = inputs(shape, seed=M + N)
    if exact:
        g = torch.Generator().manual_seed(K)
        a, la = torch.randint(-1, 2, a.shape, generator=g).half(), torch.randint(-1, 2, la.shape, generator=g).half()
    lb[0, 3, 0], lb[L - 1, 5, R - 1], lb[L - 1, N - 1, R // 2] = INF, -INF, INF
    lb[L // 2, 7, 0], lb[L // 2, 7, R - 1] = INF, -INF  # infinities of one sign or two
    lb[0, 9, R // 2] = float("nan")
    scales = [1.0, -0.5, 2.0, 1.0, 0.25][:L]
    want, t, slack = formula(a, b, la, lb, ids, scales)
    assert exact or np.abs(t[(ids >= 0) & (ids < L)]).min() > 1e-6  # no sign in doubt
    assert np.isposinf(want).any() and np.isneginf(want).any() or M == 1
    if act == "relu":
        want = np.where(want > 0, want, 0.0)
    for got in calls(gsr, native, a, b, la, lb, ids, scales, act):
        agree(got, want, slack)


def positive_inputs(shape, seed):
    """Factors above zero, A of either sign: an infinite inner sum makes
    infinities of one sign of its row."""
    a, b, la, lb, ids = inputs(shape, seed)
    return a, b.abs() + 2.0 ** -10, la.abs() + 2.0 ** -10, lb.abs() + 2.0 ** -10, ids


@pytest.mark.parametrize("shape", [(1, 64, 512, 1, 16), (16, 200, 1032, 4, 48), (150, 264, 520, 5, 16), (300, 264, 136, 3, 48),
                                   (300, 136, 72, 2, 240)], ids=lambda s: "x".join(map(str, s)))
def test_infinite_la(gsr, native, shape):
    """An infinity in La makes an infinite inner sum in every row of its adapter,
    whose chunk of ranks may be the last of an odd count."""
    a, b, la, lb, ids = positive_inputs(shape, seed=shape[0] + 1)
    a = torch.where(a == 0, torch.ones_like(a), a)
    la[0, 2, 7] = INF
    la[-1, shape[4] - 1, 9] = -INF
    scales = [1.0, -0.5, 2.0, 1.0, 0.25][:shape[3]]
    want, _, slack = formula(a, b, la, lb, ids, scales)
    assert np.isinf(want).any()
    for got in calls(gsr, native, a, b, la, lb, ids, scales, "none"):
        agree(got, want, slack)


@pytest.mark.parametrize("shape", [(1, 64, 512, 1, 1), (16, 200, 1032, 4, 8), (40, 136, 264, 3, 24), (150, 264, 520, 5, 40),
                                   (300, 136, 72, 2, 200), (33, 101, 77, 3, 5), (200, 301, 130, 4, 17)],
                         ids=lambda s: "x".join(map(str, s)))
def test_infinite_a(gsr, native, shape):
    """An infinity in A, with a rank that fills no whole chunks: the ranks that
    are not there add nothing."""
    a, b, la, lb, ids = positive_inputs(shape, seed=shape[0] + 2)
    a[0, 5] = INF
    a[-1, 1] = INF if len(a) == 1 else -INF
    a[len(a) // 2, shape[2] - 1] = INF
    scales = [1.0, 0.5, 2.0, 1.0, 0.25][:shape[3]]
    want, _, slack = formula(a, b, la, lb, ids, scales)
    assert np.isinf(want).any() and not np.isnan(want).any()
    for got in calls(gsr, native, a, b, la, lb, ids, scales, "none"):
        agree(got, want, slack)


@pytest.mark.parametrize("shape", [(1, 64, 512, 1, 16), (16, 200, 1032, 4, 8), (40, 136, 264, 3, 24), (150, 264, 520, 5, 40),
                                   (300, 264, 136, 3, 16), (300, 136, 72, 2, 256), (33, 101, 77, 3, 5), (200, 301, 130, 4, 17)],
                         ids=lambda s: "x".join(map(str, s)))
def test_infinities_on_both_sides(gsr, native, shape):
    """Infinite inner sums meet infinities of Lb, and infinite products of A and B
    meet infinite ones of the adapter, of the same sign and of the other."""
    a, b, la, lb, ids = positive_inputs(shape, seed=shape[0] + 3)
    a[len(a) // 2, 1] = -INF
    b[2, 11], b[3, 12] = INF, -INF
    a[:, 2:4] = a[:, 2:4].abs() + 1.0  # B's infinities come through with their sign
    a = torch.where(a == 0, torch.ones_like(a), a)
    la[0, 0, 4] = INF
    lb[0, 3, 0], lb[0, 5, shape[4] - 1] = INF, -INF
    lb[-1, 11, 0], lb[-1, 12, 0], lb[-1, 13, 0] = INF, INF, -INF
    scales = [1.0, 0.5, 2.0, 1.0, 0.25][:shape[3]]
    want, t, slack = formula(a, b, la, lb, ids, scales)
    fin = np.isfinite(t) & ((ids >= 0) & (ids < shape[3]))[:, None]
    assert not fin.any() or np.abs(t[fin]).min() > 1e-6  # no sign in doubt
    for got in calls(gsr, native, a, b, la, lb, ids, scales, "none"):
        agree(got, want, slack)


@pytest.mark.parametrize("shape", [(1, 64, 512, 1, 16), (16, 200, 1032, 4, 8), (40, 136, 264, 3, 24), (150, 264, 520, 5, 40),
                                   (300, 136, 72, 2, 256), (33, 101, 77, 3, 5), (200, 301, 130, 4, 17)],
                         ids=lambda s: "x".join(map(str, s)))
def test_inner_sums_of_unlike_size_keep_their_sign(gsr, native, shape):
    """An inner sum of 2^-30 and less of its row's largest, which leaves finite
    outputs alone, gives its sign to an infinity of Lb; and one far above fp16's
    range in a row with an infinite one stays finite beside it."""
    M, N, K, L, R = shape
    a, b, la, lb, ids = positive_inputs(shape, seed=shape[0] + 4)
    g = torch.Generator().manual_seed(K)
    a = torch.randint(1, 3, a.shape, generator=g).half()
    la[:, 0] = 100.0
    la[:, R - 1] = torch.randint(0, 2, (L, K), generator=g).half() * 2.0 ** -23 - 2.0 ** -24  # +-2^-24
    lb[:, 3, R - 1], lb[:, 6, R - 1] = INF, -INF
    la[L - 1, 1, 2], la[L - 1, 2] = INF, 60000.0
    lb[L - 1, :, 2] *= -1.0
    scales = [1.0, -0.5, 2.0, 1.0, 0.25][:L]
    want, t, slack = formula(a, b, la, lb, ids, scales)
    ours = t[(ids >= 0) & (ids < L)]
    assert (np.abs(ours[:, R - 1]) <= 2.0 ** -26 * np.nanmax(np.abs(np.where(np.isfinite(ours), ours, 0.0)), 1)).all()
    assert np.isinf(want[ids == L - 1][:, 8:]).all()
    for got in calls(gsr, native, a, b, la, lb, ids, scales, "none"):
        agree(got, want, slack)
