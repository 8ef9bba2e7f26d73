"""GPU tests of what the few-token layer keeps of h between its launches: the
rounded half and the rest, over fp16's range and far below it."""
import numpy as np
import pytest
import torch

import w4_reference as ref
from test_gpu_few import CASES, FORMS, call, case_inputs, dev, workspace

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gsr(native):
    import tiled_dense_gemm_scale_amd as g

    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return g


def say(msg):
    print("[gpu] " + msg, flush=True)


def whole_weights(gsr, form, group, v, scale=None):
    """Whole numbers v (E, K, N) of -8 .. 5 as weights of `form`, times `scale`
    (E, groups, N), a power of two."""
    E, K, N = v.shape
    G = -(-K // group)
    s = np.ones((E, G, N)) if scale is None else scale
    if form == "fp16":
        return dev((v * s[:, np.arange(K) // group]).astype(np.float16))
    z = None if form == "w4" else np.full((E, G, N), 10, np.uint8)
    q = v + (8 if z is None else 10)
    return gsr.W4(ref.pack(q).to(DEV), dev(s.astype(np.float16)), dev(z), K, group)


def layer(gsr, x, ids, weights, up, down, F, O, E, act="none"):
    T, k = ids.shape
    ws = gsr.new_workspace(gsr.expert_few_workspace_bytes(T, k, E, F, O))
    return gsr.expert_mlp_few(dev(x), dev(ids), dev(weights), up, down, ws, activation=act).cpu().numpy()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("tokens", [1, 3, 37])
def test_rests_of_h_arrive(gsr, form, group, tokens):
    """h = 4096 + c with c up to 8, of which fp16 keeps whole fours; the weights of
    two neighbouring h cancel the 4096, so the outputs are sums of the rests of all
    of F, its ragged end too, exactly."""
    E, H, F, O = 2, 70, 846, 70
    rng = np.random.default_rng(tokens + group)
    up = np.zeros((E, H, F), np.int64)
    up[:, 0] = 4
    up[:, H - 1] = rng.integers(-8, 6, (E, F))
    down = np.repeat(rng.integers(-5, 6, (E, F // 2, O)), 2, axis=1)
    down[:, 1::2] *= -1
    G = -(-F // group)
    scale = 2.0 ** rng.integers(0, 3, (E, G, O))
    x = np.zeros((tokens, H), np.float16)
    x[:, 0], x[:, H - 1] = 1024.0, rng.choice([1.0, -1.0, 0.5], tokens)
    ids = rng.integers(0, E, (tokens, 1)).astype(np.int32)
    h = [x[t].astype(np.float64) @ up[ids[t, 0]] for t in range(tokens)]
    assert all(np.count_nonzero(v != v.astype(np.float16).astype(np.float64)) > F // 3 for v in h)

    def sums(h):
        return np.stack([h[t] @ (down[ids[t, 0]] * scale[ids[t, 0]][np.arange(F) // group]) for t in range(tokens)])

    want = sums(h)
    # what the outputs would be without the rests, and with them in another place of their eights
    rounded = [v.astype(np.float16).astype(np.float64) for v in h]
    order = np.arange(F) // 8 * 8 + (np.arange(F) % 8 * 2 + np.arange(F) % 8 // 4) % 8
    order = np.where(order < F, order, np.arange(F))
    moved = [r + (v - r)[order] for r, v in zip(rounded, h)]
    for other in (rounded, moved):
        assert (np.abs(sums(other) - want) > ref.half_step(want) * 2).mean() > 0.5
    say(f"few rests {form} group={group} tokens={tokens}")
    got = layer(gsr, x, ids, None, whole_weights(gsr, form, group, up), whole_weights(gsr, form, group, down, scale), F, O, E)
    assert np.array_equal(got, want.astype(np.float16)), f"{np.count_nonzero(got != want.astype(np.float16))} of {want.size}"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("O", [1, 3, 40])
def test_h_below_fp16(gsr, form, group, O):
    """Three of four h are 2^-26, which fp16 rounds to zero, and one 3 2^-26, which it
    rounds to 2^-24: their sums."""
    E, H, F = 1, 8, 4096
    up = np.zeros((E, H, F), np.int64)
    up[:, 0], up[:, 0, 1::4] = 1, 3
    down = np.ones((E, F, O), np.int64)
    x = np.zeros((2, H), np.float16)
    x[0, 0], x[1, 0] = 2.0 ** -14, -(2.0 ** -14)
    su = np.full((E, 1, F), 2.0 ** -12)
    ids = np.zeros((2, 1), np.int32)
    say(f"few h below fp16 {form} group={group} O={O}")
    got = layer(gsr, x, ids, None, whole_weights(gsr, form, group, up, su.repeat(-(-H // group), 1)),
                whole_weights(gsr, form, group, down), F, O, E)
    want = F // 4 * 6 * 2.0 ** -26
    assert np.array_equal(got, np.repeat(np.array([[want], [-want]], np.float16), O, 1))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("size", [2.0 ** -3, 2.0 ** -10, 2.0 ** -14, 2.0 ** -20])
def test_small_h_keeps_its_bits(gsr, form, size):
    """Normal h of that size, its outputs brought back up by the weights of the
    choices: within 2^-22 of each h or 2^-36, and the sums' slack."""
    T, k, E, H, F, O, group = 5, 2, 3, 64, 1100, 72, 64
    case = (T, k, E, H, F, O, 0.0, group)
    x, ids, w, hs, fs, _ = case_inputs(gsr, case, form, False, False, False, seed=7)
    x = (x.astype(np.float64) * size).astype(np.float16)
    w = (w / size).astype(np.float32)
    none = dict(up=None, gate=None, down=None)
    out, slack = np.zeros((T, O)), np.zeros((T, O))
    x64 = x.astype(np.float64)
    for t in range(T):
        for j in range(k):
            e, weight = int(ids[t, j]), float(w[t, j])
            h = x64[t] @ fs["up"][e]
            dh = ref.sum_slack(H + 1, np.abs(x64[t]) @ np.abs(fs["up"][e]))
            dh = dh + np.maximum((np.abs(h) + dh) * 2.0 ** -22, 2.0 ** -36)
            out[t] += weight * (h @ fs["down"][e])
            slack[t] += weight * (dh @ np.abs(fs["down"][e]) +
                                  ref.sum_slack(F + 2 + k, (np.abs(h) + dh) @ np.abs(fs["down"][e])))
    slack = slack + ref.half_step(np.abs(out) + slack)
    say(f"few small h {form} {size}")
    got = call(gsr, x, ids, w, hs, none, "none", workspace(gsr, case)).cpu().numpy().astype(np.float64)
    err = np.abs(got - out)
    say(f"few small h {form} {size}: worst {float((err / slack).max()):.3f} of its bound")
    assert (err <= slack).all()


@pytest.mark.parametrize("O", [3, 29])
def test_infinite_weight_meets_a_small_h(gsr, O):
    """Any h that is not zero makes an infinity of its sign with an infinite weight."""
    H, F = 8, 45
    x = np.zeros((4, H), np.float16)
    x[:, 0] = 2.0 ** -15, -(2.0 ** -15), 2.0 ** -24, -(2.0 ** -24)
    up = np.full((1, H, F), 2.0 ** -16, np.float16)  # h of 2^-31 and 2^-40
    down = np.ones((1, F, O), np.float16)
    down[0, F - 1, O - 1], down[0, 2, 0] = np.inf, -np.inf
    ids = np.zeros((4, 1), np.int32)
    say(f"few infinite weight, small h, O={O}")
    got = layer(gsr, x, ids, None, dev(up), dev(down), F, O, 1)
    sign = np.array([1.0, -1.0, 1.0, -1.0])
    assert np.array_equal(got[:, O - 1], sign * np.inf) and np.array_equal(got[:, 0], -sign * np.inf)
    assert np.isfinite(got[:, 1:O - 1]).all()


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("case", [c for c in CASES if c[3] > 24], ids=lambda c: "x".join(map(str, c)))
def test_whole_numbers_all_over_h(gsr, case, form, gated):
    """Inputs that are not zero at 24 places of all of H, its last among them."""
    T, k, E, H, F, O, drop, group = case
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, True, gated, True, seed=3)
    rng = np.random.default_rng(H)
    keep = np.append(rng.choice(H - 1, 23, replace=False), H - 1)
    x[:, np.setdiff1d(np.arange(H), keep)] = 0
    x[:, H - 1] = rng.choice([-1.0, 1.0], T)
    b64 = {n: None if b is None else b.astype(np.float64) for n, b in biases.items()}
    out, _, hidden = ref.layer(x.astype(np.float64), ids, w, fs["up"], fs["gate"], fs["down"], b64, "none")
    assert not hidden or max(np.abs(h).max() for h in hidden) <= 2048
    say(f"few whole over H {case} {form} gated={gated}")
    got = call(gsr, x, ids, w, hs, biases, "none", workspace(gsr, case)).cpu().numpy()
    with np.errstate(over="ignore"):
        want = out.astype(np.float16)
    assert np.array_equal(got, want), f"{np.count_nonzero(got != want)} of {want.size} differ"


@pytest.mark.parametrize("form", FORMS)
def test_weights_of_choices_that_are_not_finite(gsr, form):
    """They make their token's outputs not finite, and no other's."""
    case = (6, 2, 4, 40, 1100, 50, 0.0, 64)
    x, ids, w, hs, fs, biases = case_inputs(gsr, case, form, False, False, True, seed=2)
    ws = workspace(gsr, case)
    base = call(gsr, x, ids, w, hs, biases, "gelu", ws).cpu().numpy()
    w[1, 0], w[4, 1] = np.inf, np.nan
    say(f"few weights not finite {form}")
    got = call(gsr, x, ids, w, hs, biases, "gelu", ws).cpu().numpy()
    bad = np.isin(np.arange(6), (1, 4))
    assert np.array_equal(got[~bad], base[~bad]) and not np.isfinite(got[bad]).any()
