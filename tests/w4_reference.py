"""4-bit weights and the few-token layer in 64 bits on the host, by their
definitions."""
import numpy as np
import torch


def pack(q):
    """codes (..., K, N) of 0..15 as int32 words (..., ceil(K / 8), N)."""
    q = np.asarray(q, dtype=np.uint32)
    K, N = q.shape[-2:]
    words = np.zeros(q.shape[:-2] + (-(-K // 8), N), np.uint32)
    for k in range(K):
        words[..., k // 8, :] |= q[..., k, :] << np.uint32(4 * (k % 8))
    return torch.from_numpy(words.view(np.int32))


def unpack(words, K):
    w = words.cpu().numpy().view(np.uint32)
    return np.stack([(w[..., k // 8, :] >> np.uint32(4 * (k % 8))) & 15 for k in range(K)], -2).astype(np.int64)


def values(q, scales, zeros, group):
    """(q - z) s, exact in 64 bits."""
    K = q.shape[-2]
    of = np.arange(K) // group
    z = 8.0 if zeros is None else zeros.astype(np.float64)[..., of, :]
    return (q.astype(np.float64) - z) * scales.astype(np.float64)[..., of, :]


def quantize(b, group, zeros):
    """q, scales (fp16) and zero points of fp16 values b (K, N), column by column."""
    K, N = b.shape
    G = -(-K // group)
    q, s, z = np.zeros((K, N), np.int64), np.zeros((G, N), np.float16), np.full((G, N), 8, np.int64)
    for j in range(G):
        v = b[j * group:(j + 1) * group].astype(np.float64)
        bad = ~np.isfinite(v).all(0)
        v = np.where(bad, 0.0, v)
        lo, hi = np.minimum(v.min(0), 0.0), np.maximum(v.max(0), 0.0)
        # the step in binary32, then binary16
        step = (hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15) if zeros else \
            np.maximum(-lo, hi).astype(np.float32) / np.float32(7)
        s[j] = np.where(bad, np.float16(np.nan), step.astype(np.float16))
        step = s[j].astype(np.float64)
        live = step > 0
        safe = np.where(live, step, 1.0)
        if zeros:
            z[j] = np.where(live, np.clip(np.rint(-lo / safe), 0, 15), 8)
        c = np.clip(np.rint(v / safe) + z[j], 0, 15)
        q[j * group:(j + 1) * group] = np.where(live, c, z[j])
    return q, s, z


def act64(v, act):
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "relu":
            return np.where(v > 0, v, 0.0)
        if act == "gelu":
            return v / (1.0 + np.exp(-2.0 * np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)))
        if act == "silu":
            return v / (1.0 + np.exp(-v))
        return v


# How far fp32 sums and activations of the kernels may be from 64 bits.  A sum of
# n products passes at most n + 64 additions (the matrix cores' own, one per
# group, per wave and per part), each off by at most 2^-23 of the terms' absolute
# sum (2^-24 to nearest; the matrix cores may cut instead of rounding).  The
# activations' derivatives are at most 1.13 in size, and their exponential,
# reciprocal and products are off by at most 2^-20 of the value.
def sum_slack(n, magnitude):
    return (n + 64) * 2.0 ** -23 * magnitude


def act_slack(slack, v, act):
    return slack if act in ("relu", "none") else 1.13 * slack + 2.0 ** -20 * np.abs(v)


def half_step(v):
    """Half a step of fp16 at v."""
    return np.maximum(np.abs(v) * 2.0 ** -11, 2.0 ** -25)


def layer(x, ids, weights, up, gate, down, biases, act):
    """out and its slack; up, gate (or None), down (E, ., .) in 64 bits, biases a
    dict of (E, .) or None each."""
    T, k = ids.shape
    E, F, O = down.shape
    out, slack = np.zeros((T, O)), np.zeros((T, O))
    hidden = []
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0 or e >= E:
                continue

            def product(m, name):
                b = biases.get(name)
                b = np.zeros(F) if b is None else b[e]
                return x[t] @ m[e] + b, sum_slack(x.shape[1] + 1, np.abs(x[t]) @ np.abs(m[e]) + np.abs(b))

            u, du = product(up, "up")
            if gate is None:
                h, dh = act64(u, act), act_slack(du, u, act)
            else:
                g, dg = product(gate, "gate")
                a, da = act64(g, act), act_slack(dg, g, act)
                h, dh = a * u, da * np.abs(u) + du * np.abs(a) + da * du + 2.0 ** -24 * np.abs(a * u)
            # h travels as two fp16 values: 2^-22 of it, 2^-25 at least
            dh = dh + np.maximum((np.abs(h) + dh) * 2.0 ** -22, 2.0 ** -25)
            hidden.append(h)
            w = 1.0 if weights is None else float(weights[t, j])
            b = np.zeros(O) if biases.get("down") is None else biases["down"][e]
            size = np.abs(h) + dh
            out[t] += w * (h @ down[e] + b)
            slack[t] += abs(w) * (dh @ np.abs(down[e]) + sum_slack(F + 2 + k, size @ np.abs(down[e]) + np.abs(b)))
    return out, slack + half_step(np.abs(out) + slack), hidden
