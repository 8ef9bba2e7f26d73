"""The operators for a few tokens as workloads: products with 4-bit weights,
and the whole layer of routed experts in fp16 and in 4 bits; their inputs, one
pass through each, its plain form in elementary torch operations, and what a
pass cannot do without.

4-bit weights of a K x N matrix are codes q in 0..15, eight of consecutive k in
one 32-bit word (bits 4i .. 4i + 3 hold k = 8r + i), an fp16 scale s for each
column and each group of `group` values of k, and a zero point z likewise (8
everywhere where there are none); the weight is (q - z) s.

  round_trip  quantize and give the values back.  Without zeros
              s = fp16(max|b| / 7), q = clamp(rint(b / s), -8, 7) + 8; with
              them lo = min(b, 0), hi = max(b, 0) over the group,
              s = fp16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15),
              q = clamp(rint(b / s) + z, 0, 15)
  gemm_w4     c = act(alpha x @ ((q - z) s) + bias)
  experts     h = act(x[t] @ up[e] + bias_up[e]), or with a gate
              h = act(x[t] @ gate[e] + bias_gate[e]) * (x[t] @ up[e] + bias_up[e]);
              out[t] = sum_j w[t, j] (h @ down[e] + bias_down[e]), e = ids[t, j],
              over the choices that name an expert
  experts_w4  the same with up, gate and down in 4 bits
"""
import math

import torch

own = False

DEV = "cuda"


# ---- the cases ------------------------------------------------------------------

def listed():
    return [
        # a checkpoint's up-projection brought into 4 bits and looked at
        dict(name="round_trip_4096x11008", op="round_trip", K=4096, N=11008, group=128, zeros=False),
        # a small matrix of odd sizes, small groups with a zero point, the last one short
        dict(name="round_trip_999x1001_zeros", op="round_trip", K=999, N=1001, group=32, zeros=True),
        # decode of one sequence through a square projection: the call whose latency counts
        dict(name="w4_decode_1x4096x4096", op="gemm_w4", rows=1, K=4096, N=4096, group=128, zeros=False, bias=False,
             act="none", alpha=1.0),
        # a decode batch of 16 through the up-projection, zero points, bias and GELU
        dict(name="w4_decode_16x11008x4096", op="gemm_w4", rows=16, K=4096, N=11008, group=64, zeros=True, bias=True,
             act="gelu", alpha=1.0),
        # a few drafted tokens, sizes that are no multiple of anything
        dict(name="w4_odd_61x1001x4093", op="gemm_w4", rows=61, K=4093, N=1001, group=32, zeros=True, bias=True,
             act="relu", alpha=0.5),
        # a ragged prompt through the up-projection
        dict(name="w4_prefill_1025x11008x4096", op="gemm_w4", rows=1025, K=4096, N=11008, group=128, zeros=False,
             bias=False, act="none", alpha=1.0),
        # decode of one sequence: one token through two of eight large experts
        dict(name="experts_1x2of8", op="experts", tokens=1, k=2, groups=8, H=4096, F=11008, gated=False, bias=False,
             act="gelu", drop=0.0),
        # a decode batch through many small gated experts, most of them hit
        dict(name="experts_16x8of64_gated", op="experts", tokens=16, k=8, groups=64, H=2048, F=1024, gated=True,
             bias=False, act="silu", drop=0.0),
        # a decode batch with a quarter of the choices over capacity, biases, odd sizes
        dict(name="experts_7x3of10_odd", op="experts", tokens=7, k=3, groups=10, H=1001, F=517, gated=False, bias=True,
             act="relu", drop=0.25),
        # the one-token step with the experts held in 4 bits
        dict(name="experts_w4_1x2of8", op="experts_w4", tokens=1, k=2, groups=8, H=4096, F=11008, gated=False,
             bias=False, act="gelu", drop=0.0, group=128, zeros=False),
        # the batch through small gated experts in 4 bits with zero points
        dict(name="experts_w4_16x8of64_gated", op="experts_w4", tokens=16, k=8, groups=64, H=2048, F=1024, gated=True,
             bias=False, act="silu", drop=0.0, group=64, zeros=True),
        # drafted tokens of 16 sequences, every large expert hit by several
        dict(name="experts_w4_64x2of8", op="experts_w4", tokens=64, k=2, groups=8, H=4096, F=11008, gated=False,
             bias=True, act="gelu", drop=0.05, group=128, zeros=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: a multiple of 64, of 8, or any."""
    w = _log_int(rng, lo, hi)
    return max({0: 64 * (w // 64), 1: 8 * (w // 8), 2: w}[rng.choice((0, 0, 1, 1, 2))], 1)


def draw(rng):
    op = rng.choice(("round_trip", "gemm_w4", "gemm_w4", "gemm_w4", "experts", "experts", "experts_w4", "experts_w4"))
    group, zeros = rng.choice((32, 64, 128, 128, 256)), rng.random() < 0.5
    if op == "round_trip":
        return dict(op=op, K=_width(rng, 64, 8192), N=_width(rng, 64, 5504), group=group, zeros=zeros)
    if op == "gemm_w4":
        K, N = _width(rng, 256, 11008), _width(rng, 256, 11008)
        rows = max(1, min(_log_int(rng, 1, 2048), (1025 * 4096 * 11008) // (K * N)))
        return dict(op=op, rows=rows, K=K, N=N, group=group, zeros=zeros, bias=rng.random() < 0.5,
                    act=rng.choice(("relu", "gelu", "none")), alpha=rng.choice((1.0, 0.5, rng.uniform(-2.0, 2.0))))
    groups, gated = _log_int(rng, 4, 128), rng.random() < 0.5
    H = _width(rng, 256, 4096)
    most = (8 * 4096 * 11008) // (groups * H * (2 if gated else 1))  # of one expert's hidden width
    case = dict(op=op, tokens=_log_int(rng, 1, 64), k=rng.randint(1, min(8, groups)), groups=groups, H=H,
                F=_width(rng, 64, max(65, min(11008, most))), gated=gated, bias=rng.random() < 0.3,
                act=rng.choice(("relu", "gelu", "silu", "none")), drop=rng.choice((0.0, rng.uniform(0.0, 0.3))))
    if op == "experts_w4":
        case.update(group=group, zeros=zeros)
    return case


# ---- inputs -----------------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).half()


def _codes(g, K, N, group, zeros, std):
    """One matrix as a checkpoint holds it: words, scales and zero points (or
    None).  The codes lie around the zero point as those of normal weights."""
    words, G = -(-K // 8), -(-K // group)
    z = torch.randint(5, 11, (G, N), generator=g, device=DEV, dtype=torch.int32) if zeros else None
    at = 8.0 if z is None else z.float().repeat_interleave(group, 0)[:K]
    q = (torch.randn(K, N, generator=g, device=DEV) * 2.5 + at).round_().clamp_(0, 15).to(torch.int32)
    q = torch.nn.functional.pad(q, (0, 0, 0, 8 * words - K)).reshape(words, 8, N)
    w = torch.zeros(words, N, dtype=torch.int32, device=DEV)
    for i in range(8):
        w |= q[:, i] << (4 * i)
    s = ((0.5 + torch.rand(G, N, generator=g, device=DEV)) * (std / 2.5)).half()
    return w, s, None if z is None else z.to(torch.uint8)


def _stack(g, E, K, N, group, zeros, std):
    parts = [_codes(g, K, N, group, zeros, std) for _ in range(E)]
    return tuple(None if parts[0][i] is None else torch.stack([p[i] for p in parts]) for i in range(3)) + (K, group)


def prepare(case, seed):
    if not own:
        return _inputs(case, seed, None)
    import tiled_dense_gemm_scale_amd as gsr

    return _inputs(case, seed, gsr)


def _inputs(case, seed, gsr):
    """The inputs, with the package's handles and workspaces where it is given."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case, "gsr": gsr}
    if op == "round_trip":
        K, N = case["K"], case["N"]
        # columns of uneven size and some off centre, as a trained matrix has
        st["b"] = (torch.randn(K, N, generator=g, device=DEV) * K ** -0.5 * torch.exp(torch.randn(N, generator=g, device=DEV) * 0.5)
                   + torch.randn(N, generator=g, device=DEV) * 0.3 * K ** -0.5).half()
        return st
    if op == "gemm_w4":
        M, K, N = case["rows"], case["K"], case["N"]
        w = _codes(g, K, N, case["group"], case["zeros"], K ** -0.5) + (K, case["group"])
        st.update(x=_normal(g, M, K), w=w, bias=_normal(g, N) if case["bias"] else None)
        if gsr:
            st["w"] = gsr.W4(*w)
            st["workspace"] = gsr.new_workspace(gsr.w4_workspace_bytes(M, N, K))
        return st
    T, k, E, H, F = case["tokens"], case["k"], case["groups"], case["H"], case["F"]
    # a router's choices: distinct experts in order of their score, experts of uneven popularity, the dropped as -1
    scores = torch.randn(T, E, generator=g, device=DEV) + 0.7 * torch.randn(1, E, generator=g, device=DEV)
    top, ids = torch.topk(scores, k, dim=1)
    if case["drop"] > 0.0:
        ids = torch.where(torch.rand(T, k, generator=g, device=DEV) < case["drop"], torch.full_like(ids, -1), ids)
    st.update(x=_normal(g, T, H), ids=ids.contiguous(), weights=torch.softmax(top, dim=1).contiguous())
    names = [("up", H, F), ("gate", H, F), ("down", F, H)]
    for name, rows, cols in names:
        if name == "gate" and not case["gated"]:
            st["gate"] = st["bias_gate"] = None
            continue
        if op == "experts":
            st[name] = torch.stack([_normal(g, rows, cols, std=rows ** -0.5) for _ in range(E)])
        else:
            st[name] = _stack(g, E, rows, cols, case["group"], case["zeros"], rows ** -0.5)
            if gsr:
                st[name] = gsr.W4(*st[name])
        st["bias_" + name] = _normal(g, E, cols, std=0.1) if case["bias"] else None
    if gsr:
        st["workspace"] = gsr.new_workspace(gsr.expert_few_workspace_bytes(T, k, E, F, H))
    else:  # the slots of every expert that is hit, for the plain form's loop
        flat = ids.reshape(-1).tolist()
        st["slots"] = [(e, torch.tensor([i for i, v in enumerate(flat) if v == e], device=DEV))
                       for e in sorted(set(flat)) if e >= 0]
    return st


# ---- one pass ------------------------------------------------------------------------

def _activate(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _values(words, scales, zeros, K, group):
    """The weights that the codes stand for, in 32 bits."""
    q = torch.stack([(words >> (4 * i)) & 15 for i in range(8)], 1).reshape(-1, words.shape[1])[:K].float()
    of = torch.arange(K, device=DEV) // group
    return (q - (8.0 if zeros is None else zeros.float()[of])) * scales.float()[of]


def _quantized(b, group, zeros):
    """codes, scales and zero points of b, as 32-bit floats."""
    K, N = b.shape
    G = -(-K // group)
    v = torch.nn.functional.pad(b.float(), (0, 0, 0, G * group - K)).reshape(G, group, N)
    if zeros:
        lo, hi = v.amin(1).clamp(max=0.0), v.amax(1).clamp(min=0.0)
        s = ((hi - lo) / 15.0).half().float()
        z = torch.where(s > 0, torch.round(-lo / s).clamp(0, 15), torch.full_like(s, 8.0))
        q = (torch.round(v / s[:, None]) + z[:, None]).clamp(0, 15)
    else:
        s = (v.abs().amax(1) / 7.0).half().float()
        z = torch.full_like(s, 8.0)
        q = torch.round(v / s[:, None]).clamp(-8, 7) + 8.0
    q = torch.where(s[:, None] > 0, q, z[:, None].expand_as(q))
    return q, s, z


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "round_trip":
        q, s, z = _quantized(st["b"], case["group"], case["zeros"])
        values = ((q - z[:, None]) * s[:, None]).reshape(-1, case["N"])[:case["K"]].half()
        return (values, s.half()) + ((z.to(torch.uint8),) if case["zeros"] else ())
    if op == "gemm_w4":
        v = case["alpha"] * (st["x"].float() @ _values(*st["w"]))
        if st["bias"] is not None:
            v = v + st["bias"].float()
        return _activate(v, case["act"]).half()
    x, T, k = st["x"].float(), case["tokens"], case["k"]
    out = torch.zeros(T, case["H"], device=DEV)

    def product(a, name, e):
        w = st[name]
        b = w[e].float() if op == "experts" else _values(w[0][e], w[1][e], None if w[2] is None else w[2][e], w[3], w[4])
        return a @ b if st["bias_" + name] is None else a @ b + st["bias_" + name][e].float()

    for e, slots in st["slots"]:
        token = torch.div(slots, k, rounding_mode="floor")
        h = product(x[token], "up", e)
        h = _activate(h, case["act"]) if not case["gated"] else _activate(product(x[token], "gate", e), case["act"]) * h
        y = product(h, "down", e) * st["weights"].reshape(-1)[slots][:, None]
        out[token] += y  # a token names an expert once
    return out.half()


def run(st):
    if not own:
        return _plain(st)
    gsr, case, op = st["gsr"], st["case"], st["case"]["op"]
    if op == "round_trip":
        w = gsr.quantize_w4(st["b"], case["group"], zeros=case["zeros"])
        return (gsr.dequantize_w4(w), w.scales) + ((w.zeros,) if case["zeros"] else ())
    if op == "gemm_w4":
        return gsr.gemm_w4(st["x"], st["w"], st["workspace"], bias=st["bias"], alpha=case["alpha"],
                           activation=case["act"])
    return gsr.expert_mlp_few(st["x"], st["ids"], st["weights"], st["up"], st["down"], st["workspace"], gate=st["gate"],
                              bias_up=st["bias_up"], bias_gate=st["bias_gate"], bias_down=st["bias_down"],
                              activation=case["act"])


# ---- what a pass cannot do without ----------------------------------------------------

def _weight_bytes(case, K, N):
    if case["op"] == "experts":
        return 2 * K * N
    return 4 * -(-K // 8) * N + -(-K // case["group"]) * N * (3 if case["zeros"] else 2)


def work(case):
    op = case["op"]
    if op == "round_trip":
        K, N = case["K"], case["N"]
        return {"bytes": 4 * K * N + 2 * _weight_bytes(case, K, N), "flops": 4 * K * N}
    if op == "gemm_w4":
        M, K, N = case["rows"], case["K"], case["N"]
        return {"bytes": 2 * M * (K + N) + _weight_bytes(case, K, N) + (2 * N if case["bias"] else 0),
                "flops": 2 * M * K * N}
    T, k, E, H, F, ups = case["tokens"], case["k"], case["groups"], case["H"], case["F"], 2 if case["gated"] else 1
    slots = T * k * (1.0 - case["drop"])
    hit = E * (1.0 - (1.0 - k / E) ** (T * (1.0 - case["drop"])))  # experts that a choice names, for choices at random
    per = ups * _weight_bytes(case, H, F) + _weight_bytes(case, F, H) + (2 * (ups * F + H) if case["bias"] else 0)
    return {"bytes": int(hit * per) + 4 * T * H + 12 * T * k, "flops": int(2 * slots * H * F * (ups + 1))}


# ---- the definitions in 64 bits ---------------------------------------------------------

def _act64(v, act):
    if act == "relu":
        return v.clamp(min=0.0)
    if act == "gelu":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def _values64(words, scales, zeros, K, group):
    """Row by row of words: eight rows of weights each."""
    out = torch.empty(8 * words.shape[0], words.shape[1], dtype=torch.float64, device=DEV)
    for i in range(8):
        out[i::8] = torch.bitwise_and(torch.bitwise_right_shift(words, 4 * i), 0xF).double()
    out = out[:K].clone()
    for j in range(scales.shape[0]):
        rows = out[j * group:(j + 1) * group]
        rows -= 8.0 if zeros is None else zeros[j].double()
        rows *= scales[j].double()
    return out


def exact(case, seed):
    st, op = _inputs(case, seed, None), case["op"]
    if op == "round_trip":
        b, group = st["b"].double(), case["group"]
        values, scales, zeros = torch.zeros_like(b), [], []
        for k0 in range(0, case["K"], group):
            v = b[k0:k0 + group]
            zero = torch.zeros_like(v[0])
            if case["zeros"]:
                top, low = torch.maximum(v.max(0).values, zero), torch.minimum(v.min(0).values, zero)
                s = ((top - low) / 15.0).half().double()
                z = (-low / s).round().clamp(0.0, 15.0)
                least, most = -z, 15.0 - z
            else:
                s, z = (torch.maximum(v.max(0).values, -v.min(0).values) / 7.0).half().double(), None
                least, most = zero - 8.0, zero + 7.0
            step = torch.minimum(torch.maximum((v / s).round(), least), most)
            values[k0:k0 + group] = torch.where(s > 0, step * s, zero)
            scales.append(s)
            if z is not None:
                zeros.append(torch.where(s > 0, z, zero + 8.0).to(torch.uint8))
        return (values, torch.stack(scales)) + ((torch.stack(zeros),) if zeros else ())
    if op == "gemm_w4":
        v = torch.matmul(st["x"].double(), _values64(*st["w"])).mul_(case["alpha"])
        if case["bias"]:
            v += st["bias"].double()
        return _act64(v, case["act"])
    ids, x = st["ids"].tolist(), st["x"].double()
    out = torch.zeros(case["tokens"], case["H"], dtype=torch.float64, device=DEV)
    for e in range(case["groups"]):
        hits = [(t, j) for t, row in enumerate(ids) for j, i in enumerate(row) if i == e]
        if not hits:
            continue
        t = torch.tensor([a for a, _ in hits], device=DEV)
        j = torch.tensor([b for _, b in hits], device=DEV)

        def through(a, name):
            w = st[name]
            full = w[e].double() if op == "experts" else _values64(w[0][e], w[1][e], None if w[2] is None else w[2][e],
                                                                   w[3], w[4])
            y = torch.matmul(a, full)
            return y + st["bias_" + name][e].double() if case["bias"] else y

        h = through(x[t], "up")
        if case["gated"]:
            h = h * _act64(through(x[t], "gate"), case["act"])
        else:
            h = _act64(h, case["act"])
        out.index_add_(0, t, through(h, "down") * st["weights"][t, j].double()[:, None])
    return out
