"""The routed-expert and adapter operators as workloads: their inputs, one pass
through each, its plain form in elementary torch operations, and what a pass
cannot do without.

Operators (E experts, T tokens with k choices each, P = T k sorted rows):

  group     slots sorted by expert, stable: offsets[e] counts the slots of the
            experts before e; rows[p] is the token of sorted row p (-1 behind
            the last expert's); positions[t, j] is the sorted row of token t's
            j-th choice (-1 where the choice was dropped)
  gather    out[p] = x[rows[p]], zeros where rows[p] names no token
  combine   out[t] = sum_j w[t, j] y[positions[t, j]] over the kept choices
  combine_backward
            dy[positions[t, j]] = w[t, j] dout[t], zeros in rows that no choice
            names; dw[t, j] = <dout[t], y[positions[t, j]]>
  experts   c[p] = act(alpha x[rows[p]] @ b[e] + bias[e]) for the rows of every
            expert e; rows behind the last expert's stay as they were
  adapters  c[m] = act(alpha (x[m] @ b + s[l] (x[m] @ la[l]^T) @ lb[l]^T) + bias)
            with l = ids[m]; rows whose id names no adapter take x[m] @ b alone
"""
import math

import torch

own = False

DEV = "cuda"


# ---- the cases ------------------------------------------------------------------

def listed():
    return [
        # one decode step of 32 sequences, two of eight experts each: the call whose latency counts
        dict(name="group_decode_32x2", op="group", tokens=32, k=2, groups=8, drop=0.0, wide=False),
        # a long prompt batch, eight of 64 experts, one choice in twenty over its expert's capacity;
        # 64-bit ids as a top-k gives them
        dict(name="group_prefill_16384x8", op="group", tokens=16384, k=8, groups=64, drop=0.05, wide=True),
        # a ragged prompt's hidden states copied in expert order
        dict(name="gather_2049x2x4096", op="gather", tokens=2049, k=2, groups=8, drop=0.02, width=4096),
        # a width whose rows start on odd elements
        dict(name="gather_777x3x1001", op="gather", tokens=777, k=3, groups=16, drop=0.0, width=1001),
        # a decode batch's expert outputs summed back
        dict(name="combine_decode_16x8x4096", op="combine", tokens=16, k=8, groups=64, drop=0.0, width=4096),
        # a training batch's gradient through the weighted sum
        dict(name="combine_backward_8192x2x4096", op="combine_backward", tokens=8192, k=2, groups=8, drop=0.05,
             width=4096),
        # decode: 16 tokens through two of eight experts' up-projections, every expert's weights read once
        dict(name="experts_up_decode_16x2", op="experts", tokens=16, k=2, groups=8, drop=0.0, K=4096, N=11008,
             gather=True, bias=True, act="gelu", alpha=1.0),
        # a ragged prompt through the experts' down-projections, rows already in expert order
        dict(name="experts_down_1025x2", op="experts", tokens=1025, k=2, groups=8, drop=0.03, K=11008, N=4096,
             gather=False, bias=False, act="none", alpha=1.0),
        # a prompt batch through the experts' up-projections (the largest case)
        dict(name="experts_up_prefill_8192x2", op="experts", tokens=8192, k=2, groups=8, drop=0.0, K=4096, N=11008,
             gather=True, bias=False, act="relu", alpha=1.0),
        # decode: one request against the down-projection with its own adapter
        dict(name="adapters_decode_1x4096x11008", op="adapters", rows=1, N=4096, K=11008, adapters=8, rank=64,
             requests=1, bare=0.0, bias=False, act="none", alpha=1.0),
        # decode: 16 requests, 16 adapters of 32 in memory
        dict(name="adapters_decode_16x11008x4096", op="adapters", rows=16, N=11008, K=4096, adapters=32, rank=16,
             requests=16, bare=0.1, bias=True, act="gelu", alpha=1.0),
        # prompts of nine requests, some without an adapter, in one batch of a ragged length
        dict(name="adapters_prefill_4097x11008x4096", op="adapters", rows=4097, N=11008, K=4096, adapters=8, rank=16,
             requests=9, bare=0.2, bias=True, act="gelu", alpha=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: a multiple of 64, of 8, or any."""
    w = _log_int(rng, lo, hi)
    return max({0: 64 * (w // 64), 1: 8 * (w // 8), 2: w}[rng.choice((0, 0, 1, 1, 2))], 1)


def draw(rng):
    op = rng.choice(("group", "gather", "combine", "combine_backward", "experts", "experts", "adapters", "adapters"))
    drop = rng.choice((0.0, rng.uniform(0.0, 0.2)))
    act = rng.choice(("relu", "gelu", "none"))
    alpha = rng.choice((1.0, 0.5, rng.uniform(-2.0, 2.0)))
    if op == "group":
        groups = _log_int(rng, 4, 512)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), k=rng.randint(1, min(8, groups)), groups=groups, drop=drop,
                    wide=rng.random() < 0.5)
    if op in ("gather", "combine", "combine_backward"):
        width, groups = _width(rng, 64, 8192), _log_int(rng, 4, 128)
        k = rng.randint(1, min(8, groups))
        tokens = _log_int(rng, 1, max(1, (1 << 26) // (width * k)))
        return dict(op=op, tokens=tokens, k=k, groups=groups, drop=drop, width=width)
    if op == "experts":
        groups = _log_int(rng, 4, 64)
        big = (8 * 4096 * 11008) // groups  # K N of one expert at most
        K = _width(rng, 256, 11008)
        N = _width(rng, 256, max(257, min(11008, big // K)))
        k = rng.randint(1, 4)
        tokens = _log_int(rng, 1, 8192)
        tokens = max(1, min(tokens, (16384 * 4096 * 11008) // (k * K * N)))
        return dict(op=op, tokens=tokens, k=k, groups=groups, drop=drop, K=K, N=N, gather=rng.random() < 0.5,
                    bias=rng.random() < 0.5, act=act, alpha=alpha)
    K, N = _width(rng, 256, 11008), _width(rng, 256, 11008)
    rows = max(1, min(_log_int(rng, 1, 8192), (4097 * 4096 * 11008) // (K * N)))
    return dict(op="adapters", rows=rows, N=N, K=K, adapters=_log_int(rng, 1, 64),
                rank=rng.choice((4, 8, 16, 16, 32, 64, 128, rng.randint(1, 128))),
                requests=_log_int(rng, 1, min(rows, 64)), bare=rng.choice((0.0, rng.uniform(0.0, 0.5))),
                bias=rng.random() < 0.5, act=act, alpha=alpha)


# ---- inputs -----------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).half()


def _routing(case, g):
    """A router's choices: ids (T, k) of distinct experts in order of their
    score, with experts of uneven popularity and dropped choices as -1, and the
    weights (the scores' softmax over the choices)."""
    T, k, E = case["tokens"], case["k"], case["groups"]
    scores = torch.randn(T, E, generator=g, device=DEV) + 0.7 * torch.randn(1, E, generator=g, device=DEV)
    top, ids = torch.topk(scores, k, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    if case["drop"] > 0.0:
        lost = torch.rand(T, k, generator=g, device=DEV) < case["drop"]
        ids = torch.where(lost, torch.full_like(ids, -1), ids)
    return ids.contiguous(), weights


def _plan(ids, groups):
    """offsets, rows and positions of the definition (inputs of the operators
    behind `group`, made once here)."""
    k = ids.shape[1]
    key = torch.where((ids >= 0) & (ids < groups), ids.long(), torch.full_like(ids.long(), groups)).reshape(-1)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=groups + 1)
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts[:groups].cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=DEV)
    kept = key < groups
    positions = torch.where(kept, place, torch.full_like(place, -1)).reshape(ids.shape)
    rows = torch.where(kept[order], order // k, torch.full_like(order, -1))
    return offsets.int(), rows.int(), positions.int()


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = {"case": case}
    if own:
        import tiled_dense_gemm_scale_amd as gsr

        st["gsr"] = gsr
    if op == "adapters":
        M, N, K, L, R = case["rows"], case["N"], case["K"], case["adapters"], case["rank"]
        # the batch is requests of uneven lengths, one behind the other, each with one adapter or none
        cuts = torch.rand(case["requests"] - 1, generator=g, device=DEV)
        bounds = (torch.sort(cuts).values * M).long()
        request = torch.searchsorted(bounds, torch.arange(M, device=DEV), right=True)
        if case["requests"] == M:
            request = torch.arange(M, device=DEV)
        of_request = torch.randperm(max(L, case["requests"]), generator=g, device=DEV)[: case["requests"]] % L
        bare = torch.rand(case["requests"], generator=g, device=DEV) < case["bare"]
        of_request = torch.where(bare, torch.full_like(of_request, -1), of_request)
        st.update(a=_normal(g, M, K), b=_normal(g, K, N, std=K ** -0.5),
                  la=_normal(g, L, R, K, std=K ** -0.5), lb=_normal(g, L, N, R, std=0.5 * R ** -0.5),
                  ids=of_request[request].int().contiguous(),
                  scales=0.5 + 1.5 * torch.rand(L, generator=g, device=DEV),
                  bias=_normal(g, N) if case["bias"] else None)
        if own:
            st["workspace"] = gsr.new_workspace(gsr.adapter_workspace_bytes(M, N, K, R))
        return st
    ids, weights = _routing(case, g)
    if op == "group":
        st["ids"] = ids if case["wide"] else ids.int()
        if own:
            st["workspace"] = gsr.new_workspace(gsr.group_workspace_bytes(ids.numel(), case["groups"]))
        return st
    offsets, rows, positions = _plan(ids, case["groups"])
    P = rows.numel()
    if op == "gather":
        st.update(x=_normal(g, case["tokens"], case["width"]), rows=rows)
    elif op == "combine":
        st.update(y=_normal(g, P, case["width"]), positions=positions, weights=weights)
    elif op == "combine_backward":
        st.update(dout=_normal(g, case["tokens"], case["width"]), y=_normal(g, P, case["width"]),
                  positions=positions, weights=weights, rows=rows)
    else:
        K, N, E = case["K"], case["N"], case["groups"]
        st.update(x=_normal(g, case["tokens"] if case["gather"] else P, K),
                  b=torch.stack([_normal(g, K, N, std=K ** -0.5) for _ in range(E)]),
                  bias=_normal(g, E, N) if case["bias"] else None,
                  offsets=offsets, rows=rows if case["gather"] else None,
                  c=torch.zeros(P, N, dtype=torch.float16, device=DEV),
                  bounds=[int(v) for v in offsets.tolist()])  # the plain form's loop bounds, on the host
    return st


# ---- one pass ------------------------------------------------------------------------

def _activate(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "group":
        return _plan(st["ids"], case["groups"])
    if op == "gather":
        keep = (st["rows"] >= 0)[:, None]
        return torch.where(keep, st["x"][st["rows"].clamp(min=0).long()], torch.zeros((), dtype=torch.float16,
                                                                                      device=DEV))
    if op == "combine":
        pos = st["positions"]
        y = st["y"][pos.clamp(min=0).long()].float()
        y = torch.where((pos >= 0)[..., None], y, torch.zeros((), device=DEV))
        return (st["weights"][..., None] * y).sum(1).half()
    if op == "combine_backward":
        pos, w, dout = st["positions"], st["weights"], st["dout"].float()
        keep = pos >= 0
        y = st["y"][pos.clamp(min=0).long()].float()
        dw = torch.where(keep, (dout[:, None, :] * y).sum(2), torch.zeros((), device=DEV))
        P = st["rows"].numel()
        dy = torch.zeros(P + 1, dout.shape[1], dtype=torch.float16, device=DEV)  # the last row takes the dropped
        to = torch.where(keep, pos.long(), torch.full_like(pos.long(), P)).reshape(-1)
        dy[to] = (w[..., None] * dout[:, None, :]).half().reshape(-1, dout.shape[1])
        return dy[:P], dw
    if op == "experts":
        c, alpha = st["c"], case["alpha"]
        for e in range(case["groups"]):
            lo, hi = st["bounds"][e], st["bounds"][e + 1]
            if lo == hi:
                continue
            x = st["x"][lo:hi] if st["rows"] is None else st["x"][st["rows"][lo:hi].long()]
            v = alpha * (x.float() @ st["b"][e].float())
            if st["bias"] is not None:
                v = v + st["bias"][e].float()
            c[lo:hi] = _activate(v, case["act"]).half()
        return c
    x, L, R = st["a"].float(), case["adapters"], case["rank"]
    v = x @ st["b"].float()
    # every row against every adapter, kept where the adapter is the row's
    t = (x @ st["la"].float().reshape(L * R, -1).t()).reshape(-1, L, R)
    mine = st["ids"][:, None] == torch.arange(L, device=DEV)[None, :]
    t = torch.where(mine[..., None], t * st["scales"][None, :, None], torch.zeros((), device=DEV))
    v = v + t.reshape(-1, L * R) @ st["lb"].float().transpose(1, 2).reshape(L * R, -1)
    v = case["alpha"] * v
    if st["bias"] is not None:
        v = v + st["bias"].float()
    return _activate(v, case["act"]).half()


def run(st):
    if not own:
        return _plain(st)
    gsr, case, op = st["gsr"], st["case"], st["case"]["op"]
    if op == "group":
        return gsr.group_rows(st["ids"], case["groups"], workspace=st["workspace"])
    if op == "gather":
        return gsr.gather_rows(st["x"], st["rows"])
    if op == "combine":
        return gsr.combine_rows(st["y"], st["positions"], st["weights"])
    if op == "combine_backward":
        return gsr.combine_rows_backward(st["dout"], st["y"], st["positions"], st["weights"], st["rows"])
    if op == "experts":
        return gsr.gemm_grouped(st["x"], st["b"], st["offsets"], rows=st["rows"], bias=st["bias"],
                                alpha=case["alpha"], activation=case["act"], c=st["c"])
    return gsr.gemm_adapters(st["a"], st["b"], st["la"], st["lb"], st["ids"], st["workspace"], scales=st["scales"],
                             bias=st["bias"], alpha=case["alpha"], activation=case["act"])


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "adapters":
        M, N, K, R = case["rows"], case["N"], case["K"], case["rank"]
        used = min(case["adapters"], case["requests"])
        by = 2 * (M * K + K * N + M * N) + 2 * used * R * (K + N) + 4 * M + 4 * used + (2 * N if case["bias"] else 0)
        return {"bytes": by, "flops": 2 * M * N * K + 2 * M * R * (K + N)}
    T, k, E = case["tokens"], case["k"], case["groups"]
    P = T * k
    if op == "group":
        return {"bytes": P * ((8 if case["wide"] else 4) + 4 + 4) + 4 * (E + 1), "flops": 0}
    if op == "experts":
        K, N = case["K"], case["N"]
        # experts that at least one choice names, at most
        by = 2 * ((T if case["gather"] else P) * K + min(E, P) * K * N + P * N) + 4 * (E + 1)
        by += (4 * P if case["gather"] else 0) + (2 * min(E, P) * N if case["bias"] else 0)
        return {"bytes": by, "flops": 2 * P * K * N}
    H = case["width"]
    if op == "gather":
        return {"bytes": 2 * T * H + 2 * P * H + 4 * P, "flops": 0}
    if op == "combine":
        return {"bytes": 2 * P * H + 2 * T * H + 8 * P, "flops": 2 * P * H}
    return {"bytes": 2 * T * H + 4 * P * H + 16 * P, "flops": 3 * P * H}


# ---- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "group":
        # expert by expert: its slots in their order, on the host
        ids, E, k = st["ids"].cpu().reshape(-1), case["groups"], case["k"]
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        rows, positions = (torch.full((ids.numel(),), -1, dtype=torch.int32) for _ in range(2))
        at = 0
        for e in range(E):
            slots = torch.nonzero(ids == e).flatten()
            rows[at:at + slots.numel()] = torch.div(slots, k, rounding_mode="floor").int()
            positions[slots] = torch.arange(at, at + slots.numel(), dtype=torch.int32)
            at += slots.numel()
            offsets[e + 1] = at
        return offsets.to(DEV), rows.to(DEV), positions.reshape(st["ids"].shape).to(DEV)
    if op == "gather":
        out = torch.zeros(st["rows"].numel(), case["width"], dtype=torch.float64, device=DEV)
        p = torch.nonzero(st["rows"] >= 0).flatten()
        out[p] = st["x"][st["rows"][p].long()].double()
        return out
    if op == "combine":
        out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device=DEV)
        for j in range(case["k"]):
            p = st["positions"][:, j].long()
            t = torch.nonzero(p >= 0).flatten()
            out[t] += st["weights"][t, j].double()[:, None] * st["y"][p[t]].double()
        return out
    if op == "combine_backward":
        dy = torch.zeros(st["rows"].numel(), case["width"], dtype=torch.float64, device=DEV)
        dw = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device=DEV)
        for j in range(case["k"]):
            p = st["positions"][:, j].long()
            t = torch.nonzero(p >= 0).flatten()
            up = st["dout"][t].double()
            dy[p[t]] = st["weights"][t, j].double()[:, None] * up
            dw[t, j] = (up * st["y"][p[t]].double()).sum(1)
        return dy, dw

    def act(v):
        if case["act"] == "relu":
            return v.clamp(min=0.0)
        if case["act"] == "gelu":
            u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
            return v * torch.sigmoid(2.0 * u)
        return v

    if op == "experts":
        out = torch.zeros(st["c"].shape, dtype=torch.float64, device=DEV)
        ends = st["offsets"].tolist()
        for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
            if hi > lo:
                x = st["x"][st["rows"][lo:hi].long()] if case["gather"] else st["x"][lo:hi]
                v = torch.matmul(x.double(), st["b"][e].double()).mul_(case["alpha"])
                if case["bias"]:
                    v += st["bias"][e].double()
                out[lo:hi] = act(v)
        return out
    v = torch.matmul(st["a"].double(), st["b"].double())
    for l in range(case["adapters"]):
        m = torch.nonzero(st["ids"] == l).flatten()
        if m.numel():
            low = torch.matmul(st["a"][m].double(), st["la"][l].double().t().contiguous())
            v[m] += torch.matmul(low, st["lb"][l].double().t().contiguous()) * st["scales"][l].double()
    v *= case["alpha"]
    if case["bias"]:
        v += st["bias"].double()
    return act(v)
