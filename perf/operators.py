"""The mixture-of-experts operators around the fused dispatch and combine, as cases to measure.

Four operators, each with its plain form (elementary torch operations) and the library's call:

  route    router logits -> experts and weights of every token (softmax or sigmoid scores, a balance
           bias that takes part in the choice only, expert groups, top-k, renormalised weights), and
           the gradient of the logits;
  slots    router choices -> the row of the receive windows that each (token, choice) pair has, and
           the pair that each row belongs to;
  combine  the experts' rows -> the tokens' weighted sums, and the gradients of rows and weights;
  w4       products of a few token rows with their experts' 4-bit weights (the decode form of the
           experts' GEMM).

`own` selects the side that prepare() and run() take: False, the plain form; True, the library's kernels.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # four tokens of a decode step choose 2 of 32 experts: latency only
        dict(name="route_decode", op="route", T=4, E=32, topk=2, groups=1, take=1, group_top=1, score="softmax",
             renorm=True, scale=1.0, dt="f32", bias=False, masked=0.0, ld=32, counts=False),
        # 8 ranks x 4096 tokens of a training step: sigmoid scores with a balance bias, 4 of 8 groups, top-8 of 256
        dict(name="route_train", op="route", T=32768, E=256, topk=8, groups=8, take=4, group_top=2, score="sigmoid",
             renorm=True, scale=2.5, dt="f32", bias=True, masked=0.0, ld=256, counts=True),
        # a ragged prompt: an odd expert count in a wider logits row, experts that are switched off for some tokens
        dict(name="route_ragged", op="route", T=4097, E=60, topk=4, groups=1, take=1, group_top=1, score="softmax",
             renorm=False, scale=1.0, dt="bf16", bias=False, masked=0.3, ld=64, counts=True),
        # the router's backward pass of a training step, where every logit has a gradient
        dict(name="route_bwd_train", op="route_bwd", T=32768, E=128, topk=8, score="softmax", renorm=False, scale=1.0,
             dt="bf16", masked=0.0),
        # one rank's 4096 tokens, top-2 over 8 ranks of 4 experts: the rows of the combine's receive windows
        dict(name="slots_rank", op="slots", T=4096, topk=2, bins=8, per_bin=4, cap=2048, none=0.0),
        # a long batch over 16 ranks of 16 experts, a tenth of the pairs dropped by the router
        dict(name="slots_long", op="slots", T=65536, topk=8, bins=16, per_bin=16, cap=40960, none=0.1),
        # a decode step's weighted sum of the experts' rows, in pair order
        dict(name="combine_decode", op="combine", T=4, topk=2, N=4096, bins=0, cap=0, none=0.0, dt="bf16", out="bf16",
             add=False),
        # one rank's 4096 tokens from 8 receive windows of 2048 rows, with the residual stream added
        dict(name="combine_windows", op="combine", T=4096, topk=2, N=4096, bins=8, cap=2048, none=0.0, dt="bf16",
             out="bf16", add=True),
        # the combine's backward pass at an odd token count and width, windows a quarter larger than their rows
        dict(name="combine_bwd_train", op="combine_bwd", T=8191, topk=8, N=2056, bins=8, cap=10240, none=0.02,
             dt="bf16", out="bf16"),
        # one token's eight experts of 64, up projection 4096 -> 1792
        dict(name="w4_token", op="w4", T=1, topk=8, E=64, K=4096, N=1792, group=128, zeros=False, out="bf16", up=True),
        # sixteen tokens, top-2 of 32 experts, down projection 1792 -> 4096 with zero points
        dict(name="w4_batch", op="w4", T=16, topk=2, E=32, K=1792, N=4096, group=64, zeros=True, out="f32", up=False),
        # one dense matrix with a few rows at sizes that end inside the weight tiles
        dict(name="w4_ragged", op="w4", T=5, topk=1, E=1, K=1048, N=8200, group=32, zeros=True, out="bf16", up=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "slots", "combine", "combine_bwd", "w4", "w4"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(2, 256 // groups)
        E = max(E, 8)
        T = _log(rng, 1, 32768)
        c = dict(op=op, T=T, E=E, topk=rng.randint(1, min(8, E // groups)), score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), dt=rng.choice(["f32", "bf16"]),
                 masked=rng.choice([0.0, 0.0, 0.2]))
        if op == "route":
            c.update(groups=groups, take=rng.randint(1, groups), group_top=rng.choice([1, 2]) if groups > 1 else 1,
                     bias=rng.random() < 0.5, ld=E + rng.choice([0, 0, 3]), counts=rng.random() < 0.5)
        return c
    if op == "slots":
        T, topk, bins = _log(rng, 1, 65536), rng.randint(1, 8), rng.randint(1, 16)
        return dict(op=op, T=T, topk=topk, bins=bins, per_bin=rng.randint(1, 16), none=rng.choice([0.0, 0.1]),
                    cap=T * topk // bins + T * topk // 2 // bins + rng.randint(16, 64))
    if op in ("combine", "combine_bwd"):
        topk, N = rng.randint(1, 8), 8 * _log(rng, 16, 512)
        T = _log(rng, 1, min(8192, 150_000_000 // (topk * N)))
        bins = rng.choice([0, 1, 8])
        c = dict(op=op, T=T, topk=topk, N=N, bins=bins, cap=T * topk // bins + T // 4 + 32 if bins else 0,
                 none=0.02 if bins else 0.0, dt=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
        if op == "combine":
            c["add"] = rng.random() < 0.5
        return c
    E = rng.choice([1, 1, 8, 32])
    T, topk = (_log(rng, 1, 64), 1) if E == 1 else (_log(rng, 1, 16), rng.choice([1, 2, 4]))
    K = 8 * _log(rng, 16, 512)
    N = 8 * _log(rng, 16, min(512, 30_000_000 // (T * topk * K) if E > 1 else 512))
    return dict(op="w4", T=T, topk=topk, E=E, K=K, N=N,
                group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]),
                up=rng.random() < 0.5)


# --------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _logits(c, g):
    T, E, ld = c["T"], c["E"], c.get("ld", c["E"])
    skew = 0.5 * torch.randn(E, generator=g, device="cuda")       # some experts are liked more than others
    x = torch.full((T, ld), float("nan"), device="cuda")          # what stands beside the logits is not theirs
    x[:, :E] = torch.randn(T, E, generator=g, device="cuda") + skew
    if c["masked"]:
        x[:, :E].masked_fill_(torch.rand(T, E, generator=g, device="cuda") < c["masked"], float("-inf"))
        x[:1, :E] = float("-inf")                                 # a token with every expert switched off
    return x.to(DT[c["dt"]])


def _choices(T, topk, E, g, none=0.0):
    """Distinct random experts for every token (int32 [T][topk]), some of them -1."""
    e = torch.rand(T, E, generator=g, device="cuda").topk(topk, dim=1).indices.to(torch.int32)
    if none:
        e.masked_fill_(torch.rand(T, topk, generator=g, device="cuda") < none, -1)
    return e


def _plain_slots(experts, bins, per_bin, cap):
    """index [T][topk] int32, pair [bins * cap] int32, counts [bins] int64 of the router choices."""
    T, topk = experts.shape
    e = experts.reshape(-1).long()
    ok = (e >= 0) & (e < bins * per_bin)
    b = torch.where(ok, e // per_bin, bins)
    onehot = (torch.arange(bins, device=e.device)[:, None] == b).int()
    pos = (onehot.cumsum(1) * onehot).sum(0) - 1                  # earlier pairs of the same bin
    keep = ok & (pos < cap)
    index = torch.where(keep, b * cap + pos, -1)
    pair = torch.full((bins * cap + 1,), -1, dtype=torch.int64, device=e.device)
    pair[torch.where(keep, index, bins * cap)] = torch.arange(e.numel(), device=e.device)
    return index.to(torch.int32).view(T, topk), pair[:-1].to(torch.int32), onehot.sum(1)


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    s = {"case": c}
    if op == "route":
        s["logits"] = _logits(c, g)[:, :c["E"]]                   # a view: its rows are ld apart
        # biases are moved in small fixed steps by the balancing that keeps them
        s["bias"] = 0.001 * torch.randint(-40, 41, (c["E"],), generator=g, device="cuda").float() if c["bias"] else None
    elif op == "route_bwd":
        s["logits"] = _logits(c, g)
        top = s["logits"].float().topk(c["topk"], dim=1)
        s["experts"] = torch.where(top.values > float("-inf"), top.indices, -1).to(torch.int32).contiguous()
        s["dweights"] = torch.randn(c["T"], c["topk"], generator=g, device="cuda")
    elif op == "slots":
        s["experts"] = _choices(c["T"], c["topk"], max(c["bins"] * c["per_bin"], c["topk"]), g, c["none"])
    elif op in ("combine", "combine_bwd"):
        T, topk, N = c["T"], c["topk"], c["N"]
        if c["bins"]:
            # four experts a window; what does not fit in them stays with other ranks
            e = _choices(T, topk, max(4 * c["bins"], topk), g, c["none"])
            s["index"], s["pair"], _ = _plain_slots(e, c["bins"], 4, c["cap"])
            R = c["bins"] * c["cap"]
        else:
            s["index"], s["pair"], R = None, None, T * topk
        s["rows"] = torch.randn(R, N, generator=g, device="cuda").to(DT[c["dt"]])
        w = torch.rand(T, topk, generator=g, device="cuda") + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        if op == "combine":
            s["add"] = torch.randn(T, N, generator=g, device="cuda").to(DT[c["out"]]) if c["add"] else None
        else:
            s["dout"] = torch.randn(T, N, generator=g, device="cuda").to(DT[c["out"]])
    else:
        T, topk, E, K, N = c["T"], c["topk"], c["E"], c["K"], c["N"]
        nb, kb, ng = -(-N // 16), -(-K // 128), -(-K // c["group"])
        s["x"] = torch.randn(T if c["up"] else T * topk, K, generator=g, device="cuda").to(torch.bfloat16)
        s["experts"] = _choices(T, topk, E, g).reshape(-1).contiguous() if E > 1 else None
        # uniform codes: every bit of the packed words is random
        s["wq"] = torch.randint(-2 ** 31, 2 ** 31, (E, nb, kb, 64, 4), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        s["scales"] = (0.01 * (0.5 + torch.rand(E, nb, ng, 16, generator=g, device="cuda"))).to(torch.bfloat16)
        s["zeros"] = torch.randint(4, 12, (E, nb, ng, 16), generator=g, device="cuda").to(torch.bfloat16) if c["zeros"] else None
    if own:
        s["call"] = _handle(s)
    return s


# ---------------------------------------------------------------------------------- the library's side

def _handle(s):
    """What a user's program keeps for its calls: output buffers, workspace and arguments."""
    from computation_collective_amd import buffers as bf
    from computation_collective_amd import hocf

    c = s["case"]
    op = c["op"]
    if op in ("route", "route_bwd"):
        how = dict(score=hocf.HOCF_SCORE_SOFTMAX if c["score"] == "softmax" else hocf.HOCF_SCORE_SIGMOID,
                   renorm=c["renorm"], scale=c["scale"])
        if op == "route":
            return bf.MoeRoute(c["T"], c["E"], c["topk"], s["logits"], bias=s["bias"], n_group=c["groups"],
                               topk_group=c["take"], group_top=c["group_top"], counts=c["counts"], **how)
        return bf.MoeRouteBwd(c["T"], c["E"], c["topk"], s["logits"], s["experts"], s["dweights"], **how)
    if op == "slots":
        return bf.MoeSlots(c["T"], c["topk"], c["bins"], c["per_bin"], c["cap"], s["experts"])
    dt = {"f32": hocf.HOCF_F32, "bf16": hocf.HOCF_BF16}
    if op == "combine":
        return bf.MoeCombine(c["T"], c["topk"], c["N"], s["rows"], s["weights"], index=s["index"], add=s["add"],
                             out_dt=dt[c["out"]])
    if op == "combine_bwd":
        return bf.MoeCombineBwd(c["T"], c["topk"], c["N"], s["rows"], s["weights"], s["dout"], index=s["index"],
                                pair=s["pair"])
    return bf.GemvW4(c["T"] * c["topk"], c["topk"] if c["up"] else 1, c["E"], 0, c["N"], c["K"], c["group"], s["x"],
                     s["experts"], s["wq"], s["scales"], s["zeros"], out_dt=dt[c["out"]])


def _bf16(t):
    return t.view(torch.bfloat16) if t.dtype == torch.int16 else t


def _run_own(s):
    op, h = s["case"]["op"], s["call"]
    h.run()
    if op == "route":
        out = {"experts": h.experts, "weights": h.weights}
        if s["case"]["counts"]:
            out["counts"] = h.counts
        return out
    if op == "route_bwd":
        return {"dlogits": _bf16(h.dlogits)}
    if op == "slots":
        return {"index": h.index, "pair": h.pair, "counts": h.counts}
    if op == "combine_bwd":
        return {"drows": _bf16(h.drows), "dweights": h.dweights}
    return {"out": _bf16(h.out)}


# ---------------------------------------------------------------------------------- the plain forms

def _scores(x, score):
    """(scores, selectable) of the logits in 64 bits: -inf and NaN logits are switched off."""
    x = x.double()
    live = x > float("-inf")
    x = torch.where(live, x, float("-inf"))
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x)), live
    top = x.amax(1, keepdim=True)
    p = torch.where(live, torch.exp(x - top), 0.0)
    return p / p.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float64).tiny), live


def _best(v, k):
    """Indices of the k largest of each row, ties to the lowest index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :k]


def _plain_route(s):
    c = s["case"]
    T, E, topk = c["T"], c["E"], c["topk"]
    score, live = _scores(s["logits"], c["score"])                # 64 bits: the choice goes by borders
    value = score if s["bias"] is None else score + s["bias"].double()
    value = torch.where(live, value, float("-inf"))
    if c["groups"] > 1:
        v = value.view(T, c["groups"], -1)
        best = torch.sort(v, dim=2, descending=True).values[:, :, :c["group_top"]]
        any_live = best[:, :, 0] > float("-inf")
        of = torch.where(best > float("-inf"), best, 0.0).sum(2)
        of = torch.where(any_live, of, float("-inf"))
        kept = torch.zeros(T, c["groups"], dtype=torch.bool, device=v.device)
        kept.scatter_(1, _best(of, c["take"]), True)
        value = torch.where(kept[:, :, None], v, float("-inf")).view(T, E)
    at = _best(value, topk)
    chosen = value.gather(1, at) > float("-inf")
    w = torch.where(chosen, score.gather(1, at), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float64).tiny)
    out = {"experts": torch.where(chosen, at, -1).to(torch.int32), "weights": (w * c["scale"]).float()}
    if c["counts"]:
        out["counts"] = ((at[:, :, None] == torch.arange(E, device=at.device)) & chosen[:, :, None]).sum((0, 1)).to(torch.int32)
    return out


def _plain_route_bwd(s):
    c = s["case"]
    score, live = _scores(s["logits"], c["score"])
    e = s["experts"].long()
    has = (e >= 0).double()
    at = e.clamp_min(0)
    sc = score.gather(1, at) * has
    dw = s["dweights"].double() * has * c["scale"]
    if c["renorm"]:                                               # w_j = scale * s_j / sum of the chosen s
        total = sc.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float64).tiny)
        ds = (dw - (dw * sc).sum(1, keepdim=True) / total) / total * has
    else:
        ds = dw
    dscore = torch.zeros_like(score).scatter_add_(1, at, ds)
    if c["score"] == "sigmoid":
        d = dscore * score * (1 - score)
    else:
        d = score * (dscore - (dscore * score).sum(1, keepdim=True))
    return {"dlogits": torch.where(live, d, 0.0).to(s["logits"].dtype)}


def _plain_combine(s):
    c = s["case"]
    T, topk, N = c["T"], c["topk"], c["N"]
    w = s["weights"]
    if s["index"] is None:
        rows = s["rows"].float().view(T, topk, N)
    else:
        at = s["index"].long()
        rows = torch.where((at >= 0)[:, :, None], s["rows"][at.clamp_min(0)].float(), 0.0)
    out = (w[:, :, None] * rows).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    return {"out": out.to(DT[c["out"]])}


def _plain_combine_bwd(s):
    c = s["case"]
    T, topk, N = c["T"], c["topk"], c["N"]
    d = s["dout"].float()
    if s["index"] is None:
        rows = s["rows"].float().view(T, topk, N)
        drows = (s["weights"][:, :, None] * d[:, None, :]).view(T * topk, N)
    else:
        at = s["index"].long()
        rows = torch.where((at >= 0)[:, :, None], s["rows"][at.clamp_min(0)].float(), 0.0)
        p = s["pair"].long()
        has = p >= 0
        p = p.clamp_min(0)
        drows = torch.where(has[:, None], s["weights"].view(-1)[p][:, None] * d[p // topk], 0.0)
    return {"drows": drows.to(s["rows"].dtype), "dweights": (rows * d[:, None, :]).sum(2)}


def _codes(wq):
    """4-bit codes [..][K padded][N padded] of the packed words [..][column block][row block][64][4].

    A block is 16 columns x 128 rows; piece q * 16 + n of its 64 holds column n's rows 32 t + 8 q + i in
    word t, row i in four bits from bit 3 + 16 (i mod 2) + 4 (i div 2), modulo 32."""
    R, nb, kb = wq.shape[:3]
    i = torch.arange(8, device=wq.device, dtype=torch.int32)
    w = ((wq >> 3) & 0x1FFFFFFF) | (wq << 29)                     # turned back by the three bits
    q = ((w.view(R, nb, kb, 4, 16, 4)[..., None] >> (16 * (i % 2) + 4 * (i // 2))) & 15).to(torch.uint8)
    return q.permute(0, 2, 5, 3, 6, 1, 4).reshape(R, kb * 128, nb * 16)


def _plain_w4(s):
    c = s["case"]
    K, N, group = c["K"], c["N"], c["group"]
    e = s["experts"].long() if s["experts"] is not None else torch.zeros(1, dtype=torch.long, device="cuda")
    q = _codes(s["wq"][e])[:, :K, :N].float()
    of = torch.arange(K, device=q.device) // group

    def spread(t):                                                # [R][nb][groups][16] -> [R][K][N]
        t = t[e].float().transpose(1, 2)
        return t.reshape(t.shape[0], t.shape[1], -1)[:, of, :N]

    w = (q - (8.0 if s["zeros"] is None else spread(s["zeros"]))) * spread(s["scales"])
    x = s["x"].float()
    if s["experts"] is None:
        out = x @ w[0]
        out = out if not c["up"] else out.repeat_interleave(c["topk"], 0)
    else:
        x = x.repeat_interleave(c["topk"], 0) if c["up"] else x
        out = torch.bmm(x[:, None, :], w.contiguous())[:, 0]
    return {"out": out.to(DT[c["out"]])}


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["case"]["op"]
    if op == "route":
        return _plain_route(s)
    if op == "route_bwd":
        return _plain_route_bwd(s)
    if op == "slots":
        c = s["case"]
        index, pair, counts = _plain_slots(s["experts"], c["bins"], c["per_bin"], c["cap"])
        return {"index": index, "pair": pair, "counts": counts}
    if op == "combine":
        return _plain_combine(s)
    if op == "combine_bwd":
        return _plain_combine_bwd(s)
    return _plain_w4(s)


# ------------------------------------------------------------------------------- what a pass must do

def work(case):
    c, op = case, case["op"]
    es = {"f32": 4, "bf16": 2}
    if op == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * es[c["dt"]] + c["T"] * c["topk"] * 8 + 4 * c["E"] * (c["bias"] + c["counts"]), "flops": 8 * n}
    if op == "route_bwd":
        n, m = c["T"] * c["E"], c["T"] * c["topk"]
        dense = c["score"] == "softmax" and not c["renorm"]       # otherwise only the chosen logits are needed
        return {"bytes": (n if dense else m) * es[c["dt"]] + n * es[c["dt"]] + m * 8, "flops": 8 * (n if dense else m)}
    if op == "slots":
        m = c["T"] * c["topk"]
        return {"bytes": 8 * m + 4 * c["bins"] * c["cap"] + 8 * c["bins"], "flops": 2 * m}
    if op in ("combine", "combine_bwd"):
        T, topk, N = c["T"], c["topk"], c["N"]
        m = T * topk
        rows, wide = m * N * es[c["dt"]], T * N * es[c["out"]]
        maps = 4 * m * (2 if c["bins"] else 1)
        if op == "combine":
            return {"bytes": rows + wide * (2 if c["add"] else 1) + maps, "flops": 2 * m * N}
        R = c["bins"] * c["cap"] if c["bins"] else m
        return {"bytes": rows + wide + R * N * es[c["dt"]] + maps + 4 * m + (4 * R if c["bins"] else 0), "flops": 3 * m * N}
    T, topk, E, K, N = c["T"], c["topk"], c["E"], c["K"], c["N"]
    hit = E * (1 - (1 - topk / E) ** T)                           # experts that some token chose, on average
    per = K * N / 2 + 2 * -(-K // c["group"]) * N * (2 if c["zeros"] else 1)
    return {"bytes": hit * per + 2 * K * (T if c["up"] else T * topk) + T * topk * N * es[c["out"]],
            "flops": 2 * T * topk * K * N}


# ----------------------------------------------------------------- the definitions, in 64 bits, apart

def _exact_route(c, s):
    x = s["logits"].double()
    on = torch.isfinite(x) | (x == float("inf"))
    if c["score"] == "softmax":
        f = torch.exp(x - torch.logsumexp(x.masked_fill(~on, float("-inf")), 1, keepdim=True)).masked_fill(~on, 0.0)
    else:
        f = torch.sigmoid(x).masked_fill(~on, 0.0)
    v = f + (s["bias"].double() if s["bias"] is not None else 0.0)
    low = float("-inf")
    v = v.masked_fill(~on, low)
    T, E = v.shape
    if c["groups"] > 1:
        size = E // c["groups"]
        u = v.unflatten(1, (c["groups"], size))
        t = u.topk(min(c["group_top"], size), dim=2).values
        gs = t.masked_fill(t == low, 0.0).sum(2).masked_fill(~(t[..., 0] > low), low)
        n = torch.arange(c["groups"], device=v.device)
        ahead = (gs[:, None, :] > gs[:, :, None]) | ((gs[:, None, :] == gs[:, :, None]) & (n[None, None, :] < n[None, :, None]))
        v = v.masked_fill((ahead.sum(2) >= c["take"]).repeat_interleave(size, 1), low)
    n = torch.arange(E, device=v.device)
    rank = torch.empty(T, E, dtype=torch.long, device=v.device)
    for i in range(0, T, 4096):                                   # how many stand before each expert
        b = v[i:i + 4096]
        rank[i:i + 4096] = ((b[:, None, :] > b[:, :, None]) | ((b[:, None, :] == b[:, :, None]) & (n < n[:, None]))).sum(2)
    taken = (rank < c["topk"]) & (v > low)
    experts = torch.full((T, c["topk"] + 1), -1, dtype=torch.long, device=v.device)
    weights = torch.zeros((T, c["topk"] + 1), dtype=torch.float64, device=v.device)
    if c["renorm"]:
        f = f / f.masked_fill(~taken, 0.0).sum(1, keepdim=True)
    place = torch.where(taken, rank, c["topk"])
    experts.scatter_(1, place, n.expand(T, E))
    weights.scatter_(1, place, f * c["scale"])
    out = {"experts": experts[:, :-1].to(torch.int32), "weights": weights[:, :-1]}
    if c["counts"]:
        out["counts"] = taken.sum(0).to(torch.int32)
    return out


def _exact_route_bwd(c, s):
    """Through the chosen logits' log-scores: dw/dx of w = scale * f, or of w = scale * f / sum f."""
    x = s["logits"].double()
    on = x > float("-inf")
    n = torch.arange(c["E"], device=x.device)
    pick = (s["experts"][:, :, None] == n).double()               # [T][topk][E]
    g = s["dweights"].double() * c["scale"]
    if c["score"] == "softmax":
        f = torch.nan_to_num(torch.softmax(x, 1))
    else:
        f = torch.sigmoid(x)
    chosen = (pick * f[:, None, :]).sum(2)
    live = pick.sum(2) > 0
    g = torch.where(live, g, 0.0)
    if c["renorm"]:
        sums = chosen.sum(1, keepdim=True)
        p = torch.where(live, chosen / sums, 0.0)
        dlog = p * (g - (p * g).sum(1, keepdim=True))             # gradient of the chosen log-scores
    else:
        dlog = chosen * g
    d = (pick * dlog[:, :, None]).sum(1)
    if c["score"] == "softmax":
        d = d - f * dlog.sum(1, keepdim=True)
    else:
        d = d * (1 - f)
    return {"dlogits": d.masked_fill(~on, 0.0)}


def _exact_slots(c, s):
    e = s["experts"].reshape(-1).long()
    b = torch.where((e >= 0) & (e < c["bins"] * c["per_bin"]), torch.div(e, c["per_bin"], rounding_mode="floor"), c["bins"])
    counts = torch.bincount(b, minlength=c["bins"] + 1)[:c["bins"]]
    order = torch.argsort(b, stable=True)                         # pairs by bin, in pair order
    first = torch.cumsum(counts, 0) - counts
    index = torch.full_like(e, -1)
    pair = torch.full((c["bins"], c["cap"]), -1, dtype=torch.long, device=e.device)
    for r in range(c["bins"]):
        mine = order[int(first[r]):int(first[r] + counts[r])][:c["cap"]]
        index[mine] = r * c["cap"] + torch.arange(mine.numel(), device=e.device)
        pair[r, :mine.numel()] = mine
    return {"index": index.view(c["T"], c["topk"]).to(torch.int32), "pair": pair.view(-1).to(torch.int32), "counts": counts}


def _exact_combine(c, s):
    T, topk, N = c["T"], c["topk"], c["N"]
    at = s["index"].long() if s["index"] is not None else torch.arange(T * topk, device="cuda").view(T, topk)
    rows, w = s["rows"], s["weights"].double()
    out = s["add"].double() if s.get("add") is not None else torch.zeros(T, N, dtype=torch.float64, device="cuda")
    drows = torch.zeros(rows.shape, dtype=torch.float64, device="cuda") if c["op"] == "combine_bwd" else None
    dw = torch.zeros(T, topk, dtype=torch.float64, device="cuda")
    for j in range(topk):
        t = (at[:, j] >= 0).nonzero()[:, 0]
        r = at[t, j]
        if drows is None:
            out[t] += w[t, j, None] * rows[r].double()
        else:
            d = s["dout"][t].double()
            drows[r] = w[t, j, None] * d
            dw[t, j] = (d * rows[r].double()).sum(1)
    return {"out": out} if drows is None else {"drows": drows, "dweights": dw}


def _exact_w4(c, s):
    K, N, group, topk = c["K"], c["N"], c["group"], c["topk"]
    wq = s["wq"].long() & 0xFFFFFFFF
    R = c["T"] * topk
    out = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    experts = s["experts"].tolist() if s["experts"] is not None else [0] * R
    k = torch.arange(K, device="cuda")
    n = torch.arange(N, device="cuda")
    piece = (k % 32 // 8)[:, None] * 16 + (n % 16)[None, :]
    shift = ((3 + 16 * (k % 2) + 4 * (k % 8 // 2)) % 32)[:, None]
    for e in sorted(set(experts)):
        word = wq[e][(n // 16)[None, :], (k // 128)[:, None], piece, (k % 128 // 32)[:, None]]
        q = ((word >> shift) | (word << (32 - shift))) & 15
        at = ((n // 16)[None, :], (k // group)[:, None], (n % 16)[None, :])
        z = s["zeros"][e][at].double() if s["zeros"] is not None else 8.0
        w = s["scales"][e][at].double() * (q.double() - z)
        mine = [r for r in range(R) if experts[r] == e]
        src = [r // topk if c["up"] else r for r in mine]
        out[mine] = s["x"][src].double() @ w
    return {"out": out}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "route":
        return _exact_route(case, s)
    if op == "route_bwd":
        return _exact_route_bwd(case, s)
    if op == "slots":
        return _exact_slots(case, s)
    if op in ("combine", "combine_bwd"):
        return _exact_combine(case, s)
    return _exact_w4(case, s)
