"""Products with 8-bit integers and their backward passes, as cases to measure.

Six operators, each with its plain form (elementary torch operations) and the library's calls:

  save     rows of activations -> 8-bit codes with one scale a row, optionally through SiLU and with the
           codes of what SiLU was given beside those of its result; and their reading back;
  weights  the experts' matrices -> 8-bit codes with one scale for each output channel, in the order the
           products read; and their reading back;
  linear   rows of activations -> codes -> their experts' products in 8-bit integers, rows grouped by
           expert (or one matrix for all);
  decode   the same for a few token rows, each with an expert of its own choice;
  dx       the gradient of a product's rows from the weights' codes, optionally through SiLU's derivative
           at the rows that were kept as codes;
  dw       the gradient of a product's weights from the rows that were kept as codes.

`own` selects the side that prepare() and run() take: False, the plain form; True, the library's kernels.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TINY = 2.0 ** -126                                                # the smallest scale


# ---------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # four tokens of a decode step before their experts' up projection: latency only
        dict(name="save_decode", op="save", T=4, K=4096, ld=4096, dt="bf16", act="none", keep=False),
        # 8 ranks x 4096 tokens' hidden rows of a training step: through SiLU, both sides of it kept
        dict(name="save_train", op="save", T=32768, K=1792, ld=1792, dt="bf16", act="silu", keep=True),
        # one rank's four experts, after an optimiser step
        dict(name="weights_rank", op="weights", E=4, K=4096, N=1792, dt="bf16"),
        # three small matrices of odd sizes in fp32
        dict(name="weights_ragged", op="weights", E=3, K=1040, N=1000, dt="f32"),
        # a prompt's 201 rows with one matrix of an odd size: fewer tiles than the device has CUs
        dict(name="linear_prompt", op="linear", E=1, T=201, K=1040, N=1000, dt="bf16", out="f32"),
        # 8192 rows on one rank's four experts, groups of any length, one of them empty: up projection
        dict(name="linear_experts", op="linear", E=4, T=8192, K=4096, N=1792, dt="bf16", out="bf16"),
        # one token's eight experts of 64, up projection 4096 -> 1792
        dict(name="decode_token", op="decode", T=1, topk=8, E=64, K=4096, N=1792, out="bf16", up=True),
        # sixteen tokens, top-2 of 32 experts, down projection 1792 -> 4096
        dict(name="decode_batch", op="decode", T=16, topk=2, E=32, K=1792, N=4096, out="f32", up=False),
        # the backward pass of a prompt-sized product, without an activation before it
        dict(name="dx_prompt", op="dx", E=1, T=333, K=1040, N=1000, act="none", out="f32"),
        # the down projection's backward pass of 8192 rows on four experts, through SiLU to its input's gradient
        dict(name="dx_experts", op="dx", E=4, T=8192, K=1792, N=4096, act="silu", out="bf16"),
        # weight gradients of a few hundred rows on three experts of an odd size, one without rows
        dict(name="dw_ragged", op="dw", E=3, T=501, K=1040, N=1000, out="bf16"),
        # weight gradients of 8192 rows on one rank's four experts, for an accumulation in fp32
        dict(name="dw_experts", op="dw", E=4, T=8192, K=4096, N=1792, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["save", "save", "weights", "linear", "linear", "decode", "decode", "dx", "dx", "dw", "dw"])
    K, N = 16 * _log(rng, 4, 256), 8 * _log(rng, 8, 512)
    if op == "save":
        dt = rng.choice(["bf16", "bf16", "f32"])
        act = rng.choice(["none", "silu"]) if dt == "bf16" else "none"
        return dict(op=op, T=_log(rng, 1, min(32768, 58_000_000 // K)), K=K, ld=K + rng.choice([0, 0, 8]), dt=dt, act=act,
                    keep=act == "silu" and rng.random() < 0.5)
    if op == "weights":
        return dict(op=op, E=rng.randint(1, max(1, min(8, 29_000_000 // (K * N)))), K=K, N=N, dt=rng.choice(["bf16", "f32"]))
    if op == "decode":
        E = rng.choice([1, 8, 32, 64])
        T, topk = (_log(rng, 1, 64), 1) if E == 1 else (_log(rng, 1, 16), rng.choice([1, 2, 4, 8]))
        if E > 1:
            N = 8 * max(1, min(N, 200_000_000 // (T * topk * K), 200_000_000 // (E * K)) // 8)
        return dict(op=op, T=T, topk=topk, E=E, K=K, N=N, out=rng.choice(["bf16", "f32"]), up=rng.random() < 0.5)
    c = dict(op=op, E=rng.choice([1, 1, 3, 8]), T=_log(rng, 1, min(16384, 6 * 10 ** 10 // (K * N))), K=K, N=N,
             out=rng.choice(["bf16", "f32"]))
    if op == "linear":
        c["dt"] = rng.choice(["bf16", "bf16", "f32"])
    elif op == "dx":
        c["act"] = rng.choice(["none", "silu"])
    return c


# --------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _codes(T, K, g, std):
    """Codes and scales of T rows of K normal numbers of this deviation."""
    x = std * torch.randn(T, K, generator=g, device="cuda")
    scale = (x.abs().amax(1) / 127).clamp_min(TINY)
    return (x / scale[:, None]).round_().to(torch.int8), scale


def _offsets(T, E, g):
    """First rows of E groups of any length, the second of three or more without rows; the longest group."""
    share = torch.rand(E, generator=g, device="cuda") + 0.2
    if E > 2:
        share[1] = 0.0
    end = (share.cumsum(0) / share.sum() * T).round().long()
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), end])
    off[-1] = T
    return off, int((off[1:] - off[:-1]).max())


def prepare(case, seed):
    c, g = case, _gen(seed)
    op, K = c["op"], c["K"]
    s = {"case": c}
    if op == "save":
        x = torch.full((c["T"], c["ld"]), float("nan"), device="cuda")   # what stands beside the rows is not theirs
        x[:, :K] = torch.randn(c["T"], K, generator=g, device="cuda") * torch.exp(torch.randn(c["T"], 1, generator=g, device="cuda"))
        if c["T"] > 2:
            x[1, :K] = 0.0                                        # a padding row
        s["x"] = x.to(DT[c["dt"]])[:, :K]                         # a view: its rows are ld apart
    elif op == "weights":
        s["w"] = (0.02 * torch.randn(c["E"], K, c["N"], generator=g, device="cuda")).to(DT[c["dt"]])
    else:
        E, T, N = c["E"], c["T"], c["N"]
        if op == "decode":
            rows = T if c["up"] else T * c["topk"]
            s["x"] = torch.randn(rows, K, generator=g, device="cuda").to(torch.bfloat16)
            s["experts"] = None
            if E > 1:
                e = torch.rand(T, E, generator=g, device="cuda").topk(c["topk"], dim=1).indices
                s["experts"] = e.to(torch.int32).reshape(-1).contiguous()
        elif op == "linear":
            s["x"] = torch.randn(T, K, generator=g, device="cuda").to(DT[c["dt"]])
        else:
            s["dy"] = (0.01 * torch.randn(T, N, generator=g, device="cuda")).to(torch.bfloat16)
        if op in ("linear", "decode", "dx"):
            wq, ws = _codes(E * N, K, g, 0.02)
            s["wq"], s["ws"] = wq.view(E, N, K), ws.view(E, N)
        if op == "dw":
            s["xq"], s["xs"] = _codes(T, K, g, 1.0)
        if op == "dx" and c["act"] == "silu":
            s["hq"], s["hs"] = _codes(T, K, g, 2.0)
        if op != "decode":
            s["offsets"], s["longest"] = _offsets(T, E, g) if E > 1 else (None, T)
    if own:
        s["calls"] = _handles(s)
    return s


# ---------------------------------------------------------------------------------- the library's side

def _handles(s):
    """What a user's program keeps for its calls: output buffers, workspaces and arguments."""
    from computation_collective_amd import buffers as bf
    from computation_collective_amd import hocf

    c = s["case"]
    op, K = c["op"], c["K"]
    dt = {"f32": hocf.HOCF_F32, "bf16": hocf.HOCF_BF16}
    if op == "save":
        q = bf.QuantI8(c["T"], K, s["x"], act=hocf.HOCF_ACT_SILU if c["act"] == "silu" else hocf.HOCF_ACT_NONE,
                       keep=c["keep"])
        back = [bf.DequantI8(c["T"], K, q.codes, q.scales, out_dt=dt[c["dt"]])]
        if c["keep"]:
            back.append(bf.DequantI8(c["T"], K, q.pre_codes, q.pre_scales, out_dt=dt[c["dt"]]))
        return [q] + back
    E, N = c["E"], c["N"]
    if op == "weights":
        q = bf.WeightsI8(E, N, K, s["w"])
        return [q, bf.DequantI8(E * N, K, q.wq.view(E * N, K), q.scales.view(E * N), out_dt=dt[c["dt"]])]
    T, out = c["T"], dt[c["out"]]
    if op == "linear":
        q = bf.QuantI8(T, K, s["x"])
        return [q, bf.GemmI8(E, T, N, K, q.codes, q.scales, s["wq"], s["ws"], offsets=s["offsets"], out_dt=out)]
    if op == "decode":
        q = bf.QuantI8(s["x"].shape[0], K, s["x"])
        return [q, bf.GemvI8(T * c["topk"], c["topk"] if c["up"] else 1, E, 0, N, K, q.codes, q.scales, s["experts"],
                             s["wq"], s["ws"], out_dt=out)]
    if op == "dx":
        return [bf.GemmI8Dx(E, T, N, K, s["dy"], s["wq"], s["ws"], offsets=s["offsets"], pre_codes=s.get("hq"),
                            pre_scales=s.get("hs"), out_dt=out)]
    return [bf.GemmI8Dw(E, T, N, K, s["xq"], s["xs"], s["dy"], offsets=s["offsets"], out_dt=out)]


def _bf16(t):
    return t.view(torch.bfloat16) if t.dtype == torch.int16 else t


def _run_own(s):
    c, calls = s["case"], s["calls"]
    calls[0].run()
    if c["op"] == "save":
        calls[1].run()
        if c["keep"]:
            calls[2].run()
            return {"x": _bf16(calls[1].out), "pre": _bf16(calls[2].out)}
        return {"x": _bf16(calls[1].out)}
    if c["op"] in ("dx", "dw"):
        return {c["op"]: _bf16(calls[0].out)}
    calls[1].run()
    return {"w" if c["op"] == "weights" else "out": _bf16(calls[1].out)}


# ---------------------------------------------------------------------------------- the plain forms

def _plain_quant(a):
    """Codes (as fp32) and scales of fp32 rows: the quotients' borders need 64 bits."""
    top = a.abs().amax(-1, keepdim=True)
    scale = (top / torch.full_like(top, 127)).clamp_min(TINY)     # (a quotient by a number would be a product)
    return torch.round(a.double() / scale.double()).float(), scale


def _read_back(q, scale, dt):
    return (q * scale).to(dt)


def _padded(s, t):
    """The groups' rows, each group filled up with zero rows: [E][longest][..]; and the rows' numbers (T: none)."""
    off = s["offsets"]
    T = t.shape[0]
    if off is None:
        return t[None], None
    at = off[:-1, None] + torch.arange(s["longest"], device=t.device)
    at = torch.where(at < off[1:, None], at, T)
    return torch.cat([t, torch.zeros_like(t[:1])])[at], at


def _unpadded(y, at, T):
    if at is None:
        return y[0]
    out = torch.zeros(T + 1, y.shape[2], device=y.device)
    out[at.reshape(-1)] = y.reshape(-1, y.shape[2])
    return out[:T]


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "save":
        dt = DT[c["dt"]]
        pre = s["x"].float()
        if c["act"] == "silu":
            x = s["x"].double()                                   # the result's rounding to bf16 has borders too
            act = (x / (1 + torch.exp(-x))).to(dt).float()
        else:
            act = pre
        out = {"x": _read_back(*_plain_quant(act), dt)}
        if c["keep"]:
            out["pre"] = _read_back(*_plain_quant(pre), dt)
        return out
    if op == "weights":
        q, scale = _plain_quant(s["w"].float().transpose(1, 2).contiguous())
        return {"w": _read_back(q, scale, DT[c["dt"]]).view(c["E"] * c["N"], c["K"])}
    T, out = c["T"], DT[c["out"]]
    if op == "linear":
        q, scale = _plain_quant(s["x"].float())
        rows, at = _padded(s, q)
        y = torch.bmm(rows, s["wq"].float().transpose(1, 2).contiguous())
        return {"out": (_unpadded(y * s["ws"][:, None, :], at, T) * scale).to(out)}
    if op == "decode":
        q, scale = _plain_quant(s["x"].float())
        if c["up"] and c["topk"] > 1:
            q, scale = q.repeat_interleave(c["topk"], 0), scale.repeat_interleave(c["topk"], 0)
        if s["experts"] is None:
            return {"out": (q @ s["wq"][0].float().t() * scale * s["ws"][0]).to(out)}
        e = s["experts"].long()
        y = torch.bmm(s["wq"][e].float(), q[:, :, None])[:, :, 0]
        return {"out": (y * scale * s["ws"][e]).to(out)}
    if op == "dx":
        w = _read_back(s["wq"].float(), s["ws"][:, :, None], torch.bfloat16).float()
        rows, at = _padded(s, s["dy"].float())
        d = _unpadded(torch.bmm(rows, w), at, T)
        if c["act"] == "silu":
            h = _read_back(s["hq"].float(), s["hs"][:, None], torch.bfloat16).float()
            p = 1 / (1 + torch.exp(-h))
            d = d * (p * (1 + h * (1 - p)))
        return {"dx": d.to(out)}
    rows, _ = _padded(s, _read_back(s["xq"].float(), s["xs"][:, None], torch.bfloat16).float())
    dy, _ = _padded(s, s["dy"].float())
    return {"dw": torch.bmm(rows.transpose(1, 2).contiguous(), dy).to(out)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    c = case
    es = {"f32": 4, "bf16": 2}
    op, K = c["op"], c["K"]
    if op == "save":                                              # codes are written, and read to be read back
        n, kinds = c["T"] * K, 2 if c["keep"] else 1
        return {"bytes": n * es[c["dt"]] * (1 + kinds) + kinds * (2 * n + 8 * c["T"]), "flops": (4 + (6 if c["act"] == "silu" else 0)) * n}
    E, N = c["E"], c["N"]
    if op == "weights":
        n = E * K * N
        return {"bytes": n * (2 * es[c["dt"]] + 2) + 8 * E * N, "flops": 4 * n}
    T = c["T"]
    if op == "decode":
        R = T * c["topk"]
        hit = E * (1 - (1 - c["topk"] / E) ** T)                  # experts that some token chose, on average
        return {"bytes": hit * N * (K + 4) + (T if c["up"] else R) * 2 * K + R * N * es[c["out"]], "flops": 2 * R * K * N}
    if op == "linear":
        return {"bytes": T * K * es[c["dt"]] + E * N * (K + 4) + T * N * es[c["out"]], "flops": 2 * T * K * N}
    if op == "dx":
        return {"bytes": T * N * 2 + E * N * (K + 4) + T * K * es[c["out"]] + (T * (K + 4) if c["act"] == "silu" else 0),
                "flops": 2 * T * K * N}
    return {"bytes": T * N * 2 + T * (K + 4) + E * K * N * es[c["out"]], "flops": 2 * T * K * N}


# ----------------------------------------------------------------- the definitions, in 64 bits, apart

def _exact_codes(v):
    """Nearest whole multiples (even on ties) of a 127th of each row's largest magnitude, that in fp32."""
    peak = v.abs().max(dim=-1).values.float()
    unit = torch.maximum(peak / torch.full_like(peak, 127.0), torch.full_like(peak, TINY)).double()
    quotient = v / unit.unsqueeze(-1)
    low = torch.floor(quotient)
    rest = quotient - low
    up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(low, 2) == 1))
    return low + up.double(), unit


def _exact_rows(c, s):
    """(first, last, expert) of the groups that have rows."""
    if s["offsets"] is None:
        return [(0, c["T"], 0)]
    o = s["offsets"].tolist()
    return [(o[e], o[e + 1], e) for e in range(c["E"]) if o[e + 1] > o[e]]


def _held(codes, scales):
    """What codes stand for where bf16 numbers are wanted."""
    return (codes.double() * scales.double().unsqueeze(-1)).to(torch.bfloat16).double()


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, op = case, case["op"]
    dev = "cuda"
    if op == "save":
        x = s["x"].double()
        y = x
        if c["act"] == "silu":
            y = (x * torch.sigmoid(x)).to(DT[c["dt"]]).double()
        q, u = _exact_codes(y)
        out = {"x": q * u[:, None]}
        if c["keep"]:
            q, u = _exact_codes(x)
            out["pre"] = q * u[:, None]
        return out
    if op == "weights":
        w = torch.empty(c["E"] * c["N"], c["K"], dtype=torch.float64, device=dev)
        for e in range(c["E"]):
            q, u = _exact_codes(s["w"][e].t().double())
            w[e * c["N"]:(e + 1) * c["N"]] = q * u[:, None]
        return {"w": w}
    if op == "decode":
        q, u = _exact_codes(s["x"].double())
        R = c["T"] * c["topk"]
        e = s["experts"].tolist() if s["experts"] is not None else [0] * R
        out = torch.empty(R, c["N"], dtype=torch.float64, device=dev)
        for r in range(R):
            i = r // c["topk"] if c["up"] else r
            out[r] = (s["wq"][e[r]].double() * s["ws"][e[r]].double()[:, None]) @ (q[i] * u[i])
        return {"out": out}
    if op == "linear":
        q, u = _exact_codes(s["x"].double())
        out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=dev)
        for a, b, e in _exact_rows(c, s):
            out[a:b] = (q[a:b] * u[a:b, None]) @ (s["wq"][e].double() * s["ws"][e].double()[:, None]).t().contiguous()
        return {"out": out}
    if op == "dx":
        d = torch.zeros(c["T"], c["K"], dtype=torch.float64, device=dev)
        for a, b, e in _exact_rows(c, s):
            d[a:b] = s["dy"][a:b].double() @ _held(s["wq"][e], s["ws"][e])
        if c["act"] == "silu":
            h = _held(s["hq"], s["hs"])
            p = torch.sigmoid(h)
            d = d * (p + h * p * torch.sigmoid(-h))
        return {"dx": d}
    dw = torch.zeros(c["E"], c["K"], c["N"], dtype=torch.float64, device=dev)
    for a, b, e in _exact_rows(c, s):
        dw[e] = _held(s["xq"][a:b], s["xs"][a:b]).t().contiguous() @ s["dy"][a:b].double()
    return {"dw": dw}
