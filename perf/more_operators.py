"""More operators of a decode step, as cases that can be timed and compared.

    norm       what stands between two blocks: the block's output through its own norm, gate and scale
               onto the residual stream, and the norm before the next block
    moe        a whole mixture-of-experts layer for a few tokens: router, choice of the experts, their
               int4 gate+up products, SwiGLU, their int4 down products, the weighted sum
    logprobs   of rows of fp16 logits: log probabilities and ranks of given tokens, the entropy, the
               first alternatives

With ``own`` false every operator is computed by elementary torch operations; with ``own`` true by the
calls of ``w4a16_weight_streaming_gb300``. The sizes are those of the dense layers here (hidden 5120; an
MLP of 17,408 columns, here as 8 experts of 2176 a token; an output head of 248,320 columns), and smaller
or odd ones of the same kinds.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one stream's decode step: latency of the smallest call
        _norm("norm_one", rows=1, width=5120, post=True, gate="none", scale=1.0, stream="f16", offset=0.0),
        # 64 streams, norms on both sides, a gate per channel and a scaled branch, weights stored as w - 1
        _norm("norm_streams", rows=64, width=5120, post=True, gate="channel", scale=0.7, stream="f16", offset=1.0),
        # one prompt chunk of the largest row count that the layer products are measured at, fp32 residual stream
        _norm("norm_chunk", rows=1024, width=5120, post=False, gate="none", scale=1.0, stream="f32", offset=0.0),
        # a whole prompt, every element gated (rows modulated one by one)
        _norm("norm_prompt", rows=8192, width=5120, post=True, gate="element", scale=1.0, stream="f16", offset=0.0),
        # one stream's decode step through 8 of 64 experts (together the dense layer's MLP)
        _moe("moe_one", tokens=1, experts=64, top=8, hidden=5120, inner=2176, group=128, sigmoid=False),
        # a few streams, small experts of odd sizes, scores by sigmoid with a balancing bias
        _moe("moe_small", tokens=5, experts=24, top=2, hidden=1280, inner=448, group=64, sigmoid=True),
        # 16 verified positions: most experts are hit, one to a few tokens each
        _moe("moe_verify", tokens=16, experts=64, top=8, hidden=5120, inner=2176, group=128, sigmoid=False),
        # 64 streams: every expert is hit, 8 tokens each on average
        _moe("moe_streams", tokens=64, experts=64, top=8, hidden=5120, inner=2176, group=128, sigmoid=True),
        # one stream's drawn token with 20 alternatives
        _logprobs("logprobs_one", rows=1, vocab=248320, pad=0, given=1, top=20, tempered=False),
        # 16 verify rows: the drafted token's and the drawn one's probability at the rows' temperatures
        _logprobs("logprobs_verify", rows=16, vocab=248320, pad=0, given=2, top=0, tempered=True),
        # 33 streams, an odd vocabulary in padded rows, 5 alternatives
        _logprobs("logprobs_odd", rows=33, vocab=32003, pad=29, given=1, top=5, tempered=True),
        # scoring a piece of a prompt: every position's own next token, the first alternative beside it
        _logprobs("logprobs_prompt", rows=1024, vocab=248320, pad=0, given=1, top=1, tempered=False),
    ]


def _norm(name, **kw):
    return dict(name=name, op="norm", **kw)


def _moe(name, **kw):
    return dict(name=name, op="moe", **kw)


def _logprobs(name, **kw):
    return dict(name=name, op="logprobs", **kw)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "moe", "moe", "logprobs"])
    if op == "norm":
        return dict(op=op, rows=_log_int(rng, 1, 8192), width=8 * _log_int(rng, 8, 640), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "element", "row"]), scale=rng.choice([1.0, 0.22, 0.7]),
                    stream=rng.choice(["f16", "f16", "f32"]), offset=rng.choice([0.0, 1.0]))
    if op == "logprobs":
        return dict(op=op, rows=_log_int(rng, 1, 1024), vocab=_log_int(rng, 1000, 248320), pad=rng.choice([0, 0, 5, 32]),
                    given=rng.choice([1, 1, 2, 7]), top=rng.choice([0, 1, 5, 20, 32]), tempered=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    unit = max(group, 64)
    experts = _log_int(rng, 4, 64)
    return dict(op=op, tokens=_log_int(rng, 1, 64), experts=experts, top=rng.randint(1, min(8, experts)),
                hidden=unit * _log_int(rng, 512 // unit, 5120 // unit), inner=unit * _log_int(rng, 256 // unit, 2176 // unit),
                group=group, sigmoid=rng.random() < 0.5)


def _hit(case):
    """Experts that a batch of independent tokens is expected to choose at least once."""
    return case["experts"] * (1.0 - (1.0 - case["top"] / case["experts"]) ** case["tokens"])


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        stream = 2 if case["stream"] == "f16" else 4
        gate = {"none": 0, "channel": 2 * case["width"], "element": 2 * n, "row": 2 * case["rows"]}[case["gate"]]
        return {"bytes": n * (2 * stream + 2 + 2) + gate + case["width"] * (4 if case["post"] else 2),
                "flops": n * (12 if case["post"] else 8)}
    if case["op"] == "logprobs":
        return {"bytes": case["rows"] * (2 * case["vocab"] + 12 * case["given"] + 8 * case["top"] + 4),
                "flops": case["rows"] * case["vocab"] * 5}
    t, h, i, g, e, k = (case[n] for n in ("tokens", "hidden", "inner", "group", "experts", "top"))
    matrix = 3 * h * i  # gate, up and down of one expert
    return {"bytes": int(_hit(case) * (matrix // 2 + matrix // g * 2)) + e * h * 2 + 2 * t * h * 2 + t * k * 8,
            "flops": 2 * t * k * matrix + 2 * t * e * h}


# --------------------------------------------------------------------------------------- inputs
def _gen(seed, part=0):
    return torch.Generator("cuda").manual_seed((seed * 1000003 + part) & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _norm_inputs(case, seed):
    m, n = case["rows"], case["width"]
    gen = _gen(seed)
    channels = torch.exp(0.5 * _randn(gen, n))  # a residual stream's channels differ, a few are large
    channels[torch.randint(0, n, (2,), generator=gen, device="cuda")] *= 20
    h = 3.0 * _randn(gen, m, n) * channels
    inp = dict(h=h if case["stream"] == "f32" else h.half(), y=_randn(gen, m, n).half())
    inp["weight"] = (1.0 - case["offset"] + 0.2 * _randn(gen, n)).half()
    inp["post"] = (1.0 - case["offset"] + 0.2 * _randn(gen, n)).half() if case["post"] else None
    shape = {"none": None, "channel": (n,), "element": (m, n), "row": (m, 1)}[case["gate"]]
    inp["gate"] = None if shape is None else (0.5 + 0.5 * torch.rand(shape, generator=gen, device="cuda")).half()
    return inp


def _matrices(gen, e, rows, cols, group):
    """Canonical int4 matrices of e experts: words of 8 codes along the rows, one fp16 scale a group."""
    words = torch.randint(-2 ** 31, 2 ** 31, (e, rows // 8, cols), generator=gen, device="cuda", dtype=torch.int32)
    scales = (0.002 * (1.0 + torch.rand((e, rows // group, cols), generator=gen, device="cuda"))).half()
    return words, scales


def _moe_inputs(case, seed):
    t, h, i, g, e = (case[n] for n in ("tokens", "hidden", "inner", "group", "experts"))
    gen = _gen(seed)
    inp = dict(x=(_randn(gen, t, h) * torch.exp(0.2 * _randn(gen, h))).half(),
               router=(_randn(gen, e, h) * (1.5 / math.sqrt(h))).half(),
               bias=0.05 * _randn(gen, e) if case["sigmoid"] else None)
    inp["gate_up"] = _matrices(gen, e, h, 2 * i, g)
    inp["down"] = _matrices(gen, e, i, h, g)
    return inp


def _logprobs_inputs(case, seed):
    m, v = case["rows"], case["vocab"]
    gen = _gen(seed)
    wide = 2.0 * _randn(gen, m, v + case["pad"])
    best = torch.randint(0, v, (m, 24), generator=gen, device="cuda")  # a few likely tokens a row
    wide.scatter_add_(1, best, 9.0 + 3.0 * _randn(gen, m, 24))
    likely = torch.rand((m, case["given"]), generator=gen, device="cuda") < 0.7
    which = torch.randint(0, 24, (m, case["given"]), generator=gen, device="cuda")
    any_ = torch.randint(0, v, (m, case["given"]), generator=gen, device="cuda")
    inp = dict(logits=wide.half()[:, :v], tokens=torch.where(likely, best.gather(1, which), any_).int(), temperature=None)
    if case["tempered"]:
        inp["temperature"] = 0.5 + torch.rand(m, generator=gen, device="cuda")
    return inp


def prepare(case, seed):
    s = dict(case=case)
    s.update({"norm": _norm_inputs, "moe": _moe_inputs, "logprobs": _logprobs_inputs}[case["op"]](case, seed))
    if own and case["op"] == "moe":
        import w4a16_weight_streaming_gb300 as W
        s["layer"] = W.Experts(*s.pop("gate_up"), *s.pop("down"), group=case["group"])
        s["workspace"] = W.moe_workspace(s["layer"])
    return s


# ---------------------------------------------------------------------------------- plain forms
def _plain_rms(x, weight, offset):
    return x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * (offset + weight.float())


def _plain_norm(s):
    case = s["case"]
    branch = s["y"].float()
    if s["post"] is not None:
        branch = _plain_rms(branch, s["post"], case["offset"])
    if s["gate"] is not None:
        branch = branch * s["gate"].float()
    h = s["h"].float() + case["scale"] * branch
    return {"h": h.to(s["h"].dtype), "x": _plain_rms(h, s["weight"], case["offset"]).half()}


def _plain_weights(words, scales, group):
    """fp32 [rows, cols] of one matrix: fp16((code - 8) * scale), the format's own rounding."""
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)[None, :, None]
    code = ((words[:, None, :] >> shift) & 15).reshape(-1, words.shape[1]) - 8
    w = code.float().unflatten(0, (-1, group)) * scales.float()[:, None, :]
    return w.flatten(0, 1).half().float()


def _plain_route(s):
    """Chosen experts [T, k] in order, and their weights. The logits are summed up in 64 bits: a choice
    next to a tie should not hang on the order of a sum."""
    case = s["case"]
    logits = (s["x"].double() @ s["router"].double().T).float()
    if case["sigmoid"]:
        score = 1.0 / (1.0 + torch.exp(-logits))
        key = score + s["bias"]
    else:
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
        key = logits
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, : case["top"]]
    w = score.gather(1, ids)
    return ids, w / w.sum(1, keepdim=True)


def _plain_expert(s, e, rows):
    case = s["case"]
    gate_up = rows @ _plain_weights(s["gate_up"][0][e], s["gate_up"][1][e], case["group"])
    gate, up = gate_up[:, : case["inner"]], gate_up[:, case["inner"]:]
    return (gate / (1.0 + torch.exp(-gate)) * up) @ _plain_weights(s["down"][0][e], s["down"][1][e], case["group"])


def _plain_moe(s):
    case = s["case"]
    ids, w = _plain_route(s)
    x = s["x"].float()
    out = torch.zeros_like(x)
    if case["tokens"] * case["top"] < case["experts"]:  # by (token, expert) pairs: fewer than experts
        for t in range(case["tokens"]):
            for j in range(case["top"]):
                at = ids[t, j:j + 1]
                one = dict(s, gate_up=[m.index_select(0, at) for m in s["gate_up"]], down=[m.index_select(0, at) for m in s["down"]])
                out[t] += w[t, j] * _plain_expert(one, 0, x[t:t + 1])[0]
    else:
        share = torch.zeros((case["tokens"], case["experts"]), device="cuda").scatter(1, ids, w)
        for e in range(case["experts"]):
            out += share[:, e:e + 1] * _plain_expert(s, e, x)
    return {"y": out.half(), "ids": ids.int(), "weights": w}


def _plain_logprobs(s):
    case = s["case"]
    x = s["logits"].float()
    t = 1.0 if s["temperature"] is None else s["temperature"][:, None]
    d = (x - x.amax(1, keepdim=True)) / t
    w = torch.exp(d)
    total = w.sum(1, keepdim=True)
    log_total = torch.log(total)
    at = s["tokens"].long()
    value = x.gather(1, at)
    index = torch.arange(x.shape[1], device="cuda")[None, :]
    rank = [((x > value[:, j:j + 1]) | ((x == value[:, j:j + 1]) & (index < at[:, j:j + 1]))).sum(1) + 1 for j in range(case["given"])]
    out = {"logprob": d.gather(1, at) - log_total, "rank": torch.stack(rank, 1).int(),
           "entropy": (log_total - (w * d).sum(1, keepdim=True) / total)[:, 0]}
    if case["top"]:
        best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, : case["top"]]
        out["top_tokens"], out["top_logprob"] = best.int(), d.gather(1, best) - log_total
    return out


def run(s):
    case = s["case"]
    if not own:
        return {"norm": _plain_norm, "moe": _plain_moe, "logprobs": _plain_logprobs}[case["op"]](s)
    import w4a16_weight_streaming_gb300 as W
    if case["op"] == "norm":
        h, x = W.block_norm(s["h"], s["y"], weight=s["weight"], post_weight=s["post"], gate=s["gate"], scale=case["scale"],
                            eps=EPS, offset=case["offset"])
        return {"h": h, "x": x}
    if case["op"] == "moe":
        y, ids, weights = W.moe(s["x"], s["layer"], s["router"], case["top"], s["workspace"], bias=s["bias"],
                                sigmoid=case["sigmoid"])
        return {"y": y, "ids": ids, "weights": weights}
    r = W.logprobs(s["logits"], s["tokens"], top=case["top"], temperature=s["temperature"])
    out = {"logprob": r.logprob, "rank": r.rank, "entropy": r.entropy}
    if case["top"]:
        out["top_tokens"], out["top_logprob"] = r.top_tokens, r.top_logprob
    return out


# --------------------------------------------------------------------------- the same in 64 bits
def _exact_norm(case, seed):
    inp = _norm_inputs(case, seed)

    def unit(v, gain):
        rms = torch.linalg.vector_norm(v, dim=1, keepdim=True).square() / v.shape[1] + EPS
        return v * rms.rsqrt() * (gain.double() + case["offset"])

    z = inp["y"].double()
    if inp["post"] is not None:
        z = unit(z, inp["post"])
    z *= case["scale"] * (1.0 if inp["gate"] is None else inp["gate"].double())
    z += inp["h"].double()
    return {"h": z, "x": unit(z, inp["weight"])}


def _decoded64(words, scales, group):
    rows, cols = words.shape[0] * 8, words.shape[1]
    out = torch.empty((rows, cols), dtype=torch.float64, device="cuda")
    wide = scales.repeat_interleave(group, dim=0)
    for j in range(8):  # code 8 stands for zero; one rounding to fp16 belongs to the format
        out[j::8] = ((words.bitwise_right_shift(4 * j).bitwise_and(15) - 8).double() * wide[j::8].double()).half().double()
    return out


def _exact_moe(case, seed):
    inp = _moe_inputs(case, seed)
    t, k, i = case["tokens"], case["top"], case["inner"]
    x = inp["x"].double()
    logits = torch.einsum("th,eh->te", x, inp["router"].double())
    score = torch.sigmoid(logits) if case["sigmoid"] else torch.softmax(logits, dim=1)
    key = score + inp["bias"].double() if case["sigmoid"] else logits
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    weights = score.gather(1, ids)
    weights /= weights.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist())):
        row, col = (ids == e).nonzero(as_tuple=True)
        both = x[row] @ _decoded64(inp["gate_up"][0][e], inp["gate_up"][1][e], case["group"])
        act = both[:, :i] * torch.sigmoid(both[:, :i]) * both[:, i:]
        y.index_add_(0, row, weights[row, col, None] * (act @ _decoded64(inp["down"][0][e], inp["down"][1][e], case["group"])))
    return {"y": y, "ids": ids.int(), "weights": weights}


def _exact_logprobs(case, seed):
    inp = _logprobs_inputs(case, seed)
    m, k = case["rows"], case["top"]
    parts = {n: [] for n in ("logprob", "rank", "entropy", "top_tokens", "top_logprob")}
    for r in range(m):
        l = inp["logits"][r].double()
        z = l / (1.0 if inp["temperature"] is None else float(inp["temperature"][r]))
        lp = z - torch.logsumexp(z, 0)
        order = torch.argsort(l, descending=True, stable=True)
        place = torch.empty_like(order)
        place[order] = torch.arange(1, len(order) + 1, device="cuda")
        at = inp["tokens"][r].long()
        parts["logprob"].append(lp[at])
        parts["rank"].append(place[at].int())
        parts["entropy"].append(-(lp.exp() * lp).sum())
        parts["top_tokens"].append(order[:k].int())
        parts["top_logprob"].append(lp[order[:k]])
    out = {n: torch.stack(v) for n, v in parts.items()}
    return out if k else {n: out[n] for n in ("logprob", "rank", "entropy")}


def exact(case, seed):
    with torch.no_grad():
        return {"norm": _exact_norm, "moe": _exact_moe, "logprobs": _exact_logprobs}[case["op"]](case, seed)
