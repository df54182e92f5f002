"""The operators between a decode step's weight products, as cases that can be timed and compared.

    append     norm and position rotation of each head of a fused qkv row, keys and values stored in a
               paged 4-bit cache (then read back as the values the codes stand for)
    attention  attention of the rotated queries over the paged 4-bit cache: one query a sequence, a few
               (verify steps) or a whole prompt chunk
    sample     one token a row from fp16 logits by temperature, top-k, top-p and min-p, from given
               random numbers

With ``own`` false every operator is computed by elementary torch operations in 32 bits; with ``own``
true by the calls of ``w4a16_weight_streaming_gb300``. The head layouts are those of the dense layers
here (hidden 5120, fused qkv 7168 columns = 20 query heads and 2 x 4 key/value heads of 256, or 40 and
2 x 8 of 128); the output head has 248,320 columns.
"""
from __future__ import annotations

import math
import random

import torch

own = False

GROUP = 64          # consecutive elements of a head that share one (scale, minimum) pair
EPS = 1e-6
POSITIONS = 16384   # rows of the rotation table
FIXED = 2.0 ** 40   # sampling weights are whole multiples of 2^-40


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one stream's decode step: latency of the smallest call
        _append("append_one", rows=1, heads=20, kv_heads=4, dim=256, rot=64, adjacent=False, norm=True, page=16),
        # 64 streams decoding, the other head layout, pairs of adjacent elements rotated, no norms
        _append("append_streams", rows=64, heads=40, kv_heads=8, dim=128, rot=128, adjacent=True, norm=False, page=32),
        # one prompt chunk of the largest row count that the layer products are measured at
        _append("append_chunk", rows=1024, heads=20, kv_heads=4, dim=256, rot=64, adjacent=False, norm=True, page=64),
        # one stream, a short context that ends inside a page
        _attention("decode_short", seqs=1, queries=1, context=777, ragged=False, heads=20, kv_heads=4, dim=256, page=16),
        # one stream, a long context: the cache read is the whole cost
        _attention("decode_long", seqs=1, queries=1, context=131072, ragged=False, heads=20, kv_heads=4, dim=256, page=64),
        # 64 streams of different lengths
        _attention("decode_streams", seqs=64, queries=1, context=8192, ragged=True, heads=40, kv_heads=8, dim=128, page=32),
        # 16 streams verifying up to 16 positions each
        _attention("verify_streams", seqs=16, queries=16, context=8192, ragged=True, heads=20, kv_heads=4, dim=256, page=64),
        # a prompt chunk of 1024 positions behind 8192 cached ones
        _attention("prompt_chunk", seqs=1, queries=1024, context=9216, ragged=False, heads=20, kv_heads=4, dim=256, page=64),
        # one stream's next token from the output head's logits
        _sample("sample_one", rows=1, vocab=248320, pad=0, temperature=0.6, top_k=20, top_p=0.95, min_p=0.0, mixed=False),
        # 16 verify rows, min-p alone
        _sample("sample_verify", rows=16, vocab=248320, pad=0, temperature=0.8, top_k=0, top_p=1.0, min_p=0.05, mixed=False),
        # 33 streams with settings of their own (greedy rows among them), an odd vocabulary in padded rows
        _sample("sample_mixed", rows=33, vocab=32003, pad=29, temperature=0.9, top_k=50, top_p=0.9, min_p=0.02, mixed=True),
        # the largest batch, top-p over the whole vocabulary
        _sample("sample_batch", rows=256, vocab=248320, pad=0, temperature=1.0, top_k=0, top_p=0.95, min_p=0.0, mixed=False),
    ]


def _append(name, **kw):
    return dict(name=name, op="append", **kw)


def _attention(name, **kw):
    return dict(name=name, op="attention", **kw)


def _sample(name, **kw):
    return dict(name=name, op="sample", **kw)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    # query heads, key/value heads, head size: the layer's two layouts, and others of the same kinds
    return rng.choice([(20, 4, 256), (40, 8, 128), (16, 16, 64), (24, 4, 256), (14, 2, 64), (32, 8, 128), (5, 1, 256),
                       (9, 3, 128)])


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "sample"])
    if op == "append":
        h, g, d = _heads(rng)
        case = dict(op=op, rows=_log_int(rng, 1, 1024), heads=h, kv_heads=g, dim=d, rot=rng.choice([0, 32, d // 2, d]),
                    adjacent=rng.random() < 0.5, norm=rng.random() < 0.6, page=rng.choice([16, 32, 64, 128]))
        if case["rot"] > d:
            case["rot"] = d
        return case
    if op == "sample":
        vocab = _log_int(rng, 1000, 248320)
        return dict(op=op, rows=_log_int(rng, 1, 256), vocab=vocab, pad=rng.choice([0, 0, 5, 32]),
                    temperature=round(rng.uniform(0.3, 1.3), 3), top_k=rng.choice([0, 1, 20, 50, 1000]),
                    top_p=round(rng.choice([1.0, rng.uniform(0.3, 0.99)]), 3),
                    min_p=round(rng.choice([0.0, rng.uniform(0.005, 0.2)]), 4), mixed=rng.random() < 0.4)
    most = max(work(c)["flops"] for c in listed() if c["op"] == "attention")
    bytes_most = max(work(c)["bytes"] for c in listed() if c["op"] == "attention")
    while True:
        h, g, d = _heads(rng)
        kind = rng.choice(["decode", "verify", "prompt"])
        queries = {"decode": 1, "verify": rng.randint(2, 16), "prompt": _log_int(rng, 17, 1024)}[kind]
        seqs = {"decode": _log_int(rng, 1, 96), "verify": _log_int(rng, 1, 32), "prompt": rng.randint(1, 3)}[kind]
        case = dict(op=op, seqs=seqs, queries=queries, context=queries + _log_int(rng, 1, 131072 if kind == "decode" else 16384),
                    ragged=rng.random() < 0.6, heads=h, kv_heads=g, dim=d, page=rng.choice([16, 32, 64, 128]))
        w = work(case)
        if w["flops"] <= most and w["bytes"] <= bytes_most:
            return case


def _shape(case):
    """(queries, tokens) of each sequence; the last `queries` tokens are the queries' own."""
    rng = random.Random(case["seqs"] * 1000003 + case["queries"] * 1009 + case["context"])
    out = []
    for _ in range(case["seqs"]):
        if case["ragged"]:
            q = rng.randint(max(1, case["queries"] // 2), case["queries"])
            out.append((q, rng.randint(max(q, case["context"] // 16), case["context"])))
        else:
            out.append((case["queries"], case["context"]))
    return out


def work(case):
    if case["op"] == "append":
        m, h, g, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]
        stored = m * 2 * g * (d // 2 + d // GROUP * 4)
        # qkv in, queries out, the cache rows written and read back, keys and values out, angles, slots, positions
        return {"bytes": m * (h + 2 * g) * d * 2 + m * h * d * 2 + 2 * stored + m * 2 * g * d * 2 + m * case["rot"] * 4 + m * 8,
                "flops": m * (h + g) * d * 8 + m * 2 * g * d * 6}
    if case["op"] == "sample":
        return {"bytes": case["rows"] * (case["vocab"] * 2 + 28), "flops": case["rows"] * case["vocab"] * 3}
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    cached = flops = rows = 0
    for q, n in _shape(case):
        cached += n * 2 * g * (d // 2 + d // GROUP * 4)
        flops += 4 * h * d * (q * n - q * (q - 1) // 2)
        rows += q
    return {"bytes": cached + 2 * rows * h * d * 2, "flops": flops}


# --------------------------------------------------------------------------------------- inputs
def _gen(seed, part=0):
    return torch.Generator("cuda").manual_seed((seed * 1000003 + part) & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rope_table(rot):
    """fp32 [POSITIONS, rot]: the cosines of the rot/2 angles of a position, then their sines."""
    inv = 1.0 / (1e6 ** (torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
    a = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def _append_inputs(case, seed):
    m, h, g, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]
    gen = _gen(seed)
    gain = torch.exp(0.5 * _randn(gen, (h + 2 * g) * d))  # channels differ, as a projection's do
    qkv = (_randn(gen, m, (h + 2 * g) * d) * gain).half()
    pages = max(65536 // case["page"], -(-m // case["page"]))
    if m > 64:  # a prompt chunk: consecutive positions of one sequence, in pages of any order
        first = int(torch.randint(0, POSITIONS - m, (1,), generator=gen, device="cuda"))
        pos = torch.arange(first, first + m, device="cuda")
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(m, device="cuda") + first % case["page"]
        slots = order[(at // case["page"]) % pages] * case["page"] + at % case["page"]
    else:  # one new token of each of m sequences
        pos = torch.randint(0, POSITIONS, (m,), generator=gen, device="cuda")
        slots = torch.randperm(pages, generator=gen, device="cuda")[:m] * case["page"] + pos % case["page"]
    inp = dict(qkv=qkv, pos=pos.int(), slots=slots.int(), pages=pages, q_norm=None, k_norm=None, rope=None)
    if case["norm"]:
        inp["q_norm"] = (1.0 + 0.2 * _randn(gen, d)).half()
        inp["k_norm"] = (1.0 + 0.2 * _randn(gen, d)).half()
    if case["rot"]:
        inp["rope"] = _rope_table(case["rot"])
    return inp


def _sequence(case, seed, b, n):
    """Keys and values (fp16 [n, kv_heads, dim]) of sequence b: channels of different size, some large."""
    g, d = case["kv_heads"], case["dim"]
    gen = _gen(seed, 17 + b)
    k = _randn(gen, n, g, d) * torch.exp(0.4 * _randn(gen, g, d))
    v = _randn(gen, n, g, d) * (0.5 * torch.exp(0.4 * _randn(gen, g, d))) + 0.1 * _randn(gen, g, d)
    return k.half(), v.half()


def _attention_inputs(case, seed):
    shape = _shape(case)
    gen = _gen(seed)
    rows = sum(q for q, _ in shape)
    q = (1.5 * _randn(gen, rows, case["heads"], case["dim"])).half()
    need = [-(-n // case["page"]) for _, n in shape]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.zeros((len(shape), max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    starts = [0]
    for a, _ in shape:
        starts.append(starts[-1] + a)
    return dict(q=q, pages=pages, table=table, need=need, shape=shape,
                starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                lens=torch.tensor([n for _, n in shape], dtype=torch.int32, device="cuda"))


def _sample_inputs(case, seed):
    m, v = case["rows"], case["vocab"]
    gen = _gen(seed)
    wide = 2.0 * _randn(gen, m, v + case["pad"])
    best = torch.randint(0, v, (m, 24), generator=gen, device="cuda")  # a few likely tokens a row
    wide.scatter_add_(1, best, 9.0 + 3.0 * _randn(gen, m, 24))
    inp = dict(logits=wide.half()[:, :v], u=torch.rand(m, generator=gen, device="cuda"))
    one = torch.ones(m, device="cuda")
    inp["temperature"] = one * case["temperature"]
    inp["top_k"] = (one * case["top_k"]).int()
    inp["top_p"] = one * case["top_p"]
    inp["min_p"] = one * case["min_p"]
    if case["mixed"]:
        r = torch.arange(m, device="cuda")
        inp["temperature"] = torch.where(r % 5 == 4, torch.zeros_like(one), inp["temperature"] * (0.5 + torch.rand(m, generator=gen, device="cuda")))
        inp["top_k"] = torch.where(r % 3 == 0, inp["top_k"], torch.zeros_like(inp["top_k"]))
        inp["top_p"] = torch.where(r % 2 == 0, inp["top_p"], one)
        inp["min_p"] = torch.where(r % 7 < 3, inp["min_p"], torch.zeros_like(one))
    return inp


def prepare(case, seed):
    if own:
        import w4a16_weight_streaming_gb300 as W
    s = dict(case=case)
    if case["op"] == "append":
        s.update(_append_inputs(case, seed))
        if own:
            s["cache"] = W.KV4Cache(s["pages"], case["page"], case["kv_heads"], case["dim"])
        else:
            s["cache"] = _plain_cache(s["pages"] * case["page"], case["kv_heads"], case["dim"])
        return s
    if case["op"] == "sample":
        s.update(_sample_inputs(case, seed))
        return s
    s.update(_attention_inputs(case, seed))
    g, d, page = case["kv_heads"], case["dim"], case["page"]
    if own:
        s["cache"] = W.KV4Cache(s["pages"], page, g, d)
        s["workspace"] = W.kv4_attention_workspace(s["cache"])
    else:
        s["cache"] = _plain_cache(s["pages"] * page, g, d)
    for b, (_, n) in enumerate(s["shape"]):
        k, v = _sequence(case, seed, b, n)
        t = torch.arange(n, device="cuda")
        slots = s["table"][b][t // page] * page + (t % page).int()
        if own:
            W.kv4_append(torch.cat([k.view(n, g * d), v.view(n, g * d)], dim=1), s["cache"], slots, heads=0)
        else:
            _plain_store(s["cache"], slots, k, v)
    s["max_queries"] = max(q for q, _ in s["shape"])
    return s


# ---------------------------------------------------------------------------------- plain forms
def _plain_cache(tokens, g, d):
    out = {}
    for x in ("k", "v"):
        out[x] = torch.zeros((tokens, g, d // 2), dtype=torch.uint8, device="cuda")
        out[x + "_scale"] = torch.zeros((tokens, g, d // GROUP, 2), dtype=torch.float16, device="cuda")
    return out


def _plain_store(cache, slots, k, v):
    """x = min + code * scale, codes 0..15, one fp16 (scale, min) for each 64 elements; decided in 32 bits."""
    at = slots.long()
    for name, x in (("k", k), ("v", v)):
        f = x.float().unflatten(-1, (-1, GROUP))
        low, high = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
        scale = ((high - low) / 15.0).half()
        div = scale.float()
        code = torch.where(div > 0, torch.round((f - low) / torch.where(div > 0, div, 1.0)).clamp(0, 15), 0.0)
        code = code.to(torch.uint8).flatten(-2)
        cache[name][at] = code[..., 0::2] | (code[..., 1::2] << 4)
        cache[name + "_scale"][at] = torch.cat([scale, low.half()], dim=-1)


def _plain_values(cache, name, at):
    packed, sm = cache[name][at], cache[name + "_scale"][at].float()
    code = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (code * sm[..., 0:1] + sm[..., 1:2]).flatten(-2)


def _plain_norm(x, weight):
    """x / rms(x) * weight. The squares are added in the order that the operator defines (8 neighbours
    in turn, then pairs of neighbouring sums), since the codes of the cache decide on the result."""
    s = (x * x).unflatten(-1, (-1, 8))
    t = s[..., 0]
    for i in range(1, 8):
        t = t + s[..., i]
    while t.shape[-1] > 1:
        t = t[..., 0::2] + t[..., 1::2]
    return (x * (1.0 / torch.sqrt(t / x.shape[-1] + EPS))) * weight.float()


def _plain_rotate(x, table, pos, adjacent):
    rot = table.shape[1]
    row = table[pos.long()][:, None, :]
    c, s = row[..., : rot // 2], row[..., rot // 2:]
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_append(s):
    case = s["case"]
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    x = s["qkv"].float().unflatten(-1, (h + 2 * g, d))
    q, k, v = x[:, :h], x[:, h:h + g], s["qkv"].unflatten(-1, (h + 2 * g, d))[:, h + g:]
    if s["q_norm"] is not None:
        q, k = _plain_norm(q, s["q_norm"]), _plain_norm(k, s["k_norm"])
    if s["rope"] is not None:
        q, k = (_plain_rotate(t, s["rope"], s["pos"], case["adjacent"]) for t in (q, k))
    _plain_store(s["cache"], s["slots"], k.half(), v)
    at = s["slots"].long()
    return {"q": q.half(), "k": _plain_values(s["cache"], "k", at).half(), "v": _plain_values(s["cache"], "v", at).half()}


def _plain_attention(s):
    case = s["case"]
    h, g, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.empty_like(s["q"])
    at = 0
    for b, (n_q, n) in enumerate(s["shape"]):
        t = torch.arange(n, device="cuda")
        where = s["table"][b].long()[t // page] * page + t % page
        k = _plain_values(s["cache"], "k", where).transpose(0, 1)
        v = _plain_values(s["cache"], "v", where).transpose(0, 1)
        q = s["q"][at:at + n_q].float().unflatten(1, (g, h // g)).transpose(0, 1).reshape(g, n_q * (h // g), d)
        score = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
        last = (n - n_q + torch.arange(n_q, device="cuda")).repeat_interleave(h // g)
        score = torch.where(t[None, :] <= last[:, None], score, float("-inf"))
        p = torch.exp(score - score.amax(-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out[at:at + n_q] = o.view(g, n_q, h // g, d).transpose(0, 1).reshape(n_q, h, d).half()
        at += n_q
    return out


def _scaled(total, numerator24):
    """floor(total * numerator24 / 2^24) for totals below 2^58, in whole numbers of 64 bits."""
    return numerator24 * (total >> 24) + ((numerator24 * (total & 0xFFFFFF)) >> 24)


def _plain_sample(s):
    x = s["logits"].float()
    v = x.shape[1]
    greedy = s["temperature"] <= 0
    temp = torch.where(greedy, 1.0, s["temperature"])[:, None]
    val, idx = torch.sort(torch.where(torch.isnan(x), float("-inf"), x), dim=1, descending=True, stable=True)
    w = torch.where(val == val[:, :1], 1.0, torch.exp((val - val[:, :1]) / temp))
    rank = torch.arange(v, device="cuda")[None, :]
    k = torch.where(greedy, 1, torch.where(s["top_k"] <= 0, v, s["top_k"]))[:, None]
    fixed = torch.where(rank < k, torch.round(w * FIXED), 0.0).to(torch.int64)
    cum = fixed.cumsum(1)
    p24 = (s["top_p"].clamp(0, 1) * 2.0 ** 24).to(torch.int64)[:, None]
    limit = torch.where(s["top_p"][:, None] < 1, _scaled(cum[:, -1:], p24), cum[:, -1:])
    keep = (rank == 0) | ((cum - fixed < limit) & (w >= s["min_p"][:, None]))
    fixed = torch.where(keep, fixed, 0)
    cum = fixed.cumsum(1)
    total = cum[:, -1:]
    u24 = (s["u"] * 2.0 ** 24).to(torch.int64).clamp(0, 2 ** 24 - 1)[:, None]
    at = (cum <= _scaled(total, u24)).sum(1, keepdim=True)
    probs = fixed.gather(1, at).float() / total.float()
    return {"tokens": idx.gather(1, at)[:, 0].int(), "probs": probs[:, 0]}


def run(s):
    case = s["case"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "sample": _plain_sample}[case["op"]](s)
    import w4a16_weight_streaming_gb300 as W
    if case["op"] == "append":
        q = W.kv4_append(s["qkv"], s["cache"], s["slots"], heads=case["heads"], positions=s["pos"] if case["rot"] else None,
                         rope=s["rope"], adjacent=case["adjacent"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        k, v = W.kv4_load(s["cache"], s["slots"])
        return {"q": q, "k": k, "v": v}
    if case["op"] == "attention":
        return W.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["starts"], max_q_len=s["max_queries"],
                               workspace=s["workspace"])
    tokens, probs = W.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                             min_p=s["min_p"])
    return {"tokens": tokens, "probs": probs}


# --------------------------------------------------------------------------- the same in 64 bits
def _stored_values64(x):
    """What 4-bit storage makes of fp16 x [n, heads, dim], the decisions in binary32 as defined."""
    n, g, d = x.shape
    f = x.to(torch.float32).reshape(n * g * (d // GROUP), GROUP)
    low = f.min(dim=1).values
    step = ((f.max(dim=1).values - low) / 15.0).to(torch.float16).to(torch.float32)
    flat = step == 0
    code = ((f - low[:, None]) / step.masked_fill(flat, 1.0)[:, None]).round().clamp(max=15.0)
    code[flat] = 0.0
    return (code.double() * step.double()[:, None] + low.double()[:, None]).reshape(n, g, d)


def _exact_append(case, seed):
    inp = _append_inputs(case, seed)
    m, h, g, d, rot = case["rows"], case["heads"], case["kv_heads"], case["dim"], case["rot"]
    q = inp["qkv"][:, : h * d].double().reshape(m, h, d)
    if case["norm"]:
        q = q * (q.pow(2).mean(dim=2, keepdim=True) + EPS).rsqrt() * inp["q_norm"].double()
    if rot:
        angles = inp["rope"].double()[inp["pos"].long()]
        i = torch.arange(rot // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + rot // 2)
        z = torch.complex(q[:, :, first], q[:, :, second])
        z = z * torch.complex(angles[:, i], angles[:, i + rot // 2])[:, None, :]
        q = q.clone()
        q[:, :, first], q[:, :, second] = z.real, z.imag
    # The codes of a key are decided on its 32-bit norm and rotation: in 64 bits a key next to a tie
    # gets another code, so the values of the stored keys have no 64-bit counterpart.
    v = _stored_values64(inp["qkv"][:, (h + g) * d:].reshape(m, g, d))
    return {"q": q, "k": None, "v": v}


def _exact_attention(case, seed):
    inp = _attention_inputs(case, seed)
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.empty((inp["q"].shape[0], h, d), dtype=torch.float64, device="cuda")
    start = 0
    for b, (n_q, n) in enumerate(inp["shape"]):
        k, v = (_stored_values64(t) for t in _sequence(case, seed, b, n))
        for head in range(h):
            q = inp["q"][start:start + n_q, head].double()
            score = (q @ k[:, head // (h // g)].T) / math.sqrt(d)
            hidden = torch.ones((n_q, n), dtype=torch.bool, device="cuda").triu(n - n_q + 1)
            out[start:start + n_q, head] = torch.softmax(score.masked_fill(hidden, -math.inf), dim=1) @ v[:, head // (h // g)]
        start += n_q
    return out


def _exact_sample(case, seed):
    inp = _sample_inputs(case, seed)
    m = case["rows"]
    tokens = torch.empty(m, dtype=torch.int64, device="cuda")
    probs = torch.empty(m, dtype=torch.float64, device="cuda")
    for r in range(m):
        val, idx = inp["logits"][r].double().sort(descending=True, stable=True)
        t, k = float(inp["temperature"][r]), int(inp["top_k"][r])
        w = ((val - val[0]) / t).exp() if t > 0 else (torch.arange(len(val), device="cuda") == 0).double()
        w = w[:k] if k > 0 else w
        before = w.cumsum(0) - w
        kept = (w >= float(inp["min_p"][r]))
        if float(inp["top_p"][r]) < 1:
            kept &= before < float(inp["top_p"][r]) * w.sum()
        kept[0] = True
        w = w[kept]
        j = int((w.cumsum(0) <= float(inp["u"][r]) * w.sum()).sum().clamp(max=len(w) - 1))
        tokens[r], probs[r] = idx[j], w[j] / w.sum()
    # A draw among thousands of kept tokens lands so near a boundary now and then that 32-bit weights
    # and 64-bit ones name neighbours; only a draw among few has a 64-bit answer. A neighbour's
    # probability is the same to that accuracy.
    few = not case["mixed"] and 0 < case["top_k"] <= 100
    return {"tokens": tokens if few else None, "probs": probs}


def exact(case, seed):
    with torch.no_grad():
        return {"append": _exact_append, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](case, seed)
