"""Plain statements of the paged 4-bit cache, attention over it and token sampling, for the tests.

`store` / `append` follow the definition in binary32 step by step (numpy float32 operations are IEEE and
unfused), so codes and queries are compared bit for bit; `attention` and `sample` are in 64 bits."""
from __future__ import annotations

import numpy as np

F32, F16 = np.float32, np.float16


def store(x: np.ndarray) -> np.ndarray:
    """float64 values that 4-bit storage makes of fp16 x [..., D] (groups of 64)."""
    f = x.astype(F16).astype(F32).reshape(x.shape[:-1] + (x.shape[-1] // 64, 64))
    lo, hi = f.min(-1, keepdims=True), f.max(-1, keepdims=True)
    scale = ((hi - lo) / F32(15)).astype(F16).astype(F32)
    div = np.where(scale > 0, scale, F32(1))
    code = np.where(scale > 0, np.clip(np.rint((f - lo) / div), 0, 15), 0)
    return (lo.astype(np.float64) + code.astype(np.float64) * scale.astype(np.float64)).reshape(x.shape)


def norm(x: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    """fp32 x [..., D]: the squares of 8 neighbours in turn, then neighbouring sums in pairs."""
    sq = (x * x).reshape(x.shape[:-1] + (-1, 8))
    t = sq[..., 0]
    for i in range(1, 8):
        t = t + sq[..., i]
    while t.shape[-1] > 1:
        t = t[..., 0::2] + t[..., 1::2]
    inv = F32(1) / np.sqrt(t / F32(x.shape[-1]) + F32(eps))
    return (x * inv) * w.astype(F32)


def rotate(x: np.ndarray, table: np.ndarray, pos: np.ndarray, adjacent: bool) -> np.ndarray:
    """fp32 x [M, heads, D]."""
    rot = table.shape[1]
    c, s = table[pos][:, None, : rot // 2], table[pos][:, None, rot // 2:]
    y = x.copy()
    ia, ib = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def append(qkv, heads, kv_heads, D, rope=None, pos=None, adjacent=False, q_norm=None, k_norm=None, eps=1e-6):
    """(q fp16, stored keys float64, stored values float64) of fp16 rows qkv [M, (heads + 2 kv_heads) D]."""
    x = qkv.reshape(qkv.shape[0], -1, D)
    q, k, v = x[:, :heads].astype(F32), x[:, heads:heads + kv_heads].astype(F32), x[:, heads + kv_heads:]
    if q_norm is not None:
        q = norm(q, q_norm, eps)
    if k_norm is not None:
        k = norm(k, k_norm, eps)
    if rope is not None:
        q, k = rotate(q, rope, pos, adjacent), rotate(k, rope, pos, adjacent)
    return q.astype(F16), store(k.astype(F16)), store(v)


def attention(q, keys, values, q_lens, scale, causal=True):
    """q fp16 [M, H, D]; keys, values: one float64 [n, KV, D] a sequence. Returns (out, lse, bound):
    bound is what rounding may do to out. Scores from fp16 roundings of k' are off by at most
    e = 2^-11 scale sum|q k'| (+ 2^-20 for the exponential), the products p v' by 2^-10 (two fp16 roundings
    a term), the sums and the division by far less, the result is rounded to fp16 once."""
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    bound = np.zeros(q.shape)
    at = 0
    for n_q, k, v in zip(q_lens, keys, values):
        n, grp = k.shape[0], q.shape[1] // k.shape[1]
        for i in range(n_q):
            see = n - n_q + i + 1 if causal else n
            if see <= 0:
                continue
            for h in range(q.shape[1]):
                x = q[at + i, h].astype(np.float64)
                kk, vv = k[:see, h // grp], v[:see, h // grp]
                s = scale * (kk @ x)
                e = (2.0 ** -11 * abs(scale) * (np.abs(kk) @ np.abs(x))).max() + 2.0 ** -20
                p = np.exp(s - s.max())
                z = p.sum()
                o = (p @ vv) / z
                a = (p @ np.abs(vv)) / z
                out[at + i, h] = o
                lse[at + i, h] = s.max() + np.log(z)
                bound[at + i, h] = 2.0 ** -10 * np.abs(o) + (2.0 ** -10 + 2.0 * e) * a + 2.0 ** -24
        at += n_q
    return out, lse, bound


class Sampled:
    """What one row's draw may be, in 64 bits: check(token, prob) says whether it is one of the answers
    that 32-bit weights may give. A weight is off by at most (2 |x| + 4) 2^-24 of itself, x = (l - l_max)/T
    (the rounding of x and the exponential), |x| <= 28.5 where the weight is not 0: 4e-6; a mass of the
    distribution by as much, plus half of 2^-40 a token, plus 2^-24 for each of u and top_p."""

    TOL = 1.0e-5

    def __init__(self, logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
        x = logits.astype(np.float64)
        x[np.isnan(x)] = -np.inf
        self.order = np.lexsort((np.arange(len(x)), -x))
        s = x[self.order]
        n = int((s > -np.inf).sum())
        self.n, self.u = n, u
        if n == 0:
            return
        t = temperature if temperature > 0 else 1.0
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.where(s == s[0], 1.0, np.exp((s - s[0]) / t))
        k = 1 if temperature <= 0 else top_k
        if 0 < k < n:
            w[k:] = 0
        w[n:] = 0
        w[w < 2.0 ** -41] = 0
        before = np.cumsum(w) - w
        total = w.sum()
        keep = w >= min_p if min_p > 0 else w > 0
        # tokens within rounding of a cut: kept or not, and as much of the distribution is open
        either = (w != min_p) & (np.abs(w - min_p) <= self.TOL * min_p) if min_p > 0 else np.zeros(len(w), bool)
        if top_p < 1:
            keep &= before < top_p * total
            either |= np.abs(before - top_p * total) <= self.TOL * total
        keep[0], either[0] = True, False
        self.either = either & (w > 0)
        self.w = np.where(keep, w, 0)
        self.slack = self.TOL + w[self.either].sum() / self.w.sum()
        self.cdf = np.cumsum(self.w) / self.w.sum()
        self.kept = int(keep.sum())

    def check(self, token, prob):
        if self.n == 0:
            return token == -1 and prob == 0
        i = int(np.nonzero(self.order == token)[0][0])
        if self.either[i] and self.w[i] == 0:
            return self.u >= 1 - self.slack
        p = self.w[i] / self.w.sum()
        low = self.cdf[i] - p
        return self.w[i] > 0 and low - self.slack <= self.u <= self.cdf[i] + self.slack and \
            abs(prob - p) <= self.slack * p + 1e-12


def rounded(x, bits):
    """x to `bits` significant bits, to nearest even."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


class Pairs:
    """Sequences of two tokens, in which a rounding of keys, values or weights shows: nothing averages it out.
    kind "weights": keys are one number each, so scores are exact; "keys": all but two elements of a group of 64
    are 7 steps of a full-width scale above 0, so that a rounding of k' is the same in all of them. Queries are
    1 (a key head's `group` query heads alike)."""

    D, SCALE = 128, 1.0 / 32

    def __init__(self, kind, seed, B=96):
        rng = np.random.default_rng(seed)
        k = np.zeros((B, 2, self.D), F16)
        if kind == "weights":
            k[:, 1] = (rng.integers(4, 64, (B, 1)) / 64).astype(F16)
        else:
            scale = (rng.integers(1024, 2048, (B, 2)) / 2048).astype(F16)  # 11 significant bits
            scale[:, 1] = (scale[:, 0].astype(np.float64) * (1 + rng.normal(size=B) / 64)).astype(F16)
            k[..., 1::64] = (15 * scale.astype(np.float64)).astype(F16)[..., None]
            # 7 steps of the scale that storage takes from a group's ends, 0 and its largest element
            step = (k[..., 1].astype(F32) / F32(15)).astype(F16).astype(np.float64)
            k[..., 2:64] = k[..., 66:128] = (7 * step).astype(F16)[..., None]
        v = (rng.normal(size=(B, 2, self.D)) + rng.normal(size=(B, 1, self.D))).astype(F16)
        self.k16, self.v16 = k, v
        self.k, self.v = store(k), store(v)
        g = self.v.reshape(B, 2, -1, 64)
        self.low = np.broadcast_to(g.min(-1, keepdims=True), g.shape).reshape(self.v.shape)
        size = np.abs(g.min(-1, keepdims=True)) + 1.01 * (g.max(-1, keepdims=True) - g.min(-1, keepdims=True))
        self.p = self.weights(self.k)
        self.want = self.mean(self.p, self.v)
        plain, size = self.mean(self.p, np.abs(self.v)), self.mean(self.p, np.broadcast_to(size, g.shape).reshape(self.v.shape))
        # what one rounding to fp16 of the output and of k', v' and the weights each may do (2^-11 of each; a score's
        # error moves the output by no more than twice itself), and what the decode kernel's two numbers leave
        e = self.SCALE * 2.0 ** -11 * np.abs(self.k).sum(-1).max(-1)[:, None] if kind == "keys" else 0.0
        self.many = 2.0 ** -11 * np.abs(self.want) + 2.0 ** -25 + (2.0 ** -10 + 2 * e + 2.0 ** -18) * plain
        self.one = 2.0 ** -11 * np.abs(self.want) + 2.0 ** -25 + 2.0 ** -16 * size

    def weights(self, k):
        s = self.SCALE * k.sum(-1)
        return np.exp(s - s.max(-1, keepdims=True))

    def mean(self, p, v, total=None):
        return (p[..., None] * v).sum(1) / (p if total is None else total).sum(1)[:, None]

    def many_with(self, keys, values, weights):
        """The output of a kernel for many rows that rounds k', v' and the weights to so many bits."""
        p = self.weights(rounded(self.k, keys))
        return self.mean(rounded(p, weights), rounded(self.v, values), p).astype(F16).astype(np.float64)

    def one_with(self, bits):
        """The output of a kernel that rounds weights times scales to so many bits, beside the minimums in full."""
        step = np.maximum(self.v - self.low, 0)
        return (self.mean(self.p, self.low) + self.mean(rounded(self.p, bits), step)).astype(F16).astype(np.float64) \
            if bits < 24 else self.want.astype(F16).astype(np.float64)
