"""logprobs against 64 bits. Tokens and ranks are whole numbers and have to be equal.

Bounds: a weight's exponent (l - l_max) / T is off by 2^-23 of itself and its exponential by 2^-22, so S, of weights
that matter (exponents down to -20 or so), by less than 2^-18 with the roundings of its sum; log S by as much, a log
probability by that and 2^-22 of itself; the entropy, which adds sum w d / S, by twice that."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    return lib()


def peaked(rng, M, V, std=2.0):
    x = std * rng.normal(size=(M, V))
    x[np.arange(M)[:, None], rng.integers(0, V, (M, 12))] += 6 + 3 * rng.normal(size=(M, 12))
    return x.astype(np.float16)


def reference(l, tokens, top, temp):
    l = l.astype(np.float64)
    masked = np.isnan(l) | (l == -np.inf)
    V = len(l)
    key = np.where(masked, -np.inf, l)
    order = np.argsort(-key, kind="stable")
    order = order[~masked[order]]
    place = np.zeros(V, np.int64)
    place[order] = np.arange(1, len(order) + 1)
    t = temp if temp > 0 else 1.0
    if len(order) == 0:
        return (np.where(tokens < 0, 0.0, -np.inf), place[tokens] * (tokens >= 0), 0.0, np.full(top, -1), np.full(top, -np.inf))
    m = key[order[0]]
    with np.errstate(all="ignore"):
        d = np.where(masked, -np.inf, np.where(key == m, 0.0, (key - m) / t))
        if np.isinf(m):
            d = np.where(key == m, 0.0, -np.inf)
        w = np.exp(d)
        lp = d - np.log(w.sum())
        p = w / w.sum()
        entropy = -np.where(p > 0, p * lp, 0.0).sum()
    best = order[:top]
    fill = top - len(best)
    return (np.where(tokens < 0, 0.0, lp[tokens]), np.where(tokens < 0, 0, place[tokens]), entropy,
            np.concatenate([best, np.full(fill, -1)]), np.concatenate([lp[best], np.full(fill, -np.inf)]))


def close(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    with np.errstate(invalid="ignore"):
        return bool(((a == b) | (np.abs(a - b) <= 2.0 ** -18 + 2.0 ** -21 * np.abs(b))).all())


def check(W, x, tokens=None, top=0, temperature=None, rows=None):
    x = x if isinstance(x, torch.Tensor) else torch.from_numpy(x).cuda()
    M = x.shape[0]
    r = W.logprobs(x, None if tokens is None else torch.from_numpy(np.asarray(tokens, np.int32)).cuda(), top,
                   None if temperature is None else torch.from_numpy(np.asarray(temperature, np.float32)).cuda())
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.OK
    h = x.cpu().numpy()
    for i in range(M) if rows is None else rows:
        tok = np.asarray(tokens[i]).reshape(-1) if tokens is not None else np.zeros(0, np.int64)
        lp, rank, entropy, best, best_lp = reference(h[i], tok, top, 1.0 if temperature is None else float(np.float32(temperature[i])))
        if tokens is not None:
            assert np.array_equal(r.rank[i].cpu().numpy().reshape(-1), rank), (i, r.rank[i], rank)
            assert close(r.logprob[i].cpu().numpy().reshape(-1), lp), (i, r.logprob[i], lp)
        assert close(r.entropy[i].item() / 2, entropy / 2), (i, r.entropy[i], entropy)
        if top:
            assert np.array_equal(r.top_tokens[i].cpu().numpy(), best), (i, r.top_tokens[i], best)
            assert close(r.top_logprob[i].cpu().numpy(), best_lp), (i, r.top_logprob[i], best_lp)
    return r


@pytest.mark.parametrize("top", [0, 1, 5, 32])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 7), (2, 8), (4, 33), (1, 1000), (5, 8193), (12, 32003), (40, 777), (200, 5001)])
def test_sizes(W, M, V, top):
    rng = np.random.default_rng(M * V + top)
    x = peaked(rng, M, V)
    for given in (0, 1, 2, 3, 8):
        check(W, x, rng.integers(0, V, (M, given)) if given else None, top)
    check(W, x, rng.integers(0, V, M), top, 0.3 + 2 * rng.random(M))


def test_the_whole_output_head(W):
    rng = np.random.default_rng(1)
    x = peaked(rng, 3, 248320)
    check(W, x, x.argmax(1)[:, None] + np.array([[0, -5]]), 20)
    check(W, x[:1], rng.integers(0, 248320, (1, 1)), 32, [0.7])


@pytest.mark.parametrize("M", [1, 40, 90, 160])  # clusters of 16, 2, 1 CTAs
@pytest.mark.parametrize("V", [65537, 262113, 1000000])
def test_long_rows(W, M, V):
    g = torch.Generator("cuda").manual_seed(V + M)
    x = torch.randn((M, V), generator=g, device="cuda").half()
    x[:, ::3] = 1.5  # a third of the tokens share a value
    tokens = np.random.default_rng(V).integers(0, V, (M, 2))
    check(W, x, tokens, 7, rows=[0, M // 2, M - 1])


@pytest.mark.parametrize("V", [1, 7, 40, 4096, 65537])
def test_equal_logits(W, V):
    x = np.full((4, V), np.float16(-3.5))
    x[1] = 65504
    x[2] = -65504
    x[3, ::2], x[3, 1::2] = 0.0, np.float16(-0.0)
    top = min(32, V + 3)
    t = np.stack([np.array([0, V - 1, V // 2])] * 4)
    r = check(W, x, t, top)
    assert r.rank[:, 1].tolist() == [V] * 4


@pytest.mark.parametrize("M", [2, 170])
def test_masked_and_infinite_logits(W, M):
    rng = np.random.default_rng(2)
    V = 9001
    x = peaked(rng, M, V)
    kind = np.arange(M) % 9
    x[kind == 0] = -np.inf
    x[kind == 1] = np.nan
    x[kind == 2, 5:] = -np.inf                      # 5 left, top 8
    x[(kind == 3)[:, None] & (rng.random((M, V)) < 0.5)] = -np.inf
    x[(kind == 4)[:, None] & (rng.random((M, V)) < 0.01)] = np.nan
    x[(kind == 5)[:, None] & (rng.random((M, V)) < 0.001)] = np.inf
    x[kind == 6] = -65504
    x[kind == 6, 77] = -np.inf                       # masked among the lowest finite ones
    x[(kind == 7), 3000:] = -65504
    x[kind == 8, :-1] = -np.inf                      # the very last token alone
    t = rng.integers(0, V, (M, 4))
    t[:, 0], t[:, 1] = 77, -1
    for top in (0, 8):
        check(W, x, t, top)
        check(W, x, t, top, 0.1 + 3 * rng.random(M))
        check(W, x, t, top, np.full(M, np.inf))


def test_temperatures(W):
    rng = np.random.default_rng(3)
    temp = np.array([1.0, 0.0, -1.0, np.nan, np.inf, 1e30, 50.0, 0.02, 1e-3, 1e-30])
    x = peaked(rng, len(temp), 3001)
    x[-1, 17] = x[-1].max()  # two equal largest ones
    check(W, x, rng.integers(0, 3001, (len(temp), 2)), 4, temp, rows=range(9))
    r = W.logprobs(torch.from_numpy(x).cuda(), top=3, temperature=torch.from_numpy(temp.astype(np.float32)).cuda())
    both = (x[-1] == x[-1].max()).sum()
    assert np.allclose(r.top_logprob[-1, :2].cpu(), -np.log(both)) and abs(r.entropy[-1].item() - np.log(both)) < 1e-5


def test_tokens_outside(W):
    x = torch.randn((3, 100), device="cuda").half()
    t = torch.tensor([[-1, 3], [-2 ** 31, 99], [5, 0]], dtype=torch.int32, device="cuda")
    r = W.logprobs(x, t)
    assert r.rank[:2, 0].tolist() == [0, 0] and r.logprob[:2, 0].tolist() == [0, 0] and W.w4a16_device_status() == W.OK
    t[2, 0] = 100
    s = W.logprobs(x, t)
    assert W.w4a16_device_status() == W.ERR_BOUNDS and W.w4a16_device_status() == W.OK
    assert s.rank[2, 0].item() == 0 and torch.equal(s.rank[:, 1], r.rank[:, 1])


@pytest.mark.parametrize("shift", [0, 1, 3, 7])
def test_rows_of_any_alignment(W, shift):
    rng = np.random.default_rng(4)
    M, V = 21, 1013
    wide = torch.full((M, V + 16), 60000.0, dtype=torch.float16, device="cuda")
    x = peaked(rng, M, V)
    wide[:, shift:shift + V] = torch.from_numpy(x).cuda()
    t = rng.integers(0, V, (M, 3))
    t[0] = [0, V - 1, 8 - shift]
    check(W, wide[:, shift:shift + V], t, 9)
    check(W, wide[:1, shift:shift + V], t[:1], 9)


@pytest.mark.parametrize("order", ["ascending", "descending", "one_group_low", "blocks"])
def test_rows_made_against_the_search(W, order):
    """Many chunk maxima above the bound that the groups of threads give: the list overflows and is cut again."""
    M, V = 160, 131072
    i = np.arange(V)
    chunk = i // 32
    v = {"ascending": i / 2048.0, "descending": -i / 2048.0,
         "one_group_low": np.where(chunk % 256 >= 248, -20.0, 5 + (chunk % 7) / 8),
         "blocks": np.where(chunk % 256 < 8, (chunk % 97) / 4.0, -30.0 - chunk % 3)}[order].astype(np.float16)
    x = torch.from_numpy(np.repeat(v[None], M, 0)).cuda()
    check(W, x, np.full((M, 1), V // 2), 32, rows=[0, M - 1])
    check(W, x[:2].contiguous(), np.full((2, 1), V // 3), 31)


def test_replay_streams_and_given_outputs(W):
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((6, 40000), generator=g, device="cuda").half()
    t = torch.randint(0, 40000, (6,), generator=g, device="cuda").int()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    W.logprobs(x, t, top=4, stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = W.logprobs(x, t, top=4)
    x.copy_(x.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    fresh = W.logprobs(x, t, top=4)
    out = W.LogProbs(None, torch.empty_like(fresh.rank), torch.empty_like(fresh.entropy), torch.empty_like(fresh.top_tokens),
                     torch.empty_like(fresh.top_logprob))
    assert W.logprobs(x, t, top=4, out=out) is out
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, fresh))
    assert all(a is None or torch.equal(a, b) for a, b in zip(out, fresh))
    greedy, _ = W.sample(x, torch.zeros(6, device="cuda"), temperature=torch.zeros(6, device="cuda"))
    assert torch.equal(greedy, fresh.top_tokens[:, 0])


def test_the_index_checking_build_gives_the_same(W):
    D = W.load_debug_bounds()
    rng = np.random.default_rng(8)
    x = torch.from_numpy(peaked(rng, 4, 30001)).cuda()
    t = torch.tensor([[5, 77], [1, 30000], [3, 4], [9, 9]], dtype=torch.int32, device="cuda")
    want = W.logprobs(x, t, top=6)
    got = W.LogProbs(*(torch.empty_like(v) for v in want))
    s = torch.cuda.current_stream().cuda_stream
    assert D.w4a16_logprobs(x.data_ptr(), 30001, 4, 30001, t.data_ptr(), 2, 6, None, *(v.data_ptr() for v in got), s) == 0
    torch.cuda.synchronize()
    assert D.w4a16_device_status(s) == W.OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_further_apart_than_32_bits(W):
    V, step = 5003, 2 ** 31 + 7
    wide = torch.zeros(2 * step + V, dtype=torch.float16, device="cuda")
    x = wide.as_strided((3, V), (step, 1))
    rng = np.random.default_rng(11)
    x.copy_(torch.from_numpy(peaked(rng, 3, V)).cuda())
    check(W, x, rng.integers(0, V, (3, 2)), 6)


def test_many_rows(W):
    g = torch.Generator("cuda").manual_seed(12)
    x = (3 * torch.randn((65536, 300), generator=g, device="cuda")).half()
    t = torch.randint(0, 300, (65536, 1), generator=g, device="cuda").int()
    r = W.logprobs(x, t, top=2)
    torch.cuda.synchronize()
    lp = torch.log_softmax(x.double(), 1)
    assert float((r.logprob.double() - lp.gather(1, t.long())).abs().max()) < 1e-5
    best = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(r.top_tokens.long(), best)
    at = x.gather(1, t.long())
    index = torch.arange(300, device="cuda")[None]
    assert torch.equal(r.rank[:, 0].long(), 1 + ((x > at) | ((x == at) & (index < t))).sum(1))
    assert float((r.entropy.double() + (lp.exp() * lp).sum(1)).abs().max()) < 1e-5


def test_two_host_threads(W):
    """Calls of one kernel with much and with little shared memory, at the same time."""
    import threading

    rows = {v: torch.randn((320, v), device="cuda").half() for v in (1000000, 1000)}
    wanted = {v: W.logprobs(x, top=3) for v, x in rows.items()}
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(v):
        try:
            s = torch.cuda.Stream()
            for _ in range(100 if v < 10000 else 25):
                got[v] = W.logprobs(rows[v], top=3, stream=s)
            s.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(v,)) for v in rows]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for v in rows:
        assert torch.equal(got[v].top_tokens, wanted[v].top_tokens) and torch.equal(got[v].entropy, wanted[v].entropy)


@pytest.mark.parametrize("M", [3, 700])
@pytest.mark.parametrize("temperature", [0.0001, 0.0901, 0.0902, 0.5, 1.0, 20.0, 32.0, 150.0])
def test_logits_far_from_zero(W, temperature, M):
    """l / T up to millions, of which the differences are what counts: 60000 / 32 in fp32 is off by 2^-14 or so."""
    rng = np.random.default_rng(15)
    V = 4099
    x = np.empty((M, V), np.float16)
    x[0::3] = 60000 - 32.0 * rng.integers(0, 40, (len(x[0::3]), V))
    x[1::3] = -33000 - 32.0 * rng.integers(0, 40, (len(x[1::3]), V))
    x[2::3] = 2000 + 1.0 * rng.integers(0, 40, (len(x[2::3]), V))
    check(W, x, rng.integers(0, V, (M, 2)), 5, [temperature] * M, rows=range(min(M, 9)))


def test_rows_of_rising_logits(W):
    """Every step brings a new largest one."""
    x = torch.linspace(-40, 40, 40000, device="cuda").half().repeat(3, 1)
    x[1] = x[1].flip(0)
    x[2] = -65504 + 0.8 * 131008 * torch.linspace(0, 1, 40000, device="cuda")
    t = np.array([[0, 39999, 20000]] * 3)
    check(W, x, t, 8, [1.0, 0.8, 300.0])
    check(W, x.repeat(250, 1), np.tile(t, (250, 1)), 8, [1.0, 0.8, 300.0] * 250, rows=[0, 1, 2, 749])


def listed_maxima(row, threads, parts, top):
    """How many maxima of chunks of 32 each CTA of a row lists at first: those not below the top-th largest of its
    threads' largest ones (a row on a 64-byte boundary; chunk i of a CTA is thread i % threads')."""
    chunks = row.astype(np.float64).reshape(-1, 32).max(1)
    per, counts = -(-len(chunks) // parts), []
    for part in range(parts):
        own = chunks[part * per:(part + 1) * per]
        place = np.empty(len(own), np.int64)
        place[np.argsort(-own, kind="stable")] = np.arange(len(own))
        counts.append(int(np.sort([place[t::threads].min() for t in range(threads)])[top - 1]) + 1)
    return counts


@pytest.mark.parametrize("M,V,threads,parts", [(160, 1000000, 256, 1), (90, 1000000, 256, 2), (700, 248320, 128, 1)])
@pytest.mark.parametrize("top", [32, 27])
def test_rows_with_more_maxima_than_the_list_holds(W, M, V, threads, parts, top):
    """top - 1 threads own every high chunk, so that the bound is a low one's and thousands of maxima pass it; the list of
    1024 is filled and cut again, once or (values rising along the row) several times."""
    chunk = np.arange(V // 32)
    own = chunk % -(-len(chunk) // parts)  # within its CTA's part
    high = own % threads < top - 1
    n = np.cumsum(high)
    rng = np.random.default_rng(V + top)
    values = [8 + (n * 7919 % 1021) / 128, np.full(len(chunk), 12.5), 8 + 24 * n / n[-1], 32 - 24 * n / n[-1], np.where(n % 9 == 4, 20.0, 11 + (n % 4) / 4)]
    rows = np.empty((len(values), V), np.float16)
    for i, v in enumerate(values):
        x = rng.normal(size=(len(chunk), 32)) - 4
        x[high] = v[high, None] - 0.25 * rng.integers(0, 5, (high.sum(), 32))
        x[high, rng.integers(0, 32, high.sum())] = v[high]
        rows[i] = x.reshape(-1)
        assert min(listed_maxima(rows[i], threads, parts, top)) > 1024
    which = np.arange(M) % len(values)
    x = torch.from_numpy(rows).cuda()[torch.from_numpy(which).cuda()]
    tokens = rng.integers(0, V, (M, 2))
    tokens[:, 0] = 32 * np.flatnonzero(high)[rng.integers(0, high.sum(), M)]
    check(W, x, tokens, top, rows=[0, 1, 2, 3, 4, M - 1])
