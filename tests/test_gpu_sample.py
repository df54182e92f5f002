"""Token sampling on the GPU. Where weights are equal (one value, masks, greedy rows) the answer is a whole
number and compared as such; elsewhere a 64-bit statement says which tokens 32-bit weights may give."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import lib
from kv4_ref import Sampled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    return lib()


def cuda(x):
    return torch.from_numpy(np.array(x)).cuda()


def draw(W, logits, u, **kw):
    M = logits.shape[0]
    t = {}
    for name, dtype in (("temperature", np.float32), ("top_k", np.int32), ("top_p", np.float32), ("min_p", np.float32)):
        if name in kw:
            t[name] = cuda(np.broadcast_to(np.asarray(kw[name], dtype), (M,)))
    x = logits if isinstance(logits, torch.Tensor) else cuda(logits)
    tokens, probs = W.sample(x, cuda(np.asarray(u, np.float32)), **t)
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.OK
    return tokens.cpu().numpy(), probs.cpu().numpy()


def peaked(rng, M, V, std=2.0):
    x = std * rng.normal(size=(M, V))
    x[np.arange(M)[:, None], rng.integers(0, V, (M, 12))] += 6 + 3 * rng.normal(size=(M, 12))
    return x.astype(np.float16)


SETTINGS = [dict(), dict(temperature=0.6, top_k=20, top_p=0.95), dict(temperature=1.3, top_p=0.8), dict(min_p=0.05),
            dict(temperature=0.7, top_k=50, min_p=0.02), dict(top_k=1000, top_p=0.5, min_p=0.001), dict(top_k=3),
            dict(temperature=5.0), dict(top_p=0.01), dict(top_p=0.0), dict(min_p=1.0), dict(min_p=2.0),
            dict(top_k=10 ** 9, top_p=1.0, min_p=0.0), dict(top_k=400), dict(top_k=700, top_p=0.9), dict(top_k=6000, top_p=0.99),
            dict(temperature=50.0), dict(temperature=50.0, top_p=0.7), dict(temperature=0.02), dict(temperature=3.0, min_p=1e-6),
            dict(temperature=50.0, min_p=0.9), dict(top_k=5, min_p=1e-9), dict(temperature=1e30), dict(temperature=np.inf),
            dict(temperature=np.inf, top_p=0.6), dict(temperature=1e-44, top_p=0.9)]


@pytest.mark.parametrize("kw", SETTINGS, ids=[str(i) for i in range(len(SETTINGS))])
@pytest.mark.parametrize("M,V", [(1, 1000), (5, 32003), (12, 5001), (40, 777)])
def test_tokens_are_what_64_bits_allow(W, M, V, kw):
    rng = np.random.default_rng(M * V)
    x = peaked(rng, M, V)
    u = rng.random(M).astype(np.float32)
    u[0] = 0.0
    u[-1] = np.float32(1 - 2.0 ** -24)
    tokens, probs = draw(W, x, u, **kw)
    for r in range(M):
        s = Sampled(x[r], float(u[r]), **kw)
        assert s.check(tokens[r], probs[r]), (r, tokens[r], probs[r], s.kept)


def test_the_whole_output_head(W):
    rng = np.random.default_rng(1)
    x = peaked(rng, 3, 248320)
    u = rng.random(3).astype(np.float32)
    tokens, probs = draw(W, x, u, temperature=0.8, top_p=0.95)
    for r in range(3):
        s = Sampled(x[r], float(u[r]), temperature=0.8, top_p=0.95)
        assert s.check(tokens[r], probs[r])


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 4096, 65537, 1000000])
def test_equal_logits_are_drawn_uniformly_by_index(W, V):
    M = 6
    u = np.array([0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.123456], np.float32)
    x = np.full((M, V), np.float16(-3.5))
    u24 = np.floor(u.astype(np.float64) * 2 ** 24).astype(np.int64)
    tokens, probs = draw(W, x, u)
    # running mass (j + 1) 2^40 exceeds floor(V 2^40 u24 / 2^24) = V u24 2^16 first at j = floor(V u24 / 2^24)
    assert np.array_equal(tokens, (u24 * V) >> 24)
    assert np.allclose(probs, 1 / V, rtol=2e-7)
    k = max(1, V // 3)
    tokens, probs = draw(W, x, u, top_k=k)  # ties: the k lowest indices
    assert np.array_equal(tokens, (u24 * k) >> 24) and np.allclose(probs, 1 / k, rtol=2e-7)
    n = -(-V // 2)  # tokens whose preceding mass is below half of V
    tokens, probs = draw(W, x, u, top_p=0.5)
    assert np.array_equal(tokens, (u24 * n) >> 24) and np.allclose(probs, 1 / n, rtol=2e-7)


def test_masked_logits_are_never_chosen(W):
    rng = np.random.default_rng(2)
    M, V = 8, 3000
    x = np.full((M, V), -np.inf, np.float16)
    allowed = [np.sort(rng.choice(V, n, replace=False)) for n in (1, 2, 5, 100, 2999, 7, 1, 0)]
    for r, a in enumerate(allowed):
        x[r, a] = np.float16(2.0)
    x[5, :50] = np.nan
    allowed[5] = np.array([i for i in allowed[5] if i >= 50], np.int64)
    u = rng.random(M).astype(np.float32)
    tokens, probs = draw(W, x, u)
    for r, a in enumerate(allowed):
        if len(a) == 0:
            assert tokens[r] == -1 and probs[r] == 0
        else:
            assert tokens[r] == a[int(np.floor(float(u[r]) * 2 ** 24)) * len(a) >> 24]
    tokens, probs = draw(W, np.full((2, 100), np.nan, np.float16), [0.5, 0.1], top_p=0.5, temperature=0.0)
    assert (tokens == -1).all() and (probs == 0).all()


def test_greedy_takes_the_first_of_the_largest(W):
    rng = np.random.default_rng(3)
    x = rng.integers(-20, 20, size=(30, 5000)).astype(np.float16)
    tokens, probs = draw(W, x, rng.random(30), temperature=0.0, top_p=0.3, min_p=0.5)
    assert np.array_equal(tokens, x.argmax(1)) and (probs == 1).all()
    tokens, _ = draw(W, -x, rng.random(30), top_k=1)
    assert np.array_equal(tokens, (-x).argmax(1))


def test_infinite_and_extreme_logits(W):
    x = np.zeros((4, 600), np.float16)
    x[0, 17] = x[0, 400] = np.inf       # the two infinite ones share everything
    x[1] = 65504
    x[1, 0] = -65504
    x[2, 5] = np.float16(-0.0)           # -0 and 0 are one value
    x[3] = np.float16(-65504)
    tokens, probs = draw(W, x, [0.7, 0.0, 5.5 / 600, 0.999])
    assert tokens.tolist() == [400, 1, 5, int(np.floor(np.float32(0.999) * 2 ** 24)) * 600 >> 24]
    assert np.allclose(probs, [0.5, 1 / 599, 1 / 600, 1 / 600], rtol=2e-7)


@pytest.mark.parametrize("shift", [0, 1, 3, 7])
def test_rows_of_any_alignment(W, shift):
    rng = np.random.default_rng(4)
    M, V = 21, 1013
    wide = torch.full((M, V + 16), 60000.0, dtype=torch.float16, device="cuda")
    x = peaked(rng, M, V)
    wide[:, shift:shift + V] = cuda(x)
    u = rng.random(M)
    part = draw(W, wide[:, shift:shift + V], u, top_k=40)
    whole = draw(W, x, u, top_k=40)
    assert np.array_equal(part[0], whole[0]) and np.array_equal(part[1], whole[1])


def test_settings_of_each_row_and_the_batch_do_not_matter_to_another(W):
    rng = np.random.default_rng(5)
    M, V = 33, 9001
    x = peaked(rng, M, V)
    u = rng.random(M).astype(np.float32)
    t = np.where(np.arange(M) % 4 == 0, 0, 0.5 + rng.random(M)).astype(np.float32)
    k = rng.integers(-1, 60, M).astype(np.int32)
    p = np.where(np.arange(M) % 3 == 0, 1.0, rng.random(M)).astype(np.float32)
    m = np.where(np.arange(M) % 5 == 0, 0.1, 0).astype(np.float32)
    tokens, probs = draw(W, x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    for r in range(M):  # one row alone: spread over more of the GPU, the same answer
        a, b = draw(W, x[r:r + 1], u[r:r + 1], temperature=t[r], top_k=k[r], top_p=p[r], min_p=m[r])
        assert a[0] == tokens[r] and b[0] == probs[r]
        s = Sampled(x[r], float(u[r]), float(t[r]), int(k[r]), float(p[r]), float(m[r]))
        assert s.check(tokens[r], probs[r])


@pytest.mark.parametrize("shape", ["negative", "narrow", "two_levels", "many_top", "steep"])
def test_rows_of_unusual_shape(W, shape):
    rng = np.random.default_rng(9)
    M, V = 7, 40000
    x = {"negative": lambda: -30 + 2 * rng.normal(size=(M, V)),           # every logit below 0
         "narrow": lambda: 1e-3 * rng.normal(size=(M, V)),                # all weights nearly equal
         "two_levels": lambda: np.where(rng.random((M, V)) < 0.5, 3.0, -3.0),
         "many_top": lambda: np.where(rng.random((M, V)) < 0.2, 5.0, rng.normal(size=(M, V))),  # 8000 equal best
         "steep": lambda: -np.arange(V)[None, :] / 500.0 + rng.normal(size=(M, V)) * 1e-2}[shape]().astype(np.float16)
    u = rng.random(M).astype(np.float32)
    for kw in (dict(), dict(top_p=0.6), dict(top_k=37), dict(min_p=0.3), dict(temperature=0.5, top_k=5000, top_p=0.9)):
        tokens, probs = draw(W, x, u, **kw)
        for r in range(M):
            s = Sampled(x[r], float(u[r]), **kw)
            assert s.check(tokens[r], probs[r]), (shape, kw, r, tokens[r], probs[r])


@pytest.mark.parametrize("M", [1, 2, 40, 300])
def test_a_row_does_not_depend_on_the_batch(W, M):
    rng = np.random.default_rng(10)
    V = 50000
    row = peaked(rng, 1, V)
    for kw in (dict(temperature=0.7, top_k=30), dict(top_p=0.9), dict(temperature=2.5), dict(min_p=0.01)):
        one = draw(W, row, [0.37], **kw)
        many = draw(W, np.repeat(row, M, axis=0), [0.37] * M, **kw)
        assert (many[0] == one[0][0]).all() and (many[1] == one[1][0]).all()


def test_uniform_numbers_cover_the_distribution(W):
    # evenly spaced numbers: a token of probability p is drawn n p times, give or take 1
    rng = np.random.default_rng(6)
    n = 2048
    row = peaked(rng, 1, 4000)
    u = (np.arange(n) + 0.5) / n
    tokens, _ = draw(W, np.repeat(row, n, axis=0), u, top_k=30, temperature=0.9)
    s = Sampled(row[0], 0.5, temperature=0.9, top_k=30)
    drawn = np.bincount(tokens, minlength=4000)
    want = np.zeros(4000)
    want[s.order] = s.w / s.w.sum() * n
    assert (np.abs(drawn - want) <= 1.0 + n * 2 * Sampled.TOL).all()


def test_out_of_range_settings_and_numbers(W):
    rng = np.random.default_rng(7)
    x = peaked(rng, 6, 500)
    u = np.array([-1.0, 2.0, np.nan, np.inf, 0.5, 0.5], np.float32)
    tokens, _ = draw(W, x, u, top_k=5, top_p=np.array([1, 1, 1, 1, -2, 7], np.float32))
    order = np.argsort(-x.astype(np.float64), axis=1, kind="stable")
    assert tokens[0] == order[0, 0] and tokens[1] == order[1, 4] and tokens[2] == order[2, 0]
    assert tokens[3] == order[3, 4] and tokens[4] == order[4, 0] and tokens[5] in order[5, :5]


def test_the_index_checking_build_gives_the_same(W):
    D = W.load_debug_bounds()
    rng = np.random.default_rng(8)
    x, u = cuda(peaked(rng, 4, 3001)), cuda(rng.random(4).astype(np.float32))
    tokens, probs = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert D.w4a16_sample(x.data_ptr(), 3001, 4, 3001, None, None, None, None, u.data_ptr(), tokens.data_ptr(),
                          probs.data_ptr(), s) == 0
    torch.cuda.synchronize()
    assert D.w4a16_device_status(s) == W.OK
    a, b = W.sample(x, u)
    assert torch.equal(a, tokens) and torch.equal(b, probs)


@pytest.mark.parametrize("M,V", [(20, 262113), (19, 300000), (10, 600000), (19, 1000000)])
def test_draws_from_below_the_window_of_long_rows(W, M, V):
    """Vocabularies so long that four or eight CTAs a row could not count them in 16 bits, and draws far below
    the largest logit, so that the counting kernel decides. A third of a row's tokens have one value: more than
    65,536 of them, as many in a CTA's slice as it holds in the rows where they lie side by side."""
    rng = np.random.default_rng(V)
    x = np.clip(rng.normal(size=(M, V)), -3, 3).astype(np.float16) - np.float16(40)
    for r in range(M):
        if r % 2:
            x[r, rng.choice(V, V // 3, replace=False)] = np.float16(-39.0)
        else:
            x[r, V // 3: 2 * (V // 3)] = np.float16(-39.0)
        x[r, rng.integers(0, V)] = np.float16(30.0)  # the largest: the others are more than 4 octaves below
    u = (1 - 2.0 ** -24 - rng.random(M) * 0.3).astype(np.float32)
    for kw in (dict(temperature=50.0), dict(temperature=50.0, top_p=0.9), dict(temperature=80.0, top_k=V // 2)):
        tokens, probs = draw(W, x, u, **kw)
        for r in range(0, M, 3):  # (both kinds of rows; a row takes half a second)
            assert Sampled(x[r], float(u[r]), **kw).check(tokens[r], probs[r]), (kw, r, tokens[r], probs[r])
