"""Refusals of the cache, attention and sampling entry points: made on the host, before any launch. Also
the size functions and the plain statements' own properties. No GPU needed."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import kv4_ref as ref

FAKE = 1 << 40  # an aligned address that nothing dereferences
GB = 1 << 30


@pytest.fixture(scope="module")
def W():
    import __graft_entry__

    __graft_entry__.build_library()
    import w4a16_weight_streaming_gb300 as W

    return W


def test_cache_bytes(W):
    for (p, t, h, d) in [(10, 16, 4, 256), (1, 4096, 1, 64), (100000, 64, 8, 128)]:
        assert W.w4a16_kv4_cache_bytes(p, t, h, d) == p * t * h * 2 * (d // 2 + d // 64 * 4)
    for bad in [(0, 16, 4, 256), (10, 8, 4, 256), (10, 24, 4, 256), (10, 8192, 4, 256), (10, 16, 0, 256), (10, 16, 4, 96),
                (10, 16, 257, 64), (1 << 27, 16, 1, 64)]:
        assert W.w4a16_kv4_cache_bytes(*bad) == 0
        with pytest.raises(W.W4A16Error):
            W.KV4Cache(*bad, device="cpu")
    for d in (64, 128, 256):
        assert W.w4a16_kv4_attention_workspace_bytes(d) % 16 == 0 and W.w4a16_kv4_attention_workspace_bytes(d) > 0
    assert W.w4a16_kv4_attention_workspace_bytes(80) == 0


def desc(W, pages=FAKE + 64 * GB, n=16, t=16, h=4, d=128):
    return W.KV4Desc(pages, n, t, h, d)


def test_append_refusals(W):
    base = dict(qkv=FAKE, stride=3584, heads=20, q_out=FAKE + GB, cache=desc(W), slots=FAKE + 2 * GB, positions=FAKE + 3 * GB,
                rope=FAKE + 4 * GB, rows=100, rot=64, adjacent=0, q_norm=FAKE + 5 * GB, k_norm=FAKE + 6 * GB, eps=1e-6, M=7)

    def call(**kw):
        a = {**base, **kw}
        return W.w4a16_kv4_append(a["qkv"], a["stride"], a["heads"], a["q_out"], a["cache"], a["slots"], a["positions"],
                                  a["rope"], a["rows"], a["rot"], a["adjacent"], a["q_norm"], a["k_norm"], a["eps"], a["M"], None)

    for kw in (dict(qkv=0), dict(slots=0), dict(q_out=0), dict(M=0), dict(heads=-4), dict(positions=0), dict(rows=0), dict(rot=0),
               dict(adjacent=2), dict(eps=-1.0), dict(eps=float("nan")), dict(stride=3576), dict(cache=desc(W, pages=0)),
               dict(cache=desc(W, n=0)), dict(q_out=FAKE + 64), dict(q_out=FAKE + 64 * GB), dict(slots=FAKE + GB + 64),
               dict(qkv=FAKE + 64 * GB + 4096)):
        assert call(**kw) == W.ERR_INVALID_ARG, kw
    for kw in (dict(cache=desc(W, t=24)), dict(cache=desc(W, d=96)), dict(heads=18), dict(heads=1028), dict(stride=3588),
               dict(rot=24), dict(rot=144), dict(M=(1 << 20) + 1)):
        assert call(**kw) == W.ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(qkv=FAKE + 8), dict(q_out=FAKE + GB + 2), dict(slots=FAKE + 2 * GB + 2), dict(rope=FAKE + 4 * GB + 4),
               dict(q_norm=FAKE + 5 * GB + 8), dict(k_norm=FAKE + 6 * GB + 8), dict(positions=FAKE + 3 * GB + 1),
               dict(cache=desc(W, pages=FAKE + 64 * GB + 8))):
        assert call(**kw) == W.ERR_MISALIGNED, kw


def test_load_refusals(W):
    f, c = W.w4a16_kv4_load, desc(W)
    assert f(c, 0, FAKE, FAKE + GB, 4, None) == 1 and f(c, FAKE, 0, FAKE + GB, 4, None) == 1
    assert f(c, FAKE, FAKE + GB, 0, 4, None) == 1 and f(c, FAKE, FAKE + GB, FAKE + 2 * GB, 0, None) == 1
    assert f(c, FAKE, FAKE + GB, FAKE + GB + 16, 4, None) == 1            # v overlaps k
    assert f(c, FAKE, FAKE + 64 * GB, FAKE + GB, 4, None) == 1            # k overlaps the pages
    assert f(c, FAKE + 2, FAKE + GB, FAKE + 2 * GB, 4, None) == 3 and f(c, FAKE, FAKE + GB + 8, FAKE + 2 * GB, 4, None) == 3
    assert f(desc(W, d=32), FAKE, FAKE + GB, FAKE + 2 * GB, 4, None) == 2
    assert f(c, FAKE, FAKE + GB, FAKE + 2 * GB, (1 << 24) + 1, None) == 2


def test_attention_refusals(W):
    n = W.w4a16_kv4_attention_workspace_bytes(128)
    base = dict(q=FAKE, stride=2560, heads=20, cache=desc(W), table=FAKE + GB, pages=8, kv=FAKE + 2 * GB, start=FAKE + 3 * GB, B=2, M=5,
                most=4, causal=1, scale=0.1, out=FAKE + 4 * GB, lse=FAKE + 5 * GB, work=FAKE + 6 * GB, bytes=n)

    def call(**kw):
        a = {**base, **kw}
        return W.w4a16_kv4_attention(a["q"], a["stride"], a["heads"], a["cache"], a["table"], a["pages"], a["kv"], a["start"], a["B"],
                                     a["M"], a["most"], a["causal"], a["scale"], a["out"], a["lse"], a["work"], a["bytes"], None)

    for kw in (dict(q=0), dict(table=0), dict(kv=0), dict(start=0), dict(out=0), dict(work=0), dict(heads=0), dict(pages=0), dict(B=0),
               dict(M=0), dict(most=0), dict(causal=2), dict(scale=float("inf")), dict(scale=float("nan")), dict(stride=2552),
               dict(bytes=n - 1), dict(out=FAKE + 64), dict(out=FAKE + 64 * GB), dict(lse=FAKE + 4 * GB + 64),
               dict(work=FAKE + 4 * GB), dict(out=FAKE + GB), dict(cache=desc(W, pages=0))):
        assert call(**kw) == W.ERR_INVALID_ARG, kw
    for kw in (dict(heads=18), dict(stride=2564), dict(cache=desc(W, d=192)), dict(cache=desc(W, t=17)), dict(B=(1 << 20) + 1),
               dict(pages=1 << 28), dict(heads=1040)):
        assert call(**kw) == W.ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 4 * GB + 8), dict(work=FAKE + 6 * GB + 4), dict(lse=FAKE + 5 * GB + 2),
               dict(table=FAKE + GB + 1), dict(kv=FAKE + 2 * GB + 2), dict(start=FAKE + 3 * GB + 2)):
        assert call(**kw) == W.ERR_MISALIGNED, kw


def test_sample_refusals(W):
    base = dict(x=FAKE, stride=1000, M=4, V=1000, t=FAKE + GB, k=FAKE + 2 * GB, p=FAKE + 3 * GB, m=FAKE + 4 * GB, u=FAKE + 5 * GB,
                tokens=FAKE + 6 * GB, probs=FAKE + 7 * GB)

    def call(**kw):
        a = {**base, **kw}
        return W.w4a16_sample(a["x"], a["stride"], a["M"], a["V"], a["t"], a["k"], a["p"], a["m"], a["u"], a["tokens"], a["probs"], None)

    for kw in (dict(x=0), dict(u=0), dict(tokens=0), dict(M=0), dict(V=0), dict(stride=999), dict(probs=FAKE + 6 * GB + 8),
               dict(tokens=FAKE + 1000), dict(probs=FAKE + 5 * GB)):
        assert call(**kw) == W.ERR_INVALID_ARG, kw
    for kw in (dict(V=1000001, stride=1000001), dict(M=65537), dict(stride=(1 << 32) + 1)):
        assert call(**kw) == W.ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=FAKE + 1), dict(t=FAKE + GB + 2), dict(k=FAKE + 2 * GB + 1), dict(p=FAKE + 3 * GB + 2), dict(m=FAKE + 4 * GB + 2),
               dict(u=FAKE + 5 * GB + 2), dict(tokens=FAKE + 6 * GB + 2), dict(probs=FAKE + 7 * GB + 1)):
        assert call(**kw) == W.ERR_MISALIGNED, kw


def test_descriptor_matches_the_header(W):
    assert ctypes.sizeof(W.KV4Desc) == 24 and W.KV4Desc.num_pages.offset == 8 and W.KV4Desc.head_dim.offset == 20


# ------------------------------------------------------------------- the plain statements themselves
def test_storage_error_is_half_a_step_and_range_ends_are_kept():
    rng = np.random.default_rng(0)
    x = (rng.normal(size=(50, 3, 128)) * 3).astype(np.float16)
    y = ref.store(x).reshape(50, 3, 2, 64)
    x = x.astype(np.float64).reshape(50, 3, 2, 64)
    step = (x.max(-1) - x.min(-1)) / 15
    assert (np.abs(y - x) <= step[..., None] * (0.5 + 2.0 ** -6)).all()  # the scale is rounded to 11 bits: 15 codes, 2^-11 each
    assert np.array_equal(y.min(-1), x.min(-1))
    z = ref.store((np.arange(64) % 16 + 2).astype(np.float16))
    assert np.array_equal(z, np.arange(64) % 16 + 2)  # whole steps are exact
    assert np.array_equal(ref.store(np.full((1, 64), 7, np.float16)), np.full((1, 64), 7.0))


def test_rotation_keeps_lengths_and_is_undone_by_the_opposite_angle():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(6, 2, 64)).astype(np.float32)
    a = rng.normal(size=(9, 16))
    t = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    back = np.concatenate([np.cos(a), -np.sin(a)], 1).astype(np.float32)
    pos = rng.integers(0, 9, 6)
    for adjacent in (False, True):
        y = ref.rotate(x, t, pos, adjacent)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-5)
        assert np.allclose(ref.rotate(y, back, pos, adjacent), x, atol=1e-5)


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(2).normal(size=(4, 3, 256)).astype(np.float32) * 7
    y = ref.norm(x, np.ones(256, np.float16), 0.0)
    assert np.allclose((y.astype(np.float64) ** 2).mean(-1), 1, rtol=1e-6)


def test_attention_statement_by_brute_force():
    rng = np.random.default_rng(3)
    q = rng.normal(size=(3, 4, 64)).astype(np.float16)
    k, v = rng.normal(size=(2, 5, 2, 64))
    out, lse, _ = ref.attention(q, [k], [v], [3], 0.2)
    for i in range(3):
        for h in range(4):
            w = [np.exp(0.2 * float(np.dot(q[i, h].astype(np.float64), k[t, h // 2]))) for t in range(5 - 3 + i + 1)]
            o = sum(a * v[t, h // 2] for t, a in enumerate(w)) / sum(w)
            assert np.allclose(out[i, h], o) and np.isclose(lse[i, h], np.log(sum(w)))
    out, lse, _ = ref.attention(q, [k[:1]], [v[:1]], [3], 0.2)  # three queries, one token: two see nothing
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2], np.repeat(v[0], 2, axis=0))


def test_sampled_statement_refuses_wrong_tokens():
    x = np.array([1.0, 3.0, 2.0, -np.inf, 3.0], np.float16)
    p = np.exp([3, 3, 2, 1]) / np.exp([3, 3, 2, 1]).sum()  # tokens 1, 4, 2, 0
    s = ref.Sampled(x, float(p[0] + p[1] / 2))
    assert s.check(4, p[1]) and not s.check(1, p[0]) and not s.check(2, p[2]) and not s.check(3, 0.0) and not s.check(4, p[0] * 1.01)
    s = ref.Sampled(x, 0.999, top_k=2)
    assert s.check(4, 0.5) and not s.check(2, p[2])
    s = ref.Sampled(x, 0.5, temperature=0.0)
    assert s.check(1, 1.0) and not s.check(4, 1.0)
    assert ref.Sampled(np.full(3, -np.inf, np.float16), 0.5).check(-1, 0)


def test_selftest_refusals(W):
    assert W.w4a16_kv4_selftest_wait_timeout(2) == W.ERR_INVALID_ARG and W.w4a16_kv4_selftest_wait_timeout(-1) == W.ERR_INVALID_ARG
    assert W.w4a16_kv4_selftest_withhold(0) == W.ERR_INVALID_ARG  # only the index-checking build leaves copies out
    debug = W.load_debug_bounds()
    assert debug.w4a16_kv4_selftest_withhold(-2) == W.ERR_INVALID_ARG
    assert debug.w4a16_kv4_selftest_withhold(3) == W.OK and debug.w4a16_kv4_selftest_withhold(-1) == W.OK


def test_choice_of_the_attention_kernel(W):
    def choice(heads=20, pages=64, B=4, M=4, most=1, **kw):
        return W.w4a16_kv4_attention_kernel(heads, desc(W, **kw), pages, B, M, most)

    assert choice() == 1 and choice(B=64, M=64) == 2                       # one query: few units, many
    assert choice(M=80, most=20, pages=4096) == 3                          # 100 rows a key head
    assert choice(M=240, most=60, pages=4096, d=256) == 4                  # 300
    assert choice(M=160, most=40, pages=4096) == 4 and choice(M=104, most=26, pages=4096) == 4
    assert choice(M=100, most=25, pages=4096) == 3                         # 125 rows: one CTA's
    for kw in (dict(heads=0), dict(heads=18), dict(heads=1028), dict(pages=0), dict(pages=1 << 28), dict(B=0), dict(M=0), dict(most=0),
               dict(d=96), dict(t=24), dict(n=0), dict(h=0), dict(B=(1 << 20) + 1), dict(M=(1 << 20) + 1)):
        assert choice(**kw) == 0, kw


def test_every_attention_kernel_is_tested(W):
    from test_gpu_kv4 import ATTENTION, LARGE

    seen = set()
    for lens, q_lens, H, KV, D, page in ATTENTION:
        for wide in (0, 2 ** 20 // page):
            pages = max(1, max(-(-n // page) for n in lens)) + wide
            seen.add((W.w4a16_kv4_attention_kernel(H, desc(W, t=page, h=KV, d=D), pages, len(lens), sum(q_lens), max(1, max(q_lens))), D))
    assert {k for k, _ in seen} == {1, 2, 3, 4}
    assert {case[0] for case in LARGE.values()} == {1, 2, 3, 4}  # each with every head size, by name


def test_the_precision_bounds_see_a_lost_bit():
    """Three bits fewer than fp16 has, of the keys, the values or the weights, and one rounding of the decode
    kernel's products instead of two: each breaks its bound somewhere; what the kernels do keeps it."""
    worst = lambda p, got, bound: float((np.abs(got - p.want) / bound).max())  # noqa: E731
    weights, keys = ref.Pairs("weights", 1), ref.Pairs("keys", 1)
    for p in (weights, keys):
        assert worst(p, p.many_with(11, 11, 11), p.many) < 1 and worst(p, p.one_with(16), p.one) < 1
        assert worst(p, p.one_with(11), p.one) > 1.5
    assert worst(weights, weights.many_with(11, 8, 11), weights.many) > 2
    assert worst(weights, weights.many_with(11, 11, 8), weights.many) > 2
    assert worst(keys, keys.many_with(8, 11, 11), keys.many) > 2


def test_kernels_that_do_not_exist_are_refused(W):
    n = W.w4a16_kv4_attention_workspace_bytes(128)
    for kernel in (-1, 5):
        assert W.w4a16_kv4_attention_ex(FAKE, 2560, 20, desc(W), FAKE + GB, 8, FAKE + 2 * GB, FAKE + 3 * GB, 2, 5, 4, 1, 0.1, FAKE + 4 * GB,
                                        None, FAKE + 6 * GB, n, kernel, None) == W.ERR_INVALID_ARG
    assert [W.KV4_AUTO, W.KV4_DECODE_WIDE, W.KV4_DECODE, W.KV4_PROMPT, W.KV4_PROMPT_PAIRS] == list(range(5))


def test_the_choice_counts_the_rows_of_the_whole_batch(W):
    """Sequences that are alike are counted as before (cost and pair rules of one sequence times the batch); a
    prompt among streams of one query no longer counts as a prompt a stream."""
    def one_by_one(H, KV, D, tokens, B, n):
        rows = n * (H // KV)
        here = {256: 11.2, 128: 10.0, 64: 8.5}[D] + {256: 0.162, 128: 0.087, 64: 0.053}[D] / 152 * B * KV * -(-rows // 8) * (tokens / 16)
        there = {256: 26.3, 128: 19.3, 64: 16.1}[D] + {256: 0.73, 128: 0.69, 64: 0.74}[D] / 152 * B * KV * -(-rows // 128) * (tokens / 64)
        if abs(here - there) < 1e-9 * here:
            return None
        if here < there:
            return 1 if 2 * B * KV * -(-rows // 8) <= 152 else 2
        units = -(-rows // 128)
        return 4 if units % 2 == 0 or units >= (3 if D == 256 else 17) else 3

    rng = np.random.default_rng(0)
    for _ in range(3000):
        KV, D, grp = int(rng.integers(1, 9)), int(rng.choice([64, 128, 256])), int(rng.integers(1, 17))
        B, n, pages = int(np.exp(rng.uniform(0, 5))), int(np.exp(rng.uniform(0, 7))), int(np.exp(rng.uniform(0, 9)))
        want = one_by_one(KV * grp, KV, D, pages * 16, B, n)
        assert want in (None, W.w4a16_kv4_attention_kernel(KV * grp, desc(W, h=KV, d=D), pages, B, B * n, n)), (KV, D, grp, B, n, pages)
    mixed = lambda streams, n, d: W.w4a16_kv4_attention_kernel(20, desc(W, h=4, d=d), 256, streams + 1, streams + n, n)  # noqa: E731
    assert mixed(63, 512, 256) == mixed(15, 512, 256) == mixed(63, 512, 128) == 3
    assert mixed(3, 1024, 256) == 4
