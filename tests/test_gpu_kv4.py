"""The paged 4-bit cache on the GPU: append and load bit for bit against a binary32 statement, attention
against 64 bits under a bound derived from its roundings, and what may go wrong around both: pages that
end inside a tile, empty sequences and rows, rows beyond the length, unwritten memory, padding rows,
places that do not exist, other streams, graphs, long offsets."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    return lib()


def cuda(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda() if dtype is None else torch.tensor(x, dtype=dtype).cuda()


def ok(W):
    torch.cuda.synchronize()
    st = W.w4a16_device_status()
    assert st == W.OK, W.status_string(st)


def table(positions, rot):
    a = np.arange(positions)[:, None] * (1.0 / 10000.0 ** (np.arange(0, rot, 2) / rot))[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def awkward(rng, M, heads, D):
    """Rows as a product gives them, and rows where storage can go wrong."""
    x = (rng.normal(size=(M, heads, D)) * np.exp(0.7 * rng.normal(size=(heads, D)))).astype(np.float16)
    x[0, -1] = 0                                                   # nothing to scale
    x[0, 0, :64] = np.float16(3.25)                                # one value
    x[-1, -1, :64] = (np.arange(64) % 16 - 5).astype(np.float16)    # exact codes
    x[-1, 0, :64] = (np.arange(64) % 31 / 2).astype(np.float16)     # ties
    x[M // 2, -1, -64:] = np.float16(6e-8)                         # subnormal
    x[M // 2, -1, -1] = np.float16(-6e-8)
    x[M // 2, 0, 5] = np.float16(30000)                            # one large element
    return x.reshape(M, heads * D)


APPEND = [(1, 20, 4, 256, 64, False, True, 16), (3, 40, 8, 128, 128, True, False, 32), (65, 8, 8, 64, 32, False, True, 64),
          (17, 6, 2, 128, 48, False, True, 16), (5, 3, 1, 256, 256, True, True, 4096), (130, 5, 1, 64, 0, False, False, 16),
          (33, 2, 2, 256, 16, True, False, 128)]


@pytest.mark.parametrize("M,H,KV,D,rot,adjacent,normed,page", APPEND)
def test_append_and_load_match_the_definition_bit_for_bit(W, M, H, KV, D, rot, adjacent, normed, page):
    rng = np.random.default_rng(M * 1000 + D + rot)
    qkv = awkward(rng, M, H + 2 * KV, D)
    pad = 24
    wide = np.full((M, qkv.shape[1] + pad), np.nan, np.float16)  # rows of a wider buffer
    wide[:, :qkv.shape[1]] = qkv
    pages = M // page + 3
    cache = W.KV4Cache(pages, page, KV, D)
    cache.pages.fill_(0xFF)
    slots = rng.permutation(pages * page)[:M].astype(np.int32)
    pos = rng.integers(0, 500, M).astype(np.int32)
    rope = table(500, rot) if rot else None
    qn = (1 + 0.3 * rng.normal(size=D)).astype(np.float16) if normed else None
    kn = (1 + 0.3 * rng.normal(size=D)).astype(np.float16) if normed else None
    q = W.kv4_append(cuda(wide)[:, :qkv.shape[1]], cache, cuda(slots), heads=H,
                     positions=cuda(pos) if rot else None, rope=cuda(rope) if rot else None, adjacent=adjacent,
                     q_norm=cuda(qn) if normed else None, k_norm=cuda(kn) if normed else None, eps=1e-5)
    k, v = W.kv4_load(cache, cuda(slots))
    ok(W)
    qr, kr, vr = ref.append(qkv, H, KV, D, rope, pos, adjacent, qn, kn, 1e-5)
    assert np.array_equal(q.cpu().numpy().view(np.uint16) & 0x7FFF, qr.view(np.uint16) & 0x7FFF)
    assert np.array_equal(q.cpu().numpy(), qr)  # (signs of zero aside)
    assert np.array_equal(k.cpu().numpy(), kr.astype(np.float32).astype(np.float16))
    assert np.array_equal(v.cpu().numpy(), vr.astype(np.float32).astype(np.float16))


def test_append_keys_and_values_alone(W):
    rng = np.random.default_rng(5)
    kv = awkward(rng, 9, 6, 128)
    cache = W.KV4Cache(2, 16, 3, 128)
    slots = cuda(np.arange(9, dtype=np.int32) + 12)  # across a page's end
    assert W.kv4_append(cuda(kv), cache, slots, heads=0) is None
    k, v = W.kv4_load(cache, slots)
    ok(W)
    _, kr, vr = ref.append(kv, 0, 3, 128)
    assert np.array_equal(k.cpu().numpy(), kr.astype(np.float16)) and np.array_equal(v.cpu().numpy(), vr.astype(np.float16))


def test_append_leaves_other_tokens_alone_and_skips_padding(W):
    rng = np.random.default_rng(6)
    a, b = awkward(rng, 32, 4, 64), awkward(rng, 5, 4, 64)
    cache = W.KV4Cache(2, 16, 2, 64)
    every = cuda(np.arange(32, dtype=np.int32))
    W.kv4_append(cuda(a), cache, every, heads=0)
    W.kv4_append(cuda(b), cache, cuda(np.array([3, -1, 16, -5, 31], np.int32)), heads=0)
    k, v = W.kv4_load(cache, every)
    nothing = W.kv4_load(cache, cuda(np.array([-1, -7], np.int32)))
    ok(W)
    a[[3, 16, 31]] = b[[0, 2, 4]]
    _, kr, vr = ref.append(a, 0, 2, 64)
    assert np.array_equal(k.cpu().numpy(), kr.astype(np.float16)) and np.array_equal(v.cpu().numpy(), vr.astype(np.float16))
    assert all(int(t.abs().sum()) == 0 for t in nothing)


def test_places_that_do_not_exist_are_reported_and_store_nothing(W):
    rng = np.random.default_rng(7)
    x = awkward(rng, 3, 4, 64)
    cache = W.KV4Cache(2, 16, 1, 64)
    every = cuda(np.arange(32, dtype=np.int32))
    W.kv4_append(cuda(awkward(rng, 32, 2, 64)), cache, every, heads=0)
    before = cache.pages.clone()
    rope = cuda(table(10, 32))
    good = cuda(np.array([1, 2, 3], np.int32))
    W.kv4_append(cuda(x), cache, cuda(np.array([32, 2 ** 31 - 1, -1], np.int32)), heads=2)
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.ERR_BOUNDS and torch.equal(cache.pages, before)
    q = W.kv4_append(cuda(x), cache, good, heads=2, rope=rope, positions=cuda(np.array([10, -1, 2 ** 31 - 1], np.int32)))
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.ERR_BOUNDS and torch.equal(cache.pages, before)
    assert int(q.abs().sum()) == 0
    k, v = W.kv4_load(cache, cuda(np.array([32, 2 ** 31 - 1], np.int32)))
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.ERR_BOUNDS and int(k.abs().sum()) == 0 and int(v.abs().sum()) == 0
    ok(W)  # taken: the next call starts clean


# ------------------------------------------------------------------------------------ attention
class Batch:
    """Sequences of given lengths in pages of random order; memory that no token was written to holds NaN
    parameters."""

    def __init__(self, W, seed, lens, q_lens, H, KV, D, page, spare=2, gain=1.0):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.cache = W.KV4Cache(sum(need) + spare, page, KV, D)
        self.cache.pages.fill_(0xFF)
        order = rng.permutation(sum(need) + spare)
        self.table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
        self.keys, self.values, at = [], [], 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            k = (rng.normal(size=(n, KV, D)) * np.exp(0.3 * rng.normal(size=(KV, D)))).astype(np.float16)
            v = (gain * (rng.normal(size=(n, KV, D)) + rng.normal(size=(KV, D)))).astype(np.float16)
            self.keys.append(ref.store(k))
            self.values.append(ref.store(v))
            if n:
                t = np.arange(n)
                slots = self.table[b, t // page] * page + t % page
                W.kv4_append(cuda(np.concatenate([k, v], axis=1).reshape(n, -1)), self.cache,
                             cuda(slots.astype(np.int32)), heads=0)
        self.q_lens, self.lens = q_lens, lens
        self.q = (1.5 * rng.normal(size=(sum(q_lens), H, D))).astype(np.float16)
        self.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.work = W.kv4_attention_workspace(self.cache)

    def args(self, wide=False):
        """wide: a block table for far longer sequences (its columns beyond theirs name no page), as it is
        allocated once for all lengths; of several query rows it makes the tcgen05 kernel the choice."""
        table = self.table
        if wide:
            table = np.full((table.shape[0], table.shape[1] + 2 ** 20 // self.cache.page_tokens), -1, np.int32)
            table[:, : self.table.shape[1]] = self.table
        return dict(block_table=cuda(table), kv_len=cuda(np.array(self.lens, np.int32)), q_start=cuda(self.start),
                    max_q_len=max(1, max(self.q_lens)), workspace=self.work)

    def want(self, scale, causal=True):
        return ref.attention(self.q, self.keys, self.values, self.q_lens, scale, causal)


def close(got, want, bound, what=""):
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - want)
    assert np.isfinite(err).all(), f"{what}: not finite"
    worst = float((err / np.maximum(bound, 1e-30)).max())
    assert (err <= bound).all(), f"{what}: worst error / bound {worst:.3f}"
    return worst


ATTENTION = [
    # lens, q_lens, H, KV, D, page
    ([1], [1], 20, 4, 256, 16),
    ([777], [1], 20, 4, 256, 16),
    ([15, 16, 17, 0, 1, 33], [1, 1, 1, 1, 1, 1], 8, 8, 64, 16),
    ([64, 65, 300, 2], [1, 1, 1, 1], 40, 8, 128, 64),
    ([130, 31, 16], [3, 16, 16], 10, 2, 256, 32),
    ([40, 3, 0, 100], [7, 5, 2, 0], 9, 3, 128, 16),          # more queries than tokens: rows that see nothing
    ([513], [2], 16, 1, 128, 128),                           # 16 query heads on one key head
    ([200, 90], [33, 70], 5, 1, 256, 64),
    ([260, 400], [129, 31], 14, 2, 64, 16),
    ([350], [200], 4, 2, 128, 4096),                         # a page longer than the sequence
    ([2500], [1], 24, 4, 256, 32),
    ([700], [150], 20, 4, 256, 64),
    ([5000], [40], 8, 2, 64, 16),                            # many pages, parts of a unit from several CTAs
    ([3000, 64, 63, 1], [26, 64, 63, 1], 20, 4, 256, 16),    # whole prompts: the first rows see a token or two
    ([900] * 12, [17] * 12, 4, 1, 128, 64),
]


@pytest.mark.parametrize("lens,q_lens,H,KV,D,page", ATTENTION, ids=[f"case{i}" for i in range(len(ATTENTION))])
@pytest.mark.parametrize("wide", [False, True], ids=["short", "wide"])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_64_bits(W, lens, q_lens, H, KV, D, page, causal, wide):
    b = Batch(W, len(lens) * 100 + D + page, lens, q_lens, H, KV, D, page)
    lse = torch.full((sum(q_lens), H), 7.0, device="cuda")
    out = W.kv4_attention(cuda(b.q), b.cache, lse=lse, causal=causal, **b.args(wide))
    ok(W)
    want, want_lse, bound = b.want(D ** -0.5, causal)
    close(out, want, bound)
    got = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got), empty)
    # an absolute error of the scores is one of their logarithm: at most 2^-11 sum|q k'| scale + 2^-18
    tol = 2.0 ** -11 * D ** -0.5 * 6.0 * np.abs(b.q.astype(np.float64)).sum(-1) + 2.0 ** -18
    assert (np.abs(got[~empty] - want_lse[~empty]) <= tol[~empty]).all()
    assert int(b.work[:256].sum()) == 0  # the workspace is ready for the next call


def test_attention_with_rows_of_a_wider_buffer_and_another_scale(W):
    b = Batch(W, 11, [90, 20], [4, 1], 6, 2, 128, 16)
    wide = np.full((5, 6 * 128 + 40), np.nan, np.float16)
    wide[:, :768] = b.q.reshape(5, -1)
    out = W.kv4_attention(cuda(wide)[:, :768].unflatten(1, (6, 128)), b.cache, scale=0.3, **b.args())
    ok(W)
    want, _, bound = b.want(0.3)
    close(out, want, bound)


@pytest.mark.parametrize("wide", [False, True], ids=["short", "wide"])
@pytest.mark.parametrize("gain", [1e-4, 300.0])
def test_attention_of_small_and_large_values(W, gain, wide):
    # values near fp16's smallest normal numbers and far above one: products p * scale keep their bits
    b = Batch(W, 12, [333, 40], [1, 9], 20, 4, 256, 16, gain=gain)
    out = W.kv4_attention(cuda(b.q), b.cache, **b.args(wide))
    ok(W)
    want, _, bound = b.want(1 / 16)
    close(out, want, bound + 2.0 ** -25)


def test_attention_of_one_dominant_token(W):
    # a key that the query points at: every other weight is below fp16's range of the products
    b = Batch(W, 13, [400], [1], 4, 4, 64, 16)
    q = b.q.copy()
    for h in range(4):
        q[0, h] = (4 * b.keys[0][170, h]).astype(np.float16)
    b.q = q
    out = W.kv4_attention(cuda(q), b.cache, scale=1.0, **b.args())
    ok(W)
    want, _, bound = b.want(1.0)
    close(out, want, bound)


def test_attention_of_equal_keys_is_the_mean_of_the_values(W):
    n, KV, D = 100, 2, 128
    rng = np.random.default_rng(14)
    k = np.tile((np.arange(D) % 16).astype(np.float16), (n, KV, 1))
    v = rng.integers(0, 16, size=(n, KV, D)).astype(np.float16)
    v[..., 0::64], v[..., 1::64] = 0, 15  # scale 1: values are stored exactly
    cache = W.KV4Cache(7, 16, KV, D)
    slots = cuda(np.arange(n, dtype=np.int32))
    W.kv4_append(cuda(np.concatenate([k, v], axis=1).reshape(n, -1)), cache, slots, heads=0)
    out = W.kv4_attention(cuda(rng.normal(size=(1, KV, D)).astype(np.float16)), cache, cuda(np.arange(7, dtype=np.int32)[None]),
                          cuda(np.array([n], np.int32)), cuda(np.array([0, 1], np.int32)), 1, W.kv4_attention_workspace(cache))
    ok(W)
    mean = v.astype(np.float64).mean(0)
    assert (np.abs(out[0].float().cpu().numpy() - mean) <= 2.0 ** -10 * 2 * mean + 1e-6).all()


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 1, 17]], ids=["one", "several"])
def test_attention_repeats_bit_for_bit_and_on_another_stream(W, q_lens):
    b = Batch(W, 15, [3000, 1200, 50], q_lens, 20, 4, 256, 32)
    q, args = cuda(b.q), b.args(wide=True)
    a = W.kv4_attention(q, b.cache, **args)
    again = W.kv4_attention(q, b.cache, **args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = W.kv4_attention(q, b.cache, stream=s, **args)
    ok(W)
    assert torch.equal(a.view(torch.int16), again.view(torch.int16))
    assert torch.equal(a.view(torch.int16), other.view(torch.int16))
    want, _, bound = b.want(1 / 16)
    close(a, want, bound)


@pytest.mark.parametrize("lens,q_lens,H,KV,D", [([14000], [3], 8, 1, 64), ([16000], [26], 5, 1, 256), ([12000], [17], 16, 2, 128),
                                                ([5000, 4100, 70], [40, 9, 26], 10, 2, 256), ([14000], [30], 5, 1, 256),
                                                ([9000, 300], [20, 33], 16, 2, 64), ([4000, 4500], [50, 5], 8, 2, 128)],
                         ids=["many64", "many256", "many128", "several", "pairs256", "pairs64", "pairs128"])
def test_parts_of_long_units_are_added_alike_whoever_is_last(W, lens, q_lens, H, KV, D):
    """One unit's tokens in the hands of up to a dozen CTAs, which finish in any order."""
    b = Batch(W, 16, lens, q_lens, H, KV, D, 64)
    q, args = cuda(b.q), b.args(wide=True)
    lse = torch.empty((sum(q_lens), H), device="cuda")
    a = W.kv4_attention(q, b.cache, lse=lse, **args)
    for _ in range(25):
        lse_again = torch.empty_like(lse)
        again = W.kv4_attention(q, b.cache, lse=lse_again, **args)
        assert torch.equal(a.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse_again)
    ok(W)
    want, _, bound = b.want(D ** -0.5)
    close(a, want, bound)
    assert int(b.work[:4096].sum()) == 0


def test_attention_with_negative_and_zero_scale(W):
    b = Batch(W, 21, [100, 300], [1, 30], 4, 2, 128, 16)
    for wide in (False, True):
        for scale in (-0.1, 0.0):
            out = W.kv4_attention(cuda(b.q), b.cache, scale=scale, **b.args(wide))
            ok(W)
            want, _, bound = b.want(scale)
            close(out, want, bound, f"{scale} {wide}")


def test_a_captured_step_replays_with_other_lengths(W):
    H, KV, D, page = 10, 2, 128, 16
    b = Batch(W, 16, [70, 200], [1, 1], H, KV, D, page)
    q, args = cuda(b.q), b.args()
    out = torch.empty((2, H, D), dtype=torch.float16, device="cuda")
    W.kv4_attention(q, b.cache, out=out, **args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            W.kv4_attention(q, b.cache, out=out, **args)
    for lens in ([70, 200], [1, 17], [0, 199]):
        args["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        ok(W)
        want, _, bound = ref.attention(b.q, [k[:n] for k, n in zip(b.keys, lens)], [v[:n] for v, n in zip(b.values, lens)],
                                       [1, 1], D ** -0.5)
        close(out, want, bound, str(lens))


def test_pages_that_do_not_exist_many_rows(W):
    b = Batch(W, 22, [200, 64], [50, 30], 4, 2, 64, 16)
    b.table[0, 2], b.table[0, 7] = -1, 10 ** 6  # tokens 32..47 and 112..127 of the first sequence
    out = W.kv4_attention(cuda(b.q), b.cache, causal=False, **b.args(wide=True))
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.ERR_BOUNDS
    left = np.r_[0:32, 48:112, 128:200]
    want, _, bound = ref.attention(b.q, [b.keys[0][left], b.keys[1]], [b.values[0][left], b.values[1]], [50, 30], 0.125, False)
    close(out, want, bound)
    ok(W)


def test_pages_and_lengths_that_do_not_exist_are_cut_off(W):
    b = Batch(W, 17, [64, 64], [1, 1], 4, 2, 64, 16)
    args = b.args()
    args["kv_len"] = cuda(np.array([64, 1000], np.int32))  # longer than the table's row: its 64 tokens
    out = W.kv4_attention(cuda(b.q), b.cache, **args)
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.ERR_BOUNDS
    want, _, bound = b.want(0.125)
    close(out, want, bound)
    for bad in (-1, 10 ** 6):
        t = b.table.copy()
        t[0, 2] = bad  # tokens 32..47 of the first sequence
        args = b.args()
        args["block_table"] = cuda(t)
        out = W.kv4_attention(cuda(b.q), b.cache, **args)
        torch.cuda.synchronize()
        assert W.w4a16_device_status() == W.ERR_BOUNDS
        left = np.r_[0:32, 48:64]
        want, _, bound = ref.attention(b.q, [b.keys[0][left], b.keys[1]], [b.values[0][left], b.values[1]], [1, 1], 0.125)
        close(out, want, bound)
    args = b.args()
    args["q_start"] = cuda(np.array([0, 1, 90], np.int32))  # more rows than q has
    out = W.kv4_attention(cuda(b.q), b.cache, causal=False, **args)
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.ERR_BOUNDS
    want, _, bound = b.want(0.125, causal=False)
    close(out, want, bound)
    ok(W)


def test_rows_of_no_sequence_are_left_alone(W):
    b = Batch(W, 18, [20, 30], [2, 2], 4, 2, 64, 16)
    out = torch.full((4, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    args = b.args()
    args["q_start"] = cuda(np.array([1, 2, 3], np.int32))
    W.kv4_attention(cuda(b.q), b.cache, out=out, **args)
    ok(W)
    assert bool((out[0] == 5).all()) and bool((out[3] == 5).all())
    want, _, bound = ref.attention(b.q[1:3], b.keys, b.values, [1, 1], 0.125)
    close(out[1:3], want, bound)


def test_offsets_beyond_32_bits(W):
    # the last pages of a cache of 4.8 GB
    KV, D, page = 4, 256, 64
    cache = W.KV4Cache(65000, page, KV, D)
    assert cache.pages.numel() > 2 ** 32
    rng = np.random.default_rng(19)
    n = 100
    x = awkward(rng, n, 2 * KV, D)
    x = np.clip(x, -20, 20)
    pages = np.array([[64999, 64990]], np.int32)
    t = np.arange(n)
    slots = cuda((pages[0, t // page] * page + t % page).astype(np.int32))
    W.kv4_append(cuda(x), cache, slots, heads=0)
    k, v = W.kv4_load(cache, slots)
    q = rng.normal(size=(1, KV, D)).astype(np.float16)
    out = W.kv4_attention(cuda(q), cache, cuda(pages), cuda(np.array([n], np.int32)), cuda(np.array([0, 1], np.int32)), 1,
                          W.kv4_attention_workspace(cache))
    ok(W)
    _, kr, vr = ref.append(x, 0, KV, D)
    assert np.array_equal(k.cpu().numpy(), kr.astype(np.float32).astype(np.float16))
    assert np.array_equal(v.cpu().numpy(), vr.astype(np.float32).astype(np.float16))
    want, _, bound = ref.attention(q, [kr], [vr], [1], 1 / 16)
    close(out, want, bound)


@pytest.mark.parametrize("wide", [False, True], ids=["short", "wide"])
def test_the_index_checking_build_runs_clean(W, wide):
    import ctypes

    D_ = W.load_debug_bounds()
    b = Batch(W, 20, [100, 17, 0], [1, 20, 1], 6, 2, 128, 16)
    s = torch.cuda.current_stream().cuda_stream
    args = b.args(wide)
    q = cuda(b.q)
    out = torch.empty_like(q)
    assert D_.w4a16_kv4_attention(q.data_ptr(), q.stride(0), 6, ctypes.byref(b.cache.desc), args["block_table"].data_ptr(),
                                  args["block_table"].shape[1], args["kv_len"].data_ptr(), args["q_start"].data_ptr(), 3, 22,
                                  20, 1, 128 ** -0.5, out.data_ptr(), None, b.work.data_ptr(), b.work.numel(), s) == 0
    x = cuda(awkward(np.random.default_rng(3), 4, 10, 128))
    cache = W.KV4Cache(1, 16, 2, 128)
    slots = cuda(np.array([15, 0, 3, 8], np.int32))
    qq = torch.empty((4, 6, 128), dtype=torch.float16, device="cuda")
    kv = torch.empty((2, 4, 2, 128), dtype=torch.float16, device="cuda")
    assert D_.w4a16_kv4_append(x.data_ptr(), 1280, 6, qq.data_ptr(), ctypes.byref(cache.desc), slots.data_ptr(), None, None,
                               0, 0, 0, None, None, 0.0, 4, s) == 0
    assert D_.w4a16_kv4_load(ctypes.byref(cache.desc), slots.data_ptr(), kv[0].data_ptr(), kv[1].data_ptr(), 4, s) == 0
    torch.cuda.synchronize()
    assert D_.w4a16_device_status(s) == W.OK
    normal = W.kv4_attention(q, b.cache, **args)
    k, v = W.kv4_load(cache, slots)
    ok(W)
    assert torch.equal(out.view(torch.int16), normal.view(torch.int16))
    assert torch.equal(kv[0], k) and torch.equal(kv[1], v)


class Sink:
    """Sequences whose scores are exact: every key is 0 but that of one token, the same in all elements, and
    every query is 1, so that one token stands `gap` powers of two above the others, which are alike. The
    values' groups of 64 have gains of their own."""

    def __init__(self, W, seed, lens, KV, D, gap, gains, sink_value=1.0, group=1):
        rng = np.random.default_rng(seed)
        self.scale = gap * np.log(2) / (0.25 * D)
        need = [-(-n // 64) for n in lens]
        self.cache = W.KV4Cache(sum(need), 64, KV, D)
        self.cache.pages.fill_(0xFF)
        self.table = np.full((len(lens), max(need)), -1, np.int32)
        self.keys, self.values, self.magnitude, at = [], [], [], 0
        gain = np.repeat(np.asarray(gains), 64)
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = at + np.arange(need[b])
            at += need[b]
            one = rng.integers(0, n)
            k = np.zeros((n, KV, D), np.float16)
            k[one] = 0.25
            v = ((rng.normal(size=(n, KV, D)) + 0.5 * rng.normal(size=(KV, D))) * gain).astype(np.float16)
            v[one] = (v[one] * sink_value).astype(np.float16)
            slots = self.table[b, np.arange(n) // 64] * 64 + np.arange(n) % 64
            W.kv4_append(cuda(np.concatenate([k, v], axis=1).reshape(n, -1)), self.cache, cuda(slots.astype(np.int32)), heads=0)
            self.keys.append(ref.store(k))
            self.values.append(ref.store(v))
            # |min| + 15 scale of each element's group: what the codes' and the minimums' parts are made of
            g = self.values[-1].reshape(n, KV, D // 64, 64)
            size = np.abs(g.min(-1, keepdims=True)) + (g.max(-1, keepdims=True) - g.min(-1, keepdims=True)) * 1.01
            self.magnitude.append(np.broadcast_to(size, g.shape).reshape(n, KV, D))
        self.lens, self.H = lens, KV * group
        self.work = W.kv4_attention_workspace(self.cache)

    def run(self, W, q_lens, pages=None):
        q = np.ones((sum(q_lens), self.H, self.cache.head_dim), np.float16)
        start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        table = self.table
        if pages:
            table = np.full((table.shape[0], pages), -1, np.int32)
            table[:, :self.table.shape[1]] = self.table
        out = W.kv4_attention(cuda(q), self.cache, cuda(table), cuda(np.array(self.lens, np.int32)), cuda(start), max(q_lens),
                              self.work, scale=self.scale, causal=False)
        ok(W)
        one = [1] * len(self.lens)  # all queries of a sequence are alike
        q1 = np.ones((len(self.lens), self.H, self.cache.head_dim), np.float16)
        want, _, _ = ref.attention(q1, self.keys, self.values, one, self.scale, False)
        size, _, _ = ref.attention(q1, self.keys, self.magnitude, one, self.scale, False)
        plain, _, _ = ref.attention(q1, self.keys, [np.abs(v) for v in self.values], one, self.scale, False)
        of = np.repeat(np.arange(len(self.lens)), q_lens)
        return out, want[of], size[of], plain[of]


@pytest.mark.parametrize("lens,KV,D,group", [([8192], 4, 256, 5), ([700], 1, 256, 8), ([777] * 40, 8, 128, 1), ([5000] * 3, 2, 128, 4),
                                             ([1500] * 24, 4, 256, 2), ([3000], 2, 64, 4)])
def test_one_query_keeps_groups_of_any_size_exact(W, lens, KV, D, group):
    """One token has half of the weight. The decode kernel takes P times scale to 2^-18 of itself, a score of
    13 in fp32 is off by 13 * 2^-22 or less and the exponential by 2^-22, sums by less: 2^-16 of what a group
    of 64 is made of, beside the output's rounding to fp16. A group may be 2^12 times smaller than another."""
    b = Sink(W, 40, lens, KV, D, 13, [1, 2.0 ** -8, 2.0 ** -12, 2.0 ** -4][:D // 64], group=group)
    out, want, size, _ = b.run(W, [1] * len(lens))
    close(out, want, 2.0 ** -11 * np.abs(want) + 2.0 ** -16 * size + 2.0 ** -25)


@pytest.mark.parametrize("lens,q_lens,KV,D,group", [([16384], [20], 4, 256, 5), ([20000, 3000], [60, 60], 2, 256, 5), ([16000], [100], 1, 128, 4),
                                                    ([9000] * 3, [300, 40, 2], 2, 64, 2), ([16384], [64], 2, 128, 4),
                                                    ([2500] * 48, [20] * 48, 4, 256, 5), ([2000] * 80, [64] * 80, 2, 128, 4)])
def test_many_queries_keep_the_weights_of_a_long_context(W, lens, q_lens, KV, D, group):
    """One token whose value is 0 has nearly all of the weight, the others 2^-20.37 of it each. Keys are exact
    in fp16; values, weights and the output are rounded to it once each, 2^-11 of themselves, and sums of up to
    2000 products in fp32 are off by less than 2^-12."""
    b = Sink(W, 41, lens, KV, D, 20.37, [1.0] * (D // 64), sink_value=0.0, group=group)
    out, want, _, plain = b.run(W, q_lens, pages=2 ** 14)
    close(out, want, 2.0 ** -11 * np.abs(want) + (2.0 ** -10 + 2.0 ** -12) * plain + 2.0 ** -25)


@pytest.mark.parametrize("q_len", [1, 40, 130], ids=["decode", "one_cta", "pair"])
def test_a_sequence_of_nearly_2_31_tokens(W, q_len):
    """The longest that a block table may hold: three pages, then one page again and again. Rows see 2^31 - 32
    tokens or a few less, so what they see is known from four pages."""
    KV, D, page = 1, 64, 32
    rng = np.random.default_rng(42)
    x = rng.normal(size=(4 * page, 2 * D)).astype(np.float16)
    cache = W.KV4Cache(4, page, KV, D)
    W.kv4_append(cuda(x), cache, cuda(np.arange(4 * page, dtype=np.int32)), heads=0)
    k, v = ref.store(x[:, :D]).reshape(4, page, D), ref.store(x[:, D:]).reshape(4, page, D)
    pages = 2 ** 31 // page - 1
    n = pages * page
    table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    table[0, :3] = torch.tensor([1, 2, 3], dtype=torch.int32)
    q = rng.normal(size=(q_len, 1, D)).astype(np.float16)
    lse = torch.empty((q_len, 1), device="cuda")
    out = W.kv4_attention(cuda(q), cache, table, cuda(np.array([n], np.int32)), cuda(np.array([0, q_len], np.int32)), q_len,
                          W.kv4_attention_workspace(cache), lse=lse)
    ok(W)
    p = np.exp(np.einsum("id,ptd->ipt", q[:, 0].astype(np.float64), k) / 8)
    weight = np.ones((q_len, 4, page))
    weight[:, 0] = pages - 3
    for i in range(q_len):
        for t in range(n - q_len + 1 + i, n):
            weight[i, 0, t % page] -= 1
    z = (weight * p).sum((1, 2))
    want = np.einsum("ipt,ptd->id", weight * p, v) / z[:, None]
    size = np.einsum("ipt,ptd->id", weight * p, np.abs(v)) / z[:, None]
    # a thread's or accumulator's sum takes at most 2^25 tiles / 152 CTAs * 4 steps, 2^-24 of itself lost in each
    lost = 2.0 ** 25 / 152 * 4 * 2.0 ** -24
    scores = 2.0 ** -11 * 6.0 / 8 * np.abs(q[:, 0].astype(np.float64)).sum(-1)
    assert (np.abs(lse[:, 0].cpu().numpy() - np.log(z)) <= scores + lost).all()
    close(out[:, 0], want, 2.0 ** -10 * np.abs(want) + (2.0 ** -10 + 2 * scores[:, None] + lost) * size)


def test_one_row_of_a_buffer_of_any_width(W):
    b = Batch(W, 43, [50], [1], 4, 2, 64, 16)
    rng = np.random.default_rng(44)
    x = awkward(rng, 1, 8, 64)
    slots = cuda(np.array([3], np.int32))
    caches, outs = [W.KV4Cache(1, 16, 2, 64) for _ in range(2)], []
    for cache, width in zip(caches, (512, 517)):
        row = torch.zeros((1, width), dtype=torch.float16, device="cuda")
        row[:, :512] = cuda(x)
        q = W.kv4_append(row[:, :512], cache, slots, heads=4)
        qrow = torch.zeros((1, width), dtype=torch.float16, device="cuda")
        qrow[:, :256] = cuda(b.q.reshape(1, -1))
        outs.append((q, *W.kv4_load(cache, slots), W.kv4_attention(qrow[:, :256].unflatten(1, (4, 64)), b.cache, **b.args())))
    ok(W)
    assert all(torch.equal(one, other) for one, other in zip(*outs))


def batch_of(kind, B, rng, most_rows, most_tokens):
    """(lens, q_lens) of a large batch. few: three sequences of rows, the others empty; gaps: runs of empty
    sequences across the multiples of 32, sequences without rows and rows without tokens."""
    lens, q_lens = [0] * B, [0] * B
    for b in range(B):
        if kind == "few":
            busy = b in (3, 32, B - 1)
            lens[b], q_lens[b] = (most_tokens - b, most_rows) if busy else (int(b % 5 == 0), 0)
        elif not any(lo <= b < lo + 8 for lo in (28, 60, 92)):
            lens[b] = int(rng.integers(0, most_tokens)) if b % 7 else 0
            q_lens[b] = int(rng.integers(1, most_rows + 1)) if b % 5 else 0
    q_lens[B - 1], lens[B - 1] = most_rows, most_tokens
    return lens, q_lens


# kernel (w4a16_kv4_kernel), kind, rows, tokens, H, KV, a table for longer sequences
LARGE = {"decode-wide": (1, "few", 1, 3000, 8, 2, False), "decode": (2, "gaps", 1, 400, 16, 8, False),
         "one-cta": (3, "gaps", 20, 300, 8, 2, True), "one-cta-few": (3, "few", 25, 3000, 4, 1, True),
         "pairs": (4, "gaps", 40, 300, 8, 2, True), "pairs-few": (4, "few", 60, 3000, 4, 1, True)}


@pytest.mark.parametrize("B,D", [(33, 64), (33, 128), (65, 256), (65, 64), (100, 128), (100, 256)])
@pytest.mark.parametrize("case", LARGE)
def test_batches_of_more_than_32_sequences(W, case, B, D):
    kernel, kind, rows, tokens, H, KV, wide = LARGE[case]
    rng = np.random.default_rng(B + D)
    lens, q_lens = batch_of(kind, B, rng, rows, tokens)
    b = Batch(W, B * D, lens, q_lens, H, KV, D, 16)
    args = b.args(wide)
    lse = torch.full((sum(q_lens), H), 7.0, device="cuda")
    out = W.kv4_attention(cuda(b.q), b.cache, lse=lse, kernel=kernel, **args)
    ok(W)
    want, want_lse, bound = b.want(D ** -0.5)
    close(out, want, bound)
    got = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got), empty)
    tol = 2.0 ** -11 * D ** -0.5 * 6.0 * np.abs(b.q.astype(np.float64)).sum(-1) + 2.0 ** -18
    assert (np.abs(got[~empty] - want_lse[~empty]) <= tol[~empty]).all()
    assert int(b.work[:4096].sum()) == 0


@pytest.mark.parametrize("kind", ["weights", "keys"])
@pytest.mark.parametrize("kernel,q_len", [(2, 1), (2, 30), (3, 10), (4, 40)])
def test_no_bit_is_lost_that_the_kernels_say_they_keep(W, kernel, q_len, kind):
    """Two tokens, so that nothing averages a rounding out; a test without a GPU shows what breaks the bounds."""
    p, group = ref.Pairs(kind, 1), 4
    B, D = p.k.shape[0], p.D
    cache = W.KV4Cache(B, 16, 1, D)
    slots = (np.arange(B)[:, None] * 16 + np.arange(2)).reshape(-1).astype(np.int32)
    W.kv4_append(cuda(np.concatenate([p.k16, p.v16], axis=2).reshape(2 * B, 2 * D)), cache, cuda(slots), heads=0)
    table = np.full((B, 2 ** 16 if kernel > 2 else 1), -1, np.int32)
    table[:, 0] = np.arange(B)
    rows = [q_len] + [1] * (B - 1)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q = np.ones((sum(rows), group, D), np.float16)
    out = W.kv4_attention(cuda(q), cache, cuda(table), cuda(np.full(B, 2, np.int32)), cuda(start), q_len, W.kv4_attention_workspace(cache),
                          scale=p.SCALE, causal=False, kernel=kernel)
    ok(W)
    of = np.repeat(np.arange(B), rows)
    close(out, np.repeat(p.want[of][:, None], group, 1), np.repeat((p.one if kernel < 3 else p.many)[of][:, None], group, 1))


def test_host_memory_is_refused(W):
    b = Batch(W, 45, [20], [1], 4, 2, 64, 16)
    args = b.args()
    q, out = cuda(b.q), torch.empty((1, 4, 64), dtype=torch.float16, device="cuda")
    base = dict(q=q, table=args["block_table"], kv=args["kv_len"], start=args["q_start"], out=out, work=b.work)
    for name in base:
        t = dict(base)
        t[name] = base[name].cpu().pin_memory()
        assert W.w4a16_kv4_attention(t["q"].data_ptr(), 256, 4, b.cache.desc, t["table"].data_ptr(), 2, t["kv"].data_ptr(),
                                     t["start"].data_ptr(), 1, 1, 1, 1, 0.1, t["out"].data_ptr(), None, t["work"].data_ptr(),
                                     t["work"].numel(), None) == W.ERR_INVALID_ARG, name
    ok(W)


@pytest.mark.parametrize("kernel", [1, 2, 3, 4])
@pytest.mark.parametrize("case", [2, 4, 5, 6, 8, 9, 13])
def test_any_kernel_takes_any_call(W, case, kernel):
    lens, q_lens, H, KV, D, page = ATTENTION[case]
    b = Batch(W, 50 + case, lens, q_lens, H, KV, D, page)
    lse = torch.full((sum(q_lens), H), 7.0, device="cuda")
    q, args = cuda(b.q), b.args()
    out = W.kv4_attention(q, b.cache, lse=lse, kernel=kernel, **args)
    ok(W)
    want, want_lse, bound = b.want(D ** -0.5)
    close(out, want, bound)
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), np.isneginf(want_lse))
    chosen = W.w4a16_kv4_attention_kernel(H, b.cache.desc, args["block_table"].shape[1], len(lens), sum(q_lens), args["max_q_len"])
    if kernel == chosen:
        assert torch.equal(out.view(torch.int16), W.kv4_attention(q, b.cache, **args).view(torch.int16))
    assert int(b.work[:4096].sum()) == 0


@pytest.mark.parametrize("kernel", [1, 2])
def test_many_rows_by_the_exact_kernel(W, kernel):
    """A prompt at the decode kernel's bound: 2^-16 of what a group is made of, beside the output's rounding."""
    p = ref.Pairs("keys", 3)
    B, D = p.k.shape[0], p.D
    cache = W.KV4Cache(B, 16, 1, D)
    slots = (np.arange(B)[:, None] * 16 + np.arange(2)).reshape(-1).astype(np.int32)
    W.kv4_append(cuda(np.concatenate([p.k16, p.v16], axis=2).reshape(2 * B, 2 * D)), cache, cuda(slots), heads=0)
    rows = [150] + [2] * (B - 1)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    out = W.kv4_attention(cuda(np.ones((sum(rows), 4, D), np.float16)), cache, cuda(np.arange(B, dtype=np.int32)[:, None]),
                          cuda(np.full(B, 2, np.int32)), cuda(start), 150, W.kv4_attention_workspace(cache), scale=p.SCALE,
                          causal=False, kernel=kernel)
    ok(W)
    of = np.repeat(np.arange(B), rows)
    close(out, np.repeat(p.want[of][:, None], 4, 1), np.repeat(p.one[of][:, None], 4, 1))
