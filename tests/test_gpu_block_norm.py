"""block_norm against the formula in 64 bits.

Bounds: a sum of squares goes through at most 24 roundings of 2^-24 (square, pairs, a thread's 8 vectors, warp, warps),
half of that after the root, 6 more in root, division and factors: below 2^-19 of z and of x. The sum h + scale gate z
adds 2^-22 of its terms. Outputs are rounded once: half a step, 2^-11 (fp16) or 2^-24 (fp32), 2^-25 among subnormals."""
from __future__ import annotations

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    return lib()


def rms(v, w, eps, offset):
    v = v * (v.square().mean(1, keepdim=True) + eps).rsqrt()
    return v if w is None else v * (offset + w.double())


def check(W, h, y=None, weight=None, post=None, gate=None, scale=1.0, eps=1e-6, offset=0.0, result=None, **kw):
    before = h.clone()
    h2, x = result if result is not None else W.block_norm(h, y, weight=weight, post_weight=post, gate=gate, scale=scale, eps=eps, offset=offset, **kw)
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.OK
    d = before.double()
    branch = torch.zeros_like(d)
    if y is not None:
        z = y.double() if post is None else rms(y.double(), post, eps, offset)
        branch = scale * z * (1.0 if gate is None else gate.double())
    ref = d + branch
    slack = 2.0 ** -19 * branch.abs() + 2.0 ** -22 * d.abs()
    if h2 is not None:
        half = 2.0 ** -11 if h.dtype is torch.float16 else 2.0 ** -24
        assert bool(((h2.double() - ref).abs() <= half * ref.abs() * 1.001 + 2.0 ** -25 + slack).all())
    if x is not None:
        q = (ref.square().mean(1, keepdim=True) + eps).rsqrt()
        f = torch.ones_like(ref) if weight is None else (offset + weight.double()).abs()
        want = rms(ref, weight, eps, offset)
        assert bool(((x.double() - want).abs() <= (2.0 ** -11 + 2.0 ** -19) * want.abs() * 1.001 + 2.0 ** -25 + slack * q * f
                     + 2.0 ** -21 * want.abs()).all())
    return h2, x


def make(M, H, f32=False, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + M * 131 + H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    h = 2 * r(M, H)
    return (h if f32 else h.half()), r(M, H).half(), (1 + 0.3 * r(H)).half(), (1 + 0.3 * r(H)).half(), r(M, H).half()


# a warp a row (1, 2, 4 vectors), a CTA a row with 1, 2, 4, 8 vectors a thread, odd row and vector counts
SIZES = [(1, 8), (5, 64), (3, 256), (7, 264), (2, 520), (400, 1000), (1, 1024), (1, 5120), (33, 5120), (400, 2048), (400, 4096),
         (400, 5120), (400, 8200), (310, 16384), (1, 8200), (2, 16392), (3, 32768), (310, 32768), (1001, 40)]


@pytest.mark.parametrize("f32", [False, True], ids=["f16", "f32"])
@pytest.mark.parametrize("M,H", SIZES)
def test_every_form_at_every_size(W, M, H, f32):
    h, y, w, p, g = make(M, H, f32)
    check(W, h, y, w)
    check(W, h, y, w, post=p, gate=g, scale=0.7, offset=1.0)
    check(W, h, y, None, post=p, gate=g[0].contiguous(), scale=-0.3)
    check(W, h, y, w, gate=g[:, :1].contiguous(), scale=2.0)
    check(W, h, y, w, gate=g[:, 3:4] if H > 8 else g[:, :1])  # one value a row of a wider tensor
    a = check(W, h, None, w)
    assert a[0] is h


@pytest.mark.parametrize("f32", [False, True])
def test_rows_with_strides(W, f32):
    M, H = 9, 1272
    h, y, w, p, g = make(M, H + 64, f32)
    check(W, h[:, 8:H + 8], y[:, 40:H + 40], w[:H].contiguous(), post=p[8:H + 8].contiguous(), gate=g[:, 16:H + 16])
    check(W, h[::2, 8:H + 8], y[::2, :H], w[:H].contiguous(), gate=g[0, 8:H + 8])
    check(W, h[:1, 8:H + 8], y[:1, 16:H + 16], w[:H].contiguous())


@pytest.mark.parametrize("f32", [False, True])
def test_in_place_and_single_outputs(W, f32):
    h, y, w, p, g = make(12, 1536, f32)
    old = h.clone()
    new, x = W.block_norm(h, y, weight=w, post_weight=p)
    x2 = torch.empty_like(x)
    assert W.block_norm(h, y, weight=w, post_weight=p, out=(h, x2))[0] is h
    torch.cuda.synchronize()
    assert torch.equal(h, new) and torch.equal(x, x2)
    check(W, old, y, w, post=p, out=(None, x2))
    check(W, old, y, w, post=p, out=(new, None))


def test_extreme_values(W):
    H = 2048
    h, y, w, p, _ = make(6, H, True)
    h[0] = 0
    y[0] = 0          # a row of nothing: eps carries the division
    y[1] *= 2.0 ** -14
    h[2] = 1e15       # squares of 1e30
    h[3, 0], y[3] = 60000.0, 0
    y[4] = 60000.0    # the largest fp16 numbers, squares of 4e9
    check(W, h, y, w, post=p)
    out = W.block_norm(h, y, weight=w, post_weight=p)[1]
    assert bool((out[0] == 0).all())
    h2, y2 = h[:3].half(), y[:3].clone()
    h2[2] = 1.0
    y2[1, 7], h2[2, 9] = float("inf"), float("nan")  # stay in their rows
    a, x = W.block_norm(h2, y2, weight=w)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(x[0]).all()) and bool(torch.isinf(a[1, 7])) and bool(torch.isnan(x[2]).any())


def test_replayed_on_another_stream(W):
    h, y, w, p, g = make(64, 5120)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    direct = W.block_norm(h, y, weight=w, post_weight=p, gate=g, stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = W.block_norm(h, y, weight=w, post_weight=p, gate=g)
    y.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    again = W.block_norm(h, y, weight=w, post_weight=p, gate=g)
    torch.cuda.synchronize()
    assert torch.equal(captured[0], again[0]) and torch.equal(captured[1], again[1])
    assert not torch.equal(direct[1], again[1])


def test_the_index_checking_build_gives_the_same(W):
    D = W.load_debug_bounds()
    h, y, w, p, g = make(5, 1336)
    a, x = torch.empty_like(h), torch.empty_like(h)
    s = torch.cuda.current_stream().cuda_stream
    assert D.w4a16_block_norm(h.data_ptr(), 1336, 0, y.data_ptr(), 1336, p.data_ptr(), g.data_ptr(), 1336, 0, 0.5, w.data_ptr(), 0.0, 1e-6,
                              a.data_ptr(), x.data_ptr(), 5, 1336, s) == 0
    torch.cuda.synchronize()
    assert D.w4a16_device_status(s) == W.OK
    b = W.block_norm(h, y, weight=w, post_weight=p, gate=g, scale=0.5)
    assert torch.equal(a, b[0]) and torch.equal(x, b[1])


def test_rows_further_apart_than_32_bits(W):
    H, step = 1024, 2 ** 31 + 8
    wide = torch.zeros(2 * step + H, dtype=torch.float16, device="cuda")
    h = wide.as_strided((3, H), (step, 1))
    h.copy_(make(3, H)[0])
    _, y, w, p, _ = make(3, H, seed=5)
    check(W, h, y, w, post=p)
    check(W, y, h, w, post=p, gate=h)


@pytest.mark.parametrize("H", [512, 5120])
def test_weights_that_earlier_calls_write(W, H):
    """Norm weights out of gemm, with a call of something else in between: every kernel here may start while the ones
    before it still run, the weights are those of their own step all the same. check()'s bounds."""
    K, steps = 8192, 24
    g = torch.Generator("cuda").manual_seed(H)
    codes = torch.randint(-2 ** 31, 2 ** 31, (K // 8, 2 * H), generator=g, device="cuda", dtype=torch.int32)
    matrix = W.repack(codes, (0.002 * (1 + torch.rand((K // 128, 2 * H), generator=g, device="cuda"))).half().view(torch.int16))
    inputs = torch.randn((steps, 1, K), generator=g, device="cuda").half()
    h, y, *_ = make(3, H)
    small = torch.randn((1, 64), generator=g, device="cuda").half()
    both = torch.zeros((1, 2 * H), dtype=torch.float16, device="cuda")  # post_weight and weight, written anew every step
    kept = torch.empty((steps, 2 * H), dtype=torch.float16, device="cuda")
    outs = [(torch.empty_like(h), torch.empty_like(h)) for _ in range(steps)]
    spare = (torch.empty_like(small), torch.empty_like(small))

    def run():
        for i in range(steps):
            W.gemm(inputs[i], *matrix, 2 * H, K, y=both)
            for _ in range(1 + i % 3):
                W.block_norm(small, small, out=spare)
            W.block_norm(h, y, weight=both[0, H:], post_weight=both[0, :H], offset=1.0, out=outs[i])
            kept[i] = both[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    both.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.OK
    for i, out in enumerate(outs):
        assert i == 0 or not torch.equal(kept[i], kept[i - 1])
        check(W, h, y, kept[i, H:], post=kept[i, :H], offset=1.0, result=out)
