"""The mixture-of-experts layer against 64 bits.

Choice: logits are sums of exact fp16 products in fp32; a chain is H / 512 + 9 roundings long at most, so a logit is
off by less than 2^-19 of sum|x router| for H <= 5120. A choice has to be one that logits within that bound allow;
the rest is compared for the choice made.
Products: an instruction adds 16 products to an fp32 sum, off by 2^-21 of sum|x w| at most; with up to 2^5 in a chain and
the warps' sums, below 2^-16 of sum|x w|. a = silu(g) u is off by 1.1 |u| dg + |silu(g)| du, 2^-20 of itself for the
fp32 exponential and division, and its rounding, 2^-11 (2^-25 among subnormals). y by sum r (da |Wd|), as much of
sum r |a Wd|, the weights' own error (twice that of a logit, and 2^-20), and 2^-11 of itself."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import w4a16_inputs as inputs
from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    return lib()


def dequantised(q, s, group):
    """float64 [E, K, N] of int4 codes [E, K / 8, N] (int32) and fp16 scales: one rounding to fp16."""
    k = torch.arange(8, device=q.device) * 4
    code = ((q[:, :, None, :] >> k[None, None, :, None]) & 15).flatten(1, 2) - 8
    return (code.float() * s.float().repeat_interleave(group, 1)).half().double()


E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def dequantised_nvfp4(q, s8, factor):
    k = torch.arange(8, device=q.device) * 4
    code = ((q[:, :, None, :] >> k[None, None, :, None]) & 15).flatten(1, 2).long()
    value = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=q.device)[code]
    scale = s8.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return value * scale * factor.double()[:, None, None]


class Layer:
    def __init__(self, W, E, H, I, group=64, seed=0, nvfp4=False):
        g = torch.Generator("cuda").manual_seed(seed)
        self.E, self.H, self.I = E, H, I

        def codes(rows, cols):
            return torch.randint(-2 ** 31, 2 ** 31, (E, rows // 8, cols), generator=g, device="cuda", dtype=torch.int32)

        up, down = codes(H, 2 * I), codes(I, H)
        if nvfp4:
            s = [torch.randint(0x30, 0x40, (E, r // 16, c), generator=g, device="cuda").to(torch.uint8) for r, c in ((H, 2 * I), (I, H))]
            f = [(1 + torch.rand(E, generator=g, device="cuda")) / 256 for _ in range(2)]
            self.m = W.Experts(up, s[0], down, s[1], gate_up_scale=f[0], down_scale=f[1])
            self.up, self.down = dequantised_nvfp4(up, s[0], f[0]), dequantised_nvfp4(down, s[1], f[1])
        else:
            s = [(0.004 * (1 + torch.rand((E, r // group, c), generator=g, device="cuda"))).half() for r, c in ((H, 2 * I), (I, H))]
            self.m = W.Experts(up, s[0], down, s[1], group)
            self.up, self.down = dequantised(up, s[0], group), dequantised(down, s[1], group)
        self.router = (torch.randn((E, H), generator=g, device="cuda") * 1.5 / H ** 0.5).half()
        self.bias = 0.1 * torch.randn(E, generator=g, device="cuda")
        self.work = W.moe_workspace(self.m)

    def x(self, T, seed=0):
        g = torch.Generator("cuda").manual_seed(seed + 7 * T)
        return torch.randn((T, self.H), generator=g, device="cuda").half()


def check(W, L, x, k, sigmoid=False, renormalize=True, scale=1.0, bias=None, result=None, work=None):
    y, ids, w = result or W.moe(x, L.m, L.router, k, L.work if work is None else work, bias=bias, sigmoid=sigmoid,
                                renormalize=renormalize, scale=scale)
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.OK
    T = x.shape[0]
    xd, r = x.double(), L.router.double()
    logits, off = xd @ r.T, 2.0 ** -19 * (xd.abs() @ r.abs().T)
    score = torch.sigmoid(logits) if sigmoid else torch.softmax(logits, 1)
    key = score + (0 if bias is None else bias.double()) if sigmoid else logits
    key_off = off / 4 + 2.0 ** -22 if sigmoid else off
    chosen = ids.long()
    assert int(chosen.min()) >= 0 and int(chosen.max()) < L.E
    picked = torch.zeros_like(key, dtype=torch.bool).scatter(1, chosen, True)
    assert bool((picked.sum(1) == k).all())  # all different
    worst_in = (key + key_off).gather(1, chosen).amin(1)
    best_out = torch.where(picked, -torch.inf, key - key_off).amax(1)
    assert bool((worst_in >= best_out).all())
    got = key.gather(1, chosen)
    slack = key_off.gather(1, chosen)
    assert bool((got[:, :-1] + slack[:, :-1] >= got[:, 1:] - slack[:, 1:]).all())  # in order
    s = score.gather(1, chosen)
    s = s / s.sum(1, keepdim=True) if renormalize else s
    rel = 2 * off.amax(1, keepdim=True) + 2.0 ** -20
    assert bool(((w.double() - scale * s).abs() <= rel * scale * s).all())
    ref, bound = torch.zeros_like(xd), torch.zeros_like(xd)
    for e in range(L.E):
        t, j = (chosen == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        both, mass = xd[t] @ L.up[e], xd[t].abs() @ L.up[e].abs() * 2.0 ** -16
        g, u, dg, du = both[:, :L.I], both[:, L.I:], mass[:, :L.I], mass[:, L.I:]
        a = g * torch.sigmoid(g) * u
        da = 1.1 * u.abs() * dg + (g * torch.sigmoid(g)).abs() * du + 1.1 * dg * du + (2.0 ** -11 + 2.0 ** -20) * a.abs() + 2.0 ** -25
        weight = scale * s[t, j][:, None]
        ref.index_add_(0, t, weight * (a @ L.down[e]))
        sums = a.abs() @ L.down[e].abs()
        bound.index_add_(0, t, weight * (da @ L.down[e].abs() + (2.0 ** -16 + rel[t]) * sums))
    bound += 2.0 ** -11 * ref.abs() + 2.0 ** -25
    assert bool(((y.double() - ref).abs() <= bound * 1.01).all()), float(((y.double() - ref).abs() / bound).max())
    # the bound is a worst case; errors are independent, so a lost expert or token would still be far outside this
    assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -10
    return y, ids, w


# (experts, hidden, inner, group): odd counts, K not a multiple of 128, one group a row, a single column tile
SHAPES = [(4, 128, 128, 128), (5, 192, 64, 64), (24, 1280, 448, 64), (16, 320, 320, 32), (7, 640, 960, 160), (40, 512, 192, 64), (3, 64, 576, 32)]


@pytest.mark.parametrize("E,H,I,G", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 17, 33, 64])
def test_sizes(W, E, H, I, G, T):
    L = Layer(W, E, H, I, G, seed=E)
    x = L.x(T)
    check(W, L, x, min(2, E))
    check(W, L, x, min(6, E), sigmoid=True, bias=L.bias, scale=2.5)
    check(W, L, x, 1, renormalize=False)
    check(W, L, x, E if E <= 16 else 16, sigmoid=True, renormalize=False)


# scales within 2^-10 .. 2^-4, where codes become weights in one step, on the borders, and outside of them
SCALES = {"usual": lambda u: 0.002 + 0.01 * u, "wide": lambda u: 2.0 ** (-16 + 18 * u), "borders": lambda u: 2.0 ** (-10 - (u > 0.5) * 2.0 ** -10),
          "top": lambda u: 0.0625 * (1 - 2.0 ** -11 * (u > 0.3).float()), "odd": lambda u: torch.where(u < 0.1, -0.01, torch.where(u < 0.2, 0.0, torch.where(u < 0.3, 3e-7, 0.01)))}


@pytest.mark.parametrize("T", [1, 12, 60])  # 8, 16 and 32 tokens at a time
@pytest.mark.parametrize("G", [32, 64, 128, 192, 384])
@pytest.mark.parametrize("kind", SCALES)
def test_weights_are_the_formats_own(W, kind, G, T):
    """Rows with a single 1, and a down matrix of one power of two a column: y is a itself, of weights rounded once, times
    2^-7. silu and the product in fp32 are off by 2^-20, so a by half a step and that."""
    H = I = 384
    if T == 60 and G == 64:
        H = I = 320  # K not a multiple of 128
    if H % G:
        pytest.skip("the group does not divide K")
    g = torch.Generator("cuda").manual_seed(G)
    up = torch.randint(-2 ** 31, 2 ** 31, (1, H // 8, 2 * I), generator=g, device="cuda", dtype=torch.int32)
    scales = SCALES[kind](torch.rand((1, H // G, 2 * I), generator=g, device="cuda")).half()
    code = torch.full((I, H), 8, dtype=torch.int32, device="cuda")
    code.fill_diagonal_(9)
    down = torch.zeros((I // 8, H), dtype=torch.int32, device="cuda")
    for j in range(8):
        down |= code[j::8] << (4 * j)
    m = W.Experts(up, scales, down[None].contiguous(), torch.full((1, I // G, H), 2.0 ** -7, device="cuda").half(), G)
    at = torch.randint(0, H, (T,), generator=g, device="cuda")
    big = 64.0 if kind != "wide" else 1.0  # so that a is no subnormal number
    x = (torch.nn.functional.one_hot(at, H) * big).half()
    y, _, _ = W.moe(x, m, torch.zeros((1, H), device="cuda").half(), 1, W.moe_workspace(m))
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.OK
    both = big * dequantised(up, scales, G)[0][at]
    gate, upper = both[:, :I], both[:, I:]
    a = gate * torch.sigmoid(gate) * upper
    a16 = a.half().double()
    got = y.double() * 128.0
    near = 2.0 ** -20 * a.abs() + 2.0 ** -11 * a.abs() * 1.01 + 2.0 ** -24 * 65
    assert bool(((got - a).abs() <= near).all()), float(((got - a).abs() / near).max())
    if kind == "usual":  # half a step off at most, and nearly always the nearest
        assert float((got != a16).double().mean()) < 0.01


@pytest.mark.parametrize("T", [1, 6, 20, 64])
def test_nvfp4_experts(W, T):
    for E, H, I in ((8, 256, 192), (5, 192, 448)):
        L = Layer(W, E, H, I, nvfp4=True, seed=3)
        check(W, L, L.x(T), 3)


@pytest.mark.parametrize("T", [1, 16, 64])
def test_the_dense_layers_width(W, T):
    L = Layer(W, 12, 5120, 2176, 128, seed=1)
    check(W, L, L.x(T), 8)


def test_many_experts(W):
    L = Layer(W, 512, 128, 64, 64, seed=2)
    for T in (1, 64):
        check(W, L, L.x(T), 16, sigmoid=True, bias=L.bias)
        check(W, L, L.x(T), 8, renormalize=False)


@pytest.mark.parametrize("T", [9, 64])
def test_every_token_to_the_same_experts(W, T):
    L = Layer(W, 16, 256, 192, 64, seed=4)
    bias = torch.zeros(16, device="cuda")
    bias[5], bias[11] = 10.0, 20.0
    _, ids, _ = check(W, L, L.x(T), 2, sigmoid=True, bias=bias)
    assert ids.tolist() == [[11, 5]] * T


def test_ties_go_to_the_lower_index(W):
    L = Layer(W, 40, 256, 64, 64, seed=5)
    L.router[:] = L.router[7]
    for sigmoid in (False, True):
        _, ids, w = check(W, L, L.x(11), 5, sigmoid=sigmoid)
        assert ids.tolist() == [[0, 1, 2, 3, 4]] * 11
        assert torch.allclose(w, torch.full_like(w, 0.2), rtol=1e-6)
    L.router[33] = 2 * L.router[33]
    x = L.x(11)
    _, ids, _ = W.moe(x, L.m, L.router, 3, L.work)
    up = (x.double() @ L.router[33].double()) > 0
    assert all(r == ([33, 0, 1] if u else [0, 1, 2]) for r, u in zip(ids.tolist(), up.tolist()))


def test_infinities_and_nan_stay_in_their_row(W):
    L = Layer(W, 12, 256, 128, 64, seed=6)
    x = L.x(20)
    want, ids, _ = W.moe(x, L.m, L.router, 4, L.work)
    bad = x.clone()
    bad[3, 17], bad[9] = float("nan"), float("inf")
    got, got_ids, _ = W.moe(bad, L.m, L.router, 4, L.work)
    torch.cuda.synchronize()
    rest = [t for t in range(20) if t not in (3, 9)]
    assert torch.equal(got_ids[rest], ids[rest])
    # the list of experts may differ by the bad rows' choices, and with it the order of sums
    assert bool(((got[rest].double() - want[rest].double()).abs() <= 2.0 ** -9 * want[rest].double().abs().amax()).all())
    assert bool(torch.isnan(got[3]).all()) and int(got_ids.min()) >= 0 and int(got_ids.max()) < 12
    assert got_ids[3].tolist() == [0, 1, 2, 3]


def test_rows_with_a_stride_and_given_outputs(W):
    L = Layer(W, 6, 192, 128, 64, seed=7)
    wide = torch.randn((10, 264), device="cuda").half()
    check(W, L, wide[:, 8:200], 2)
    check(W, L, wide[4:5, 8:200], 2)
    y = torch.full((10, 192), 7.0, device="cuda").half()
    a = W.moe(wide[:, 8:200], L.m, L.router, 2, L.work, out=(y, None, None))
    b = W.moe(wide[:, 8:200], L.m, L.router, 2, L.work)
    torch.cuda.synchronize()
    assert a[0] is y and torch.equal(y, b[0])


def test_repeats_batches_and_a_shared_workspace(W):
    L = Layer(W, 24, 512, 320, 64, seed=8)
    x = L.x(48)
    first = W.moe(x, L.m, L.router, 4, L.work)
    for T in (1, 7, 48, 13, 48):  # the workspace is ready for any batch after any other
        again = W.moe(x[:T], L.m, L.router, 4, L.work)
        if T == 48:
            assert all(torch.equal(a, b) for a, b in zip(first, again))
        else:
            check(W, L, x[:T], 4, result=again)


def test_replayed_and_chained_calls(W):
    L = Layer(W, 16, 512, 256, 128, seed=9)
    x = L.x(5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    W.moe(x, L.m, L.router, 2, L.work, stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):  # the second layer takes the first one's output
        a = W.moe(x, L.m, L.router, 2, L.work)
        b = W.moe(a[0], L.m, L.router, 3, L.work, sigmoid=True)
    x.copy_(L.x(5, seed=33))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check(W, L, x, 2, result=a)
    check(W, L, a[0], 3, sigmoid=True, result=b)


def test_two_calls_at_once_with_their_own_workspaces(W):
    L = Layer(W, 16, 512, 256, 128, seed=10)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [L.work, W.moe_workspace(L.m)]
    xs = [L.x(8, seed=1), L.x(40, seed=2)]
    torch.cuda.synchronize()
    out = [None, None]
    for _ in range(10):
        for i in range(2):
            out[i] = W.moe(xs[i], L.m, L.router, 3, work[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check(W, L, xs[i], 3, result=out[i])


@pytest.mark.parametrize("nvfp4", [False, True])
def test_the_index_checking_build_gives_the_same(W, nvfp4):
    D = W.load_debug_bounds()
    L = Layer(W, 9, 320, 192, 64, seed=11, nvfp4=nvfp4)
    s = torch.cuda.current_stream().cuda_stream
    for T in (1, 21):
        x = L.x(T)
        want = W.moe(x, L.m, L.router, 3, L.work)
        got = [torch.empty_like(v) for v in want]
        assert D.w4a16_moe(x.data_ptr(), 320, L.m.ref, L.router.data_ptr(), None, 3, 0, 1, 1.0, *(v.data_ptr() for v in got), T,
                           L.work.data_ptr(), L.work.numel(), s) == 0
        torch.cuda.synchronize()
        assert D.w4a16_device_status(s) == W.OK
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_one_expert_is_the_dense_layer(W):
    """One expert that every token takes with weight 1: gemm, silu_mul and gemm of the same matrices, within the bounds."""
    H, I, G, T = 512, 256, 128, 12
    d = [inputs.generate_weights(H, 2 * I, G, seed=1), inputs.generate_weights(I, H, G, seed=2)]
    t = [(torch.from_numpy(q).cuda(), torch.from_numpy(s.view(np.int16)).cuda().view(torch.float16)) for q, s in d]
    m = W.Experts(t[0][0][None], t[0][1][None], t[1][0][None], t[1][1][None], G)
    x = torch.randn((T, H), device="cuda").half()
    y, ids, w = W.moe(x, m, torch.randn((1, H), device="cuda").half(), 1, W.moe_workspace(m))
    up = [W.repack(q, s.view(torch.int16), G) for q, s in t]
    act = W.silu_mul(W.gemm(x, *up[0], 2 * I, H, G))
    dense = W.gemm(act, *up[1], H, I, G)
    torch.cuda.synchronize()
    assert bool((ids == 0).all()) and bool((w == 1).all())
    y_ref, abs_ref = oracle.gemm(act.cpu().numpy().view(np.uint16), d[1][0], d[1][1], G)
    # gate and up rounded to fp16 there: 2^-11 of each, so act by 2^-9 at most
    assert bool((np.abs(y.double().cpu().numpy() - y_ref) <= 2.0 ** -10 * np.abs(y_ref) + 2.0 ** -8 * abs_ref).all())
    assert bool(((y.double() - dense.double()).abs() <= 0.02 * dense.double().abs().amax()).all())


def test_experts_and_rows_further_apart_than_32_bits(W):
    """300 experts of 2560 x 12288 and 6144 x 2560: 4.7 and 2.4 GB of codes. Only the chosen ones are looked at."""
    E, H, I, G = 300, 2560, 6144, 128
    g = torch.Generator("cuda").manual_seed(13)
    up = torch.randint(-2 ** 31, 2 ** 31, (E, H // 8, 2 * I), generator=g, device="cuda", dtype=torch.int32)
    down = torch.randint(-2 ** 31, 2 ** 31, (E, I // 8, H), generator=g, device="cuda", dtype=torch.int32)
    su = (0.004 * (1 + torch.rand((E, H // G, 2 * I), generator=g, device="cuda"))).half()
    sd = (0.004 * (1 + torch.rand((E, I // G, H), generator=g, device="cuda"))).half()
    m = W.Experts(up, su, down, sd, G)
    assert up.numel() * 4 > 2 ** 32
    step = 2 ** 31 + 8
    wide = torch.zeros(2 * step + H, dtype=torch.float16, device="cuda")
    x = wide.as_strided((3, H), (step, 1))
    x.copy_(torch.randn((3, H), generator=g, device="cuda").half())
    bias = torch.zeros(E, device="cuda")
    bias[[299, 150, 1]] = 5.0
    y, ids, w = W.moe(x, m, (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).half(), 3, W.moe_workspace(m), bias=bias, sigmoid=True)
    torch.cuda.synchronize()
    assert all(sorted(r) == [1, 150, 299] for r in ids.tolist())
    ref = torch.zeros((3, H), dtype=torch.float64, device="cuda")
    for e in (1, 150, 299):
        both = x.double() @ dequantised(up[e:e + 1], su[e:e + 1], G)[0]
        a = both[:, :I] * torch.sigmoid(both[:, :I]) * both[:, I:]
        share = torch.where(ids == e, w, 0.0).sum(1, keepdim=True).double()
        ref += share * (a @ dequantised(down[e:e + 1], sd[e:e + 1], G)[0])
    assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -10


@pytest.mark.parametrize("T", [5, 24, 64])
def test_experts_with_every_load(W, T):
    """One expert that every token takes, some that a few take, some that none does; tokens in every place of 8."""
    L = Layer(W, 20, 384, 256, 128, seed=14)
    g = torch.Generator("cuda").manual_seed(T)
    for _ in range(4):
        bias = torch.randn(20, generator=g, device="cuda")
        bias[int(torch.randint(0, 20, (1,), generator=g, device="cuda"))] = 9.0
        check(W, L, L.x(T, seed=int(torch.randint(0, 99, (1,), generator=g, device="cuda"))), 5, sigmoid=True, bias=bias)


@pytest.mark.parametrize("T", [1, 9])
def test_a_router_that_earlier_calls_write(W, T):
    """The router out of gemm, with a norm of something else in between: every kernel here may start while the ones before
    it still run, the choice is that of its own step's router all the same."""
    E, K, steps = 16, 8192, 24
    L = Layer(W, E, 512, 128, 128, seed=15)
    g = torch.Generator("cuda").manual_seed(15)
    codes = torch.randint(-2 ** 31, 2 ** 31, (K // 8, 512), generator=g, device="cuda", dtype=torch.int32)
    matrix = W.repack(codes, (0.0002 * (1 + torch.rand((K // 128, 512), generator=g, device="cuda"))).half().view(torch.int16))
    rows = torch.randn((steps, E, K), generator=g, device="cuda").half()
    x = L.x(T)
    small = torch.randn((1, 64), generator=g, device="cuda").half()
    spare = (torch.empty_like(small), torch.empty_like(small))
    kept = torch.empty((steps, E, 512), dtype=torch.float16, device="cuda")
    outs = [(torch.empty_like(x), torch.empty((T, 3), dtype=torch.int32, device="cuda"), torch.empty((T, 3), device="cuda")) for _ in range(steps)]

    def run():
        for i in range(steps):
            W.gemm(rows[i], *matrix, 512, K, y=L.router)
            for _ in range(1 + i % 3):
                W.block_norm(small, small, out=spare)
            W.moe(x, L.m, L.router, 3, L.work, out=outs[i])
            kept[i] = L.router

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    L.router.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert i == 0 or not torch.equal(kept[i], kept[i - 1])
        L.router = kept[i]
        check(W, L, x, 3, result=out)


@pytest.mark.parametrize("T", [1, 9])
def test_a_nan_score_reaches_every_weight_that_it_is_summed_into(W, T):
    L = Layer(W, 4, 128, 64, 64, seed=16)
    x = L.x(T)
    for value in (float("nan"), float("inf")):
        L.router[2] = 0
        L.router[2, 5] = value  # logits: NaN, or infinities of x's sign
        for k, sigmoid, renormalize in ((4, False, True), (2, False, False), (4, True, True), (4, True, False)):
            y, ids, w = W.moe(x, L.m, L.router, k, L.work, sigmoid=sigmoid, renormalize=renormalize)
            torch.cuda.synchronize()
            logits = x.double() @ L.router.double().T
            score = torch.sigmoid(logits) if sigmoid else torch.softmax(logits, 1)
            want = score.gather(1, ids.long())
            if renormalize:  # (softmax over the chosen ones: all of them here)
                want = want / want.sum(1, keepdim=True)
            assert torch.equal(torch.isnan(w), torch.isnan(want)), (value, k, sigmoid, renormalize)
            fine = ~torch.isnan(want)
            # a logit of 128 products off by 2^-19 of sum|x router| (below 32 here): 2^-14; scores and weights by four times that at most
            assert bool(((w.double() - want)[fine].abs() <= 2.0 ** -12 * want[fine]).all())
            assert bool(torch.isnan(y).all(1)[torch.isnan(want).any(1)].all())


@pytest.mark.parametrize("highest", [0.0, -16.0, -24.0, -64.0, -80.0, -96.0, -256.0, -1280.0])
def test_sigmoids_far_below_zero_share_what_there_is(W, highest):
    """Logits are exact here (64 products of one number). Scores are within 2^-22 of themselves, their sum within 2^-20, so a
    weight within 2^-19; scores below fp32's numbers beside one of e^-20 or more are 0: 2^-96 of the sum."""
    L = Layer(W, 6, 64, 64, 64, seed=17)
    x = torch.ones((9, 64), device="cuda").half()
    logits = torch.tensor([highest - 16, highest, highest - 1, highest - 80, highest, -torch.inf], device="cuda")
    L.router[:] = (logits / 64).half()[:, None]
    L.router[5] = 0
    L.router[5, 3] = -torch.inf
    order = [1, 4, 2, 0, 3, 5]
    for T in (1, 9):
        for k in range(1, 7):
            y, ids, w = W.moe(x[:T], L.m, L.router, k, L.work, sigmoid=True, scale=1.5, bias=torch.arange(0, -60, -10, device="cuda").float()[torch.tensor(order).argsort()])
            torch.cuda.synchronize()
            assert ids.tolist() == [order[:k]] * T
            log_score = torch.nn.functional.logsigmoid(logits.double())[order[:k]]
            want = 1.5 * torch.softmax(log_score, 0)
            assert bool(((w.double() - want).abs() <= 2.0 ** -19 * want + 2.0 ** -95).all()), (k, w[0], want)
            assert bool(torch.isfinite(y).all())
    L.router[:] = L.router[5]  # nothing but -inf
    y, ids, w = W.moe(x, L.m, L.router, 3, L.work, sigmoid=True)
    torch.cuda.synchronize()
    assert bool((w == 0).all()) and bool((y == 0).all())


@pytest.mark.parametrize("logits", [[17.5, 18, 30, 100, 25, 18], [-90, -100, -96, -200, -89, -96], [200, -200, 90, -90, 17, -17]])
def test_sigmoids_that_are_alike_in_fp32_are_chosen_by_their_logits(W, logits):
    """Logits are exact here (64 products of one number)."""
    L = Layer(W, 6, 64, 64, 64, seed=18)
    x = torch.ones((9, 64), device="cuda").half()
    L.router[:] = (torch.tensor(logits, device="cuda") / 64).half()[:, None]
    order = sorted(range(6), key=lambda e: (-logits[e], e))
    for T in (1, 9):
        for k in (1, 2, 3, 6):
            for renormalize in (False, True):
                _, ids, w = W.moe(x[:T], L.m, L.router, k, L.work, sigmoid=True, renormalize=renormalize)
                torch.cuda.synchronize()
                assert ids.tolist() == [order[:k]] * T
                log_score = torch.nn.functional.logsigmoid(torch.tensor(logits, dtype=torch.float64))[order[:k]]
                want = torch.softmax(log_score, 0) if renormalize else log_score.exp()
                # as above; a score itself below 2^-126 may be 0
                assert bool(((w.double().cpu() - want).abs() <= 2.0 ** -19 * want + 2.0 ** -95).all())
