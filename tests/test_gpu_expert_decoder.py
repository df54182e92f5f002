"""Block norms, experts and log probabilities as a decoder uses them together.

* the example decoder with experts and a norm on both sides of every block: replayed steps are the steps, bit for bit,
  and so are their scores;
* one layer's end and the output head against 64 bits, for the choice of experts that was made. Errors, as shares of a
  row's norm: inputs of the experts rounded once (2^-11), gate, up and a within 2^-9 together, y 2^-11, the residual
  and its norm 2^-11 each, the head's weights and sums 2^-10, logits rounded once: below 2^-7 in all."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import w4a16_inputs as inputs
from gpu_util import lib

pytestmark = pytest.mark.gpu

SIZES = dict(hidden=512, heads=8, kv_heads=2, head_dim=64, mlp=512, vocab=1024, page=16, rot=32, experts=8, expert_mlp=256, top_k=3,
             block_norms=True)


@pytest.fixture(scope="module")
def E():
    lib()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_step

    return decode_step


@pytest.mark.parametrize("change", [dict(), dict(block_norms=False), dict(experts=0)], ids=["both", "experts", "norms"])
def test_replayed_steps_are_the_steps(E, change):
    g = torch.Generator("cuda").manual_seed(2)
    prompt = torch.randint(0, 1024, (3, 30), generator=g, device="cuda")  # 90 rows: two calls of the experts a layer
    u = torch.rand((9, 3), generator=g, device="cuda")
    one = torch.ones(3, device="cuda")
    kw = dict(temperature=one, top_k=(100 * one).int(), top_p=0.9 * one, min_p=0.001 * one)
    runs = []
    for graph in (False, True):
        model = E.Decoder(2, 3, 48, **{**SIZES, **change})
        scores = torch.full_like(u, 7.0)
        runs.append((E.generate(model, prompt, 9, u, graph=graph, scores=scores, **kw), scores))
    torch.cuda.synchronize()
    assert E.W.w4a16_device_status() == E.W.OK
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    tokens, scores = runs[0]
    assert int(tokens.min()) >= 0 and int(tokens.max()) < 1024 and bool((scores <= 0).all())
    assert len(set(tokens.flatten().tolist())) > 3


def test_a_layers_end_against_64_bits(E):
    W = E.W
    H, I, X, K, T, V = 512, 384, 12, 3, 11, 2048
    g = torch.Generator("cuda").manual_seed(5)

    def r(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def codes(rows, cols):
        q = torch.randint(-2 ** 31, 2 ** 31, (X, rows // 8, cols), generator=g, device="cuda", dtype=torch.int32)
        return q, (0.004 * (1 + torch.rand((X, rows // 128, cols), generator=g, device="cuda"))).half()

    up, down = codes(H, 2 * I), codes(I, H)
    m = W.Experts(*up, *down, group=128)
    work = W.moe_workspace(m)
    router = (r(X, H) * 2 / H ** 0.5).half()
    h, y, w1, w2, p1, p2 = r(T, H), r(T, H).half(), *((1 + 0.1 * r(H)).half() for _ in range(4))
    qw, sc = inputs.generate_weights(H, V, 128, seed=3)
    qw, sc = torch.from_numpy(qw).cuda(), torch.from_numpy(sc.view(np.int16)).cuda()
    packed = W.repack(qw, sc, 128)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda").int()

    h1, x1 = W.block_norm(h, y, weight=w1, post_weight=p1, scale=0.5)  # fp32 residual stream
    z, ids, share = W.moe(x1, m, router, K, work)
    h2, x2 = W.block_norm(h1, z, weight=w2, post_weight=p2, scale=0.5)
    logits = W.gemm(x2, *packed, V, H, 128)
    got = W.logprobs(logits, tokens, top=4)
    torch.cuda.synchronize()
    assert W.w4a16_device_status() == W.OK

    def rms(v, weight):
        return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * weight.double()

    def weights(q, s):
        c = ((q[:, None, :] >> (4 * torch.arange(8, device="cuda"))[None, :, None]) & 15).flatten(0, 1) - 8
        return (c.float() * s.float().repeat_interleave(128, 0)).half().double()

    h64 = h.double() + 0.5 * rms(y.double(), p1)
    x64 = rms(h64, w1)
    score = torch.softmax(x64 @ router.double().T, 1).gather(1, ids.long())
    score = score / score.sum(1, keepdim=True)
    z64 = torch.zeros_like(x64)
    for t in range(T):
        for j in range(K):
            e = int(ids[t, j])
            both = x64[t] @ weights(up[0][e], up[1][e])
            a = both[:I] * torch.sigmoid(both[:I]) * both[I:]
            z64[t] += score[t, j] * (a @ weights(down[0][e], down[1][e]))
    h64 = h64 + 0.5 * rms(z64, p2)
    l64 = rms(h64, w2) @ weights(qw, sc.view(torch.float16))

    def off(a, b):
        return float(((a.double() - b).norm(dim=1) / b.norm(dim=1)).max())

    assert off(h2, h64) < 2.0 ** -7 and off(logits, l64) < 2.0 ** -7 and float((share - score).abs().max()) < 2.0 ** -8
    lp = torch.log_softmax(logits.double(), 1)  # of the logits as they are: exact tokens
    assert torch.equal(got.top_tokens.long(), torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :4])
    assert float((got.logprob - lp.gather(1, tokens.long()[:, None])[:, 0]).abs().max()) < 1e-5
