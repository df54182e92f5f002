"""Refusals of w4a16_logprobs, w4a16_block_norm and w4a16_moe on the host: no call here reaches a launch."""
from __future__ import annotations

import pytest
import torch

FAKE = 1 << 40  # never dereferenced


@pytest.fixture(scope="module")
def W():
    import __graft_entry__

    __graft_entry__.build_library()
    import w4a16_weight_streaming_gb300 as W

    return W


LOGPROBS = dict(logits=FAKE, stride=1000, M=4, V=1000, tokens=FAKE * 2, given=1, top=3, temperature=FAKE * 3, logprob=FAKE * 4,
                rank=FAKE * 5, entropy=FAKE * 6, top_tokens=FAKE * 7, top_logprob=FAKE * 8, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), 1), (dict(M=0), 1), (dict(V=0), 1), (dict(stride=999), 1), (dict(tokens=None), 1), (dict(given=0), 1),
    (dict(given=-1), 1), (dict(top=-1), 1), (dict(top=0), 1), (dict(top_tokens=None), 1), (dict(top_logprob=None), 1),
    (dict(given=0, tokens=None, logprob=None, rank=None, entropy=None, top=0, top_tokens=None, top_logprob=None), 1),
    (dict(given=0, tokens=None, rank=None), 1),
    (dict(given=9), 2), (dict(top=33), 2), (dict(V=1000001, stride=1000001), 2), (dict(M=65537), 2), (dict(stride=(1 << 32) + 1), 2),
    (dict(logits=FAKE + 1), 3), (dict(tokens=FAKE * 2 + 2), 3), (dict(entropy=FAKE * 6 + 1), 3), (dict(temperature=FAKE * 3 + 2), 3),
    (dict(logprob=FAKE + 400), 1), (dict(rank=FAKE * 4 + 8), 1), (dict(top_tokens=FAKE * 2), 1), (dict(entropy=FAKE * 3 + 12), 1),
])
def test_logprobs(W, change, code):
    assert W.w4a16_logprobs(**{**LOGPROBS, **change}) == code


NORM = dict(h=FAKE, h_stride=512, h_f32=0, y=FAKE * 2, y_stride=512, post_weight=FAKE * 3, gate=FAKE * 4, gate_stride=512, gate_per_row=0,
            scale=1.0, weight=FAKE * 5, offset=0.0, eps=1e-6, h_out=FAKE * 6, x=FAKE * 7, M=4, H=512, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(h=None), 1), (dict(h_out=None, x=None), 1), (dict(M=0), 1), (dict(H=0), 1), (dict(h_f32=2), 1), (dict(gate_per_row=-1), 1),
    (dict(y=None), 1), (dict(y=None, gate=None), 1), (dict(scale=float("inf")), 1), (dict(eps=-1.0), 1), (dict(offset=float("nan")), 1),
    (dict(h_stride=504), 1), (dict(y_stride=0), 1), (dict(gate_stride=504), 1), (dict(gate_stride=-8), 1),
    (dict(H=508), 2), (dict(H=32776, h_stride=32776, y_stride=32776, gate_stride=0), 2), (dict(M=(1 << 20) + 1), 2),
    (dict(h_stride=513), 2), (dict(y_stride=514), 2), (dict(gate_stride=516), 2), (dict(h_stride=1 << 33), 2),
    (dict(h=FAKE + 2), 3), (dict(gate=FAKE * 4 + 2), 3), (dict(gate=FAKE * 4 + 1, gate_per_row=1), 3), (dict(x=FAKE * 7 + 8), 3),
    (dict(weight=FAKE * 5 + 2), 3),
    (dict(h_out=FAKE + 512), 1), (dict(x=FAKE), 1), (dict(x=FAKE * 2), 1), (dict(x=FAKE * 6 + 1024), 1), (dict(h_out=FAKE * 4), 1),
    (dict(h_out=FAKE, h_stride=520), 1),  # in place only where the rows are dense
])
def test_block_norm(W, change, code):
    assert W.w4a16_block_norm(**{**NORM, **change}) == code


def desc(W, **kw):
    d = dict(gate_up_q=FAKE * 10, gate_up_s=FAKE * 11, down_q=FAKE * 12, down_s=FAKE * 13, gate_up_scale=None, down_scale=None,
             experts=8, hidden=512, inner=256, group=64, nvfp4=0)
    d.update(kw)
    return W.MoEDesc(**d)


MOE = dict(x=FAKE, x_stride=512, router=FAKE * 2, bias=None, top_k=2, scoring=0, renormalize=1, scale=1.0, y=FAKE * 3, ids=FAKE * 4,
           weights=FAKE * 5, tokens=6, workspace=FAKE * 6, workspace_bytes=1 << 26, stream=None)


@pytest.mark.parametrize("change,experts,code", [
    (dict(x=None), {}, 1), (dict(router=None), {}, 1), (dict(y=None), {}, 1), (dict(workspace=None), {}, 1), (dict(tokens=0), {}, 1),
    (dict(top_k=0), {}, 1), (dict(top_k=9), {}, 1), (dict(scoring=2), {}, 1), (dict(renormalize=2), {}, 1), (dict(scale=float("nan")), {}, 1),
    (dict(bias=FAKE * 7), {}, 1), (dict(workspace_bytes=1000), {}, 1), (dict(x_stride=504), {}, 1),
    ({}, dict(gate_up_q=None), 1), ({}, dict(down_s=None), 1), ({}, dict(experts=0), 1), ({}, dict(nvfp4=2), 1), ({}, dict(nvfp4=1), 1),
    ({}, dict(gate_up_scale=FAKE), 1),
    (dict(tokens=65), {}, 2), (dict(top_k=17), dict(experts=64), 2), ({}, dict(experts=513), 2), ({}, dict(hidden=480), 2), ({}, dict(inner=224), 2),
    ({}, dict(group=48), 2), ({}, dict(group=96), 2), ({}, dict(group=512), 2), ({}, dict(group=0), 2), (dict(x_stride=516), {}, 2),
    (dict(x=FAKE + 8), {}, 3), (dict(y=FAKE * 3 + 4), {}, 3), (dict(workspace=FAKE * 6 + 8), {}, 3), (dict(ids=FAKE * 4 + 2), {}, 3),
    ({}, dict(down_q=FAKE * 12 + 4), 3), (dict(scoring=1, bias=FAKE * 7 + 2), {}, 3),
    (dict(y=FAKE), {}, 1), (dict(workspace=FAKE * 3), {}, 1), (dict(ids=FAKE * 5), {}, 1), (dict(y=FAKE * 12), {}, 1), (dict(weights=FAKE * 2), {}, 1),
])
def test_moe(W, change, experts, code):
    a = {**MOE, **change}
    if a["stream"] is None and experts.get("hidden"):
        a["x_stride"] = experts["hidden"]
    assert W.w4a16_moe(experts=desc(W, **experts), **a) == code


def test_workspace_bytes(W):
    assert W.w4a16_moe_workspace_bytes(64, 5120, 2176) > 64 * 16 * 2176 * 2
    for bad in ((0, 512, 256), (513, 512, 256), (8, 96, 256), (8, 512, 100), (8, 512, 65600)):
        assert W.w4a16_moe_workspace_bytes(*bad) == 0


def test_tensors_that_are_refused(W):
    """The binding's own checks, on CPU tensors: nothing is launched."""
    x = torch.zeros((4, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        W.logprobs(x)
    with pytest.raises(ValueError):
        W.block_norm(x, x)
    with pytest.raises(ValueError):
        W.Experts(torch.zeros((2, 8, 128), dtype=torch.int32), x, x, x)


@pytest.mark.parametrize("shape", [(), (8,), (8, 128), (1, 2, 8, 128)])
def test_experts_of_other_ranks_are_refused(W, shape):
    m, s = torch.zeros(shape, dtype=torch.int32), torch.zeros((2, 1, 128), dtype=torch.float16)
    for codes in ((m, m), (m, torch.zeros((2, 8, 64), dtype=torch.int32)), (torch.zeros((2, 8, 128), dtype=torch.int32), m)):
        with pytest.raises(ValueError):
            W.Experts(codes[0], s, codes[1], s)
