"""The example decoder: prompt chunk, decode steps and sampling together, small sizes.

* replaying the captured step gives the tokens of the same steps run one by one, bit for bit;
* a prompt taken in one chunk and the same tokens taken one at a time leave the same cache up to the
  roundings of the products (different tiles), and logits that differ by no more than these explain."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

SIZES = dict(hidden=512, heads=8, kv_heads=2, head_dim=64, mlp=512, vocab=1024, page=16, rot=32)


@pytest.fixture(scope="module")
def E():
    lib()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_step

    return decode_step


def test_replayed_steps_are_the_steps(E):
    g = torch.Generator("cuda").manual_seed(2)
    prompt = torch.randint(0, 1024, (3, 21), generator=g, device="cuda")
    u = torch.rand((9, 3), generator=g, device="cuda")
    one = torch.ones(3, device="cuda")
    kw = dict(temperature=one, top_k=(100 * one).int(), top_p=0.9 * one, min_p=0.001 * one)
    runs = []
    for graph in (False, True):
        model = E.Decoder(2, 3, 40, **SIZES)
        runs.append(E.generate(model, prompt, 9, u, graph=graph, **kw))
    torch.cuda.synchronize()
    assert E.W.w4a16_device_status() == E.W.OK
    assert torch.equal(runs[0], runs[1])
    assert int(runs[0].min()) >= 0 and int(runs[0].max()) < 1024
    assert len(set(runs[0].flatten().tolist())) > 3


def test_a_prompt_in_one_chunk_and_token_by_token(E):
    g = torch.Generator("cuda").manual_seed(3)
    n = 37
    prompt = torch.randint(0, 1024, (2, n), generator=g, device="cuda")
    a, b = E.Decoder(1, 2, 48, **SIZES), E.Decoder(1, 2, 48, **SIZES)
    chunk = a.prompt(prompt)
    for i in range(n):
        steps = b.step(prompt[:, i].int())
    torch.cuda.synchronize()
    assert E.W.w4a16_device_status() == E.W.OK
    # One layer: the qkv rows agree within the product's bound (2^-10 of sum|x w|, about 1 % of a row's
    # size at worst), so the same cached codes but for a few that are one step (1/15 of the range) apart.
    slots = (a.table[:, torch.arange(n, device="cuda") // 16] * 16 + torch.arange(n, device="cuda").int() % 16).reshape(-1)
    for x, y in zip(E.W.kv4_load(a.caches[0], slots), E.W.kv4_load(b.caches[0], slots)):
        x, y = x.float(), y.float()
        step = (x.amax(-1) - x.amin(-1)) / 15
        assert bool(((x - y).abs() <= 1.1 * step[..., None]).all())
        assert float(((x - y).abs() > 0.5 * step[..., None]).float().mean()) < 0.02
    # the logits: one code step in 2 % of the values is 0.02^0.5 / 15 of the range or so, below 3 % of them
    scale = chunk.float().std()
    assert float((chunk.float() - steps.float()).abs().max() / scale) < 0.25
    assert float((chunk.float() - steps.float()).square().mean().sqrt() / scale) < 0.05
