"""A small decoder on the library's kernels: prompt chunks, then decode steps replayed as one CUDA graph.

    python examples/decode_step.py [--layers 2] [--streams 4] [--prompt 40] [--steps 16] [--experts 16] [--block-norms]

Every stream has its own pages of one 4-bit key/value cache per layer. A step of a layer is

    qkv product -> kv4_append (norms of q and k, rotation, keys and values stored) -> kv4_attention
    -> output projection -> gate+up product -> silu_mul -> down projection

and after the last layer the output head and `sample`. Weights are random int4 (repacked once); torch adds
the residuals and norms the rows. With --experts the MLP is a layer of experts (`moe`), two a token; with
--block-norms every block has a norm before and behind it, and the kernels keep the residual stream
(`block_norm`). `logprobs` scores the tokens that were drawn. The sizes are the dense layer's: hidden 5120, 20 query heads and 4
key/value heads of 256, MLP width 17,408; a small vocabulary, so that the example starts quickly."""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import w4a16_inputs as inputs  # noqa: E402
import w4a16_weight_streaming_gb300 as W  # noqa: E402

GROUP = 128


def rotation_table(positions: int, rot: int, base: float = 1e6) -> torch.Tensor:
    """float32 [positions, rot]: the cosines of the rot / 2 angles of a position, then their sines."""
    inv = 1.0 / base ** (torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float().cuda()


def rms_norm(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).half()


class Matrix:
    """A random int4 matrix [K, N] in the device layout."""

    def __init__(self, K: int, N: int, seed: int):
        qw, sc = inputs.generate_weights(K, N, GROUP, seed=seed)
        self.K, self.N = K, N
        self.r = W.repack(torch.from_numpy(qw).cuda(), torch.from_numpy(sc.view("int16")).cuda(), GROUP)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return W.gemm(x, *self.r, self.N, self.K, GROUP)


def random_experts(experts: int, hidden: int, inner: int, g: torch.Generator) -> W.Experts:
    def matrices(rows, cols):
        words = torch.randint(-2 ** 31, 2 ** 31, (experts, rows // 8, cols), generator=g, device="cuda", dtype=torch.int32)
        return words, (0.002 * (1 + torch.rand((experts, rows // GROUP, cols), generator=g, device="cuda"))).half()

    return W.Experts(*matrices(hidden, 2 * inner), *matrices(inner, hidden), group=GROUP)


class Decoder:
    def __init__(self, layers: int, streams: int, max_tokens: int, hidden: int = 5120, heads: int = 20, kv_heads: int = 4,
                 head_dim: int = 256, mlp: int = 17408, vocab: int = 8192, page: int = 32, rot: int = 64, seed: int = 0,
                 experts: int = 0, expert_mlp: int = 2176, top_k: int = 2, block_norms: bool = False):
        self.heads, self.kv_heads, self.head_dim, self.page, self.streams, self.vocab = heads, kv_heads, head_dim, page, streams, vocab
        qkv = (heads + 2 * kv_heads) * head_dim
        self.layers = [dict(qkv=Matrix(hidden, qkv, seed + 10 * i), o=Matrix(heads * head_dim, hidden, seed + 10 * i + 1))
                       for i in range(layers)]
        if not experts:
            for i, layer in enumerate(self.layers):
                layer.update(gu=Matrix(hidden, 2 * mlp, seed + 10 * i + 2), down=Matrix(mlp, hidden, seed + 10 * i + 3))
        self.head = Matrix(hidden, vocab, seed + 1000)
        g = torch.Generator("cuda").manual_seed(seed)
        self.embedding = torch.randn((vocab, hidden), generator=g, device="cuda").half()
        self.q_norm = (1 + 0.1 * torch.randn(head_dim, generator=g, device="cuda")).half()
        self.k_norm = (1 + 0.1 * torch.randn(head_dim, generator=g, device="cuda")).half()
        per = -(-max_tokens // page)
        self.rope = rotation_table(per * page, rot)
        self.table = torch.randperm(streams * per, generator=g, device="cuda").int().view(streams, per)
        self.caches = [W.KV4Cache(streams * per, page, kv_heads, head_dim) for _ in range(layers)]
        self.workspace = W.kv4_attention_workspace(self.caches[0])
        self.length = torch.zeros(streams, dtype=torch.int32, device="cuda")  # cached tokens of each stream
        self.top_k, self.block_norms = top_k, block_norms
        if experts:
            for layer in self.layers:
                layer["experts"] = random_experts(experts, hidden, expert_mlp, g)
                layer["router"] = (torch.randn((experts, hidden), generator=g, device="cuda") / hidden ** 0.5).half()
            self.moe_workspace = W.moe_workspace(self.layers[0]["experts"])
        if block_norms:  # before attention, behind it, before the MLP, behind it; and before the output head
            self.norms = (1 + 0.1 * torch.randn((layers * 4 + 1, hidden), generator=g, device="cuda")).half()

    def forward(self, tokens: torch.Tensor, stream_of: torch.Tensor, positions: torch.Tensor, q_start: torch.Tensor,
                max_q_len: int) -> torch.Tensor:
        """Hidden states of the rows: row r is the token at `positions[r]` of stream `stream_of[r]`; self.length
        already counts the rows."""
        slots = self.table[stream_of.long(), positions.long() // self.page] * self.page + positions % self.page
        h = self.embedding[tokens.long()]

        def attention(x, layer, cache):
            q = W.kv4_append(layer["qkv"](x), cache, slots, heads=self.heads, positions=positions, rope=self.rope,
                             q_norm=self.q_norm, k_norm=self.k_norm)
            return layer["o"](W.kv4_attention(q, cache, self.table, self.length, q_start, max_q_len, self.workspace).flatten(1))

        if self.block_norms:
            _, x = W.block_norm(h, weight=self.norms[0])
            for i, (layer, cache) in enumerate(zip(self.layers, self.caches)):
                n = self.norms[4 * i:]
                h, x = W.block_norm(h, attention(x, layer, cache), weight=n[2], post_weight=n[1])
                h, x = W.block_norm(h, self.mlp(x, layer), weight=n[4], post_weight=n[3])
            return x
        for layer, cache in zip(self.layers, self.caches):
            h = h + attention(rms_norm(h), layer, cache)
            h = h + self.mlp(rms_norm(h), layer)
        return h

    def mlp(self, x: torch.Tensor, layer: dict) -> torch.Tensor:
        if "experts" not in layer:
            return layer["down"](W.silu_mul(layer["gu"](x)))
        return torch.cat([W.moe(x[i:i + 64], layer["experts"], layer["router"], self.top_k, self.moe_workspace)[0]
                          for i in range(0, x.shape[0], 64)])

    def logits(self, h: torch.Tensor) -> torch.Tensor:
        return self.head(h if self.block_norms else rms_norm(h))  # (block norms: the last one is done)

    def prompt(self, tokens: torch.Tensor) -> torch.Tensor:
        """The same number of prompt tokens [streams, n] for every stream; returns the last rows' logits."""
        n = tokens.shape[1]
        stream_of = torch.arange(self.streams, device="cuda").repeat_interleave(n)
        at = torch.arange(n, device="cuda").repeat(self.streams)
        positions = (self.length[stream_of.long()] + at).int()
        self.length += n
        q_start = torch.arange(0, (self.streams + 1) * n, n, dtype=torch.int32, device="cuda")
        h = self.forward(tokens.reshape(-1), stream_of, positions, q_start, n)
        return self.logits(h.view(self.streams, n, -1)[:, -1].contiguous())

    def step(self, tokens: torch.Tensor) -> torch.Tensor:
        """One token of every stream; returns the logits of the next."""
        stream_of = torch.arange(self.streams, device="cuda")
        positions = self.length.clone()
        self.length += 1
        q_start = torch.arange(self.streams + 1, dtype=torch.int32, device="cuda")
        return self.logits(self.forward(tokens, stream_of, positions, q_start, 1))


def generate(model: Decoder, prompt: torch.Tensor, steps: int, u: torch.Tensor, graph: bool = True, scores: torch.Tensor | None = None,
             **settings) -> torch.Tensor:
    """Tokens [steps, streams] after the prompt; u [steps, streams] uniform numbers, settings as of W.sample. scores
    float32 [steps, streams] takes the tokens' log probabilities, before any temperature or cut."""
    out = torch.empty((steps, model.streams), dtype=torch.int32, device="cuda")
    logits = model.prompt(prompt)
    tokens, _ = W.sample(logits, u[0], **settings)
    out[0] = tokens
    token, number = tokens.clone(), torch.empty_like(u[0])
    score = None if scores is None else W.logprobs(logits, token)
    if scores is not None:
        scores[0] = score.logprob

    def one():
        logits = model.step(token)
        W.sample(logits, number, out=(token, probs), **settings)
        if scores is not None:
            W.logprobs(logits, token, out=score)

    probs = torch.empty(model.streams, device="cuda")
    g = None
    for i in range(1, steps):
        number.copy_(u[i])
        if graph and i == 2:  # (the first step ran without: kernels are loaded)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one()
        if g is not None:
            g.replay()
        else:
            one()
        out[i] = token
        if scores is not None:
            scores[i] = score.logprob
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--streams", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=40)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--experts", type=int, default=0, help="experts of a layer instead of its MLP (0: the dense MLP)")
    ap.add_argument("--block-norms", action="store_true", help="a norm before and behind every block")
    a = ap.parse_args()
    model = Decoder(a.layers, a.streams, a.prompt + a.steps, experts=a.experts, block_norms=a.block_norms)
    g = torch.Generator("cuda").manual_seed(1)
    prompt = torch.randint(0, model.vocab, (a.streams, a.prompt), generator=g, device="cuda")
    u = torch.rand((a.steps, a.streams), generator=g, device="cuda")
    ones = torch.ones(a.streams, device="cuda")
    scores = torch.empty_like(u)
    tokens = generate(model, prompt, a.steps, u, scores=scores, temperature=0.8 * ones, top_k=(50 * ones).int(), top_p=0.95 * ones)
    torch.cuda.synchronize()
    status = W.w4a16_device_status()
    print("device status:", W.status_string(status))
    for b in range(a.streams):
        print(f"stream {b} (log probability {float(scores[:, b].sum()):.2f}):", tokens[:, b].tolist())
    return status


if __name__ == "__main__":
    sys.exit(main())
