"""A stack of KDA layers served with the operators of linear_attention_chunked_02_gb300.

    python examples/kda_layers.py [--dtype bfloat16] [--layers 4] [--dim 2048] [--heads 16] [--new-tokens 64]

Prompts of unequal lengths go through every layer packed (add_norm, projections, delta_prefill,
gated_norm, output projection); their states land in a pool, a slot to a request.  Then all requests
generate token by token (delta_step in delta_prefill's place) from a captured CUDA graph.  The weights
are random: the program shows how the operators fit together and what they cost, and checks that a
sequence generated token by token gives what the same tokens give as one prompt.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_attention_chunked_02_gb300 as kda  # noqa: E402


class Layer:
    """Weights of one layer, and the layer over packed prompts or single tokens.

    x [tokens, dim] is the output of the layer before, residual the running sum it belongs to
    (None before the first layer).
    """

    def __init__(self, dim: int, heads: int, width: int, dtype: torch.dtype, device, gen: torch.Generator):
        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5).to(dtype)

        self.heads, self.width = heads, width
        n = heads * width
        self.norm = torch.ones(dim, dtype=dtype, device=device)
        self.head_norm = torch.ones(width, dtype=dtype, device=device)
        self.qkvz = weight(4 * n, dim)                      # queries, keys, values, output gate
        self.decay = weight(n, dim)
        self.beta = weight(heads, dim)
        self.out = weight(dim, n)
        self.rate = torch.rand(heads, 1, generator=gen, device=device) * 0.1 + 0.01

    def inputs(self, x, residual):
        y, residual = kda.add_norm(x, residual, self.norm)
        q, k, v, z = (y @ self.qkvz.T).view(-1, 4, self.heads, self.width).unbind(1)
        q, k = F.normalize(q.float(), dim=-1).to(x.dtype), F.normalize(k.float(), dim=-1).to(x.dtype)
        g = -self.rate * F.softplus((y @ self.decay.T).float().view(-1, self.heads, self.width))
        beta = torch.sigmoid((y @ self.beta.T).float()).to(x.dtype)
        return (q, k, v, g, beta), z, residual

    def finish(self, o, z):
        return kda.gated_norm(o, z, self.head_norm).view(o.shape[0], -1) @ self.out.T

    def prefill(self, x, residual, cu_seqlens, pool, slots, fresh: bool):
        """cu_seqlens int32 [N + 1]; the requests' states go to pool [entries, heads, width, width]."""
        (q, k, v, g, beta), z, residual = self.inputs(x, residual)
        if fresh:                                           # no state yet: the slots hold another request's
            pool.index_fill_(0, slots.long(), 0.0)
        o, _ = kda.delta_prefill(q[None], k[None], v[None], g[None], beta[None], cu_seqlens, initial_state=pool,
                                 slots=slots)
        return self.finish(o[0], z), residual

    def step(self, x, residual, pool, slots):
        (q, k, v, g, beta), z, residual = self.inputs(x, residual)
        return self.finish(kda.delta_step(q, k, v, g, beta, pool, slots), z), residual


class Model:
    def __init__(self, layers: int, dim: int, heads: int, width: int, entries: int, dtype: torch.dtype, device="cuda",
                 seed: int = 0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.layers = [Layer(dim, heads, width, dtype, device, gen) for _ in range(layers)]
        self.pools = [torch.zeros(entries, heads, width, width, device=device) for _ in range(layers)]
        self.norm = torch.ones(dim, dtype=dtype, device=device)

    def prefill(self, x, cu_seqlens, slots, fresh: bool = True):
        residual = None
        for layer, pool in zip(self.layers, self.pools):
            x, residual = layer.prefill(x, residual, cu_seqlens, pool, slots, fresh)
        return kda.add_norm(x, residual, self.norm)[0]

    def step(self, x, slots):
        residual = None
        for layer, pool in zip(self.layers, self.pools):
            x, residual = layer.step(x, residual, pool, slots)
        return kda.add_norm(x, residual, self.norm)[0]


def run(dtype=torch.bfloat16, layers=4, dim=2048, heads=16, width=128, lengths=(700, 33, 512, 1, 250), new_tokens=64,
        device="cuda", seed=0):
    """Serves the prompts; returns ({name: figure}, the largest deviation relative to the largest output)."""
    model = Model(layers, dim, heads, width, len(lengths) + 3, dtype, device, seed)
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    requests = len(lengths)
    slots = (torch.randperm(requests + 3, generator=gen, device=device)[:requests]).to(torch.int32)
    cu = torch.tensor([0, *lengths], device=device).cumsum(0).to(torch.int32)
    prompt = torch.randn(int(cu[-1]), dim, generator=gen, device=device).to(dtype)
    # the tokens that follow: here given, so that both ways see the same
    follow = torch.randn(new_tokens, requests, dim, generator=gen, device=device).to(dtype)

    def timed(fn, n):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        fn()
        start.record()
        for _ in range(n):
            fn()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) / n

    figures = {"prefill ms": timed(lambda: model.prefill(prompt, cu, slots), 3)}
    model.prefill(prompt, cu, slots)
    # the decode step as a graph over fixed buffers
    token = follow[0].clone()
    kept = [p.clone() for p in model.pools]
    side = torch.cuda.Stream(device)
    side.wait_stream(torch.cuda.current_stream(device))
    with torch.cuda.stream(side):
        model.step(token, slots)                            # warm-up: the libraries' own first calls
    torch.cuda.current_stream(device).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = model.step(token, slots)
    figures["step ms"] = timed(graph.replay, 20)
    for pool, was in zip(model.pools, kept):                # the warm-up and timing steps are taken back
        pool.copy_(was)
    outputs = []
    for t in range(new_tokens):
        token.copy_(follow[t])
        graph.replay()
        outputs.append(result.clone())
    # the same tokens as prompts
    whole = torch.cat([torch.cat([prompt[int(cu[n]):int(cu[n + 1])], follow[:, n]]) for n in range(requests)])
    cu2 = cu + new_tokens * torch.arange(requests + 1, device=device, dtype=torch.int32)
    ref = model.prefill(whole, cu2, slots)
    worst, largest = 0.0, float(ref.float().abs().max())
    for n in range(requests):
        tail = ref[int(cu2[n + 1]) - new_tokens:int(cu2[n + 1])]
        worst = max(worst, float((torch.stack(outputs)[:, n].float() - tail.float()).abs().max()))
    return figures, worst / largest


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", default="bfloat16", choices=("float32", "bfloat16", "float16"))
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--dim", type=int, default=2048)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--new-tokens", type=int, default=64)
    a = ap.parse_args()
    figures, off = run(getattr(torch, a.dtype), a.layers, a.dim, a.heads, new_tokens=a.new_tokens)
    for name, value in figures.items():
        print(f"{name}: {value:.3f}")
    print(f"token by token against one prompt: {off:.2e} of the largest output")


if __name__ == "__main__":
    main()
