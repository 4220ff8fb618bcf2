"""A small decoder of attention and mixture-of-experts layers that answers a batch of prompts.

The layers that the pages describe side by side, run as a serving program runs them: the packed
prompts go through attn_prefill, their keys and values into the paged cache (kv_append), and the
rows through the Q4 experts (prefill); then every step appends one token per sequence, attends to
the cache (attn_decode) and runs the experts' small-batch decode, the whole step captured once in a
CUDA graph. Weights are random, the next token is the largest logit against the embedding, and the
projections are plain torch products.

    python examples/generate.py [--e4m3] [--steps 16]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_grouped_gemm_router_gb300 as moe  # noqa: E402
from synthetic import LayerShape, make_layer  # noqa: E402

BF16 = torch.bfloat16


def bits(x: torch.Tensor) -> torch.Tensor:
    """bf16 values as the int16 bit patterns that the library takes."""
    return x.view(torch.int16)


def norm(x: torch.Tensor) -> torch.Tensor:
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(BF16)


class Block:
    """One layer: attention over a cache of its own, then the experts."""

    def __init__(self, dims: moe.AttnDims, shape: LayerShape, seed: int, n_pages: int, page: int, e4m3: bool):
        g = torch.Generator(device="cuda").manual_seed(seed)
        hq, hkv, dh = dims.n_q_heads, dims.n_kv_heads, dims.head_dim

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)).to(BF16)

        self.dims, self.heads = dims, (hq, hkv, dh)
        self.w_qkv, self.w_o = weight((hq + 2 * hkv) * dh, shape.d), weight(shape.d, hq * dh)
        self.experts = moe.upload_layer(make_layer(shape, seed=seed))
        # e4m3 holds up to 448 scale: keys and values here are of size 1, and 7 is far out
        scale = torch.full((hkv,), 1 / 64, device="cuda") if e4m3 else None
        self.cache = moe.KvCache.empty(dims, n_pages, page, scale, scale)

    def qkv(self, x: torch.Tensor):
        hq, hkv, dh = self.heads
        rows = bits(norm(x) @ self.w_qkv.t()).view(-1, hq + 2 * hkv, dh)
        return rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]

    def project(self, x: torch.Tensor, o: torch.Tensor) -> torch.Tensor:
        return x + o.view(BF16).reshape(x.shape[0], -1) @ self.w_o.t()

    def prompts(self, x, cu, start, table, attn_ws, moe_ws):
        q, k, v = self.qkv(x)
        moe.kv_append(self.cache, k, v, cu, start, table, attn_ws)
        x = self.project(x, moe.attn_prefill(self.dims, q, k, v, cu, cu, attn_ws))
        return x + moe.prefill(self.experts, bits(norm(x)), moe_ws).view(BF16)

    def token(self, x, cu, start, lens, table, attn_ws, moe_ws):
        q, k, v = self.qkv(x)
        moe.kv_append(self.cache, k, v, cu, start, table, attn_ws)
        x = self.project(x, moe.attn_decode(self.cache, q, lens, table, attn_ws))
        return x + moe.decode_batch(self.experts, bits(norm(x)), moe_ws).view(BF16)


class Decoder:
    def __init__(self, dims: moe.AttnDims, shape: LayerShape, layers: int, vocab: int, batch: int, longest: int,
                 page: int = 16, e4m3: bool = False, seed: int = 0):
        per = (longest + page - 1) // page
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn(vocab, shape.d, generator=g, device="cuda").to(BF16)
        self.blocks = [Block(dims, shape, 1000 * (seed + 1) + i, batch * per, page, e4m3) for i in range(layers)]
        # pages are handed out in a scattered order, as a running server's are
        order = torch.randperm(batch * per, generator=g, device="cuda").to(torch.int32)
        self.table = order.view(batch, per).contiguous()
        self.attn_ws = moe.attn_workspace(dims)
        self.dims, self.shape, self.batch, self.longest = dims, shape, batch, longest
        self.cu_one = torch.arange(batch + 1, dtype=torch.int32, device="cuda")

    def logits(self, x: torch.Tensor) -> torch.Tensor:
        return norm(x).float() @ self.embed.float().t() / math.sqrt(self.shape.d)

    def prefill(self, prompts: list[list[int]]) -> torch.Tensor:
        """Logits of each prompt's last token; the caches hold the prompts afterwards."""
        lens = [len(p) for p in prompts]
        if not all(lens):
            raise ValueError("a prompt has at least one token")
        cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        start = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        x = self.embed[torch.tensor([t for p in prompts for t in p], device="cuda")]
        ws = moe.workspace(self.blocks[0].experts.dims, len(x))
        for b in self.blocks:
            x = b.prompts(x, cu, start, self.table, self.attn_ws, ws)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return self.logits(x[cu[1:].long() - 1])

    def step(self, tokens: torch.Tensor, ws: torch.Tensor) -> torch.Tensor:
        """One token per sequence (written to the caches): its logits. self.lens grows by one."""
        start = self.lens.clone()
        self.lens += 1
        x = self.embed[tokens]
        for b in self.blocks:
            x = b.token(x, self.cu_one, start, self.lens, self.table, self.attn_ws, ws)
        return self.logits(x)

    def generate(self, prompts: list[list[int]], steps: int) -> tuple[torch.Tensor, torch.Tensor]:
        """The tokens that follow the prompts [batch, steps] and the logits of the last step."""
        longest = max(len(p) for p in prompts) + steps
        if len(prompts) != self.batch or longest > self.longest:
            raise ValueError(f"{self.batch} prompts that end within {self.longest} tokens are wanted")
        if steps < 1:
            raise ValueError("at least one token follows a prompt")
        logits = self.prefill(prompts)
        ws = moe.workspace(self.blocks[0].experts.dims, self.batch)
        tokens = logits.argmax(-1)
        out = [tokens.clone()]
        if steps > 1:
            kept = self.lens.clone()
            side = torch.cuda.Stream()  # one step outside the graph first: every kernel is loaded
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.step(tokens, ws)
                self.lens.copy_(kept)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                logits = self.step(tokens, ws)
                tokens.copy_(logits.argmax(-1))
            for _ in range(steps - 1):
                graph.replay()
                out.append(tokens.clone())
        for w in (ws, self.attn_ws):
            status = moe.read_device_status(w)
            if status:
                raise moe.MoeError(status, "generate")
        return torch.stack(out, 1), logits


def small(e4m3: bool = False) -> Decoder:
    return Decoder(moe.AttnDims(8, 2, 64), LayerShape(d=256, n_experts=16, top_k=2, inter=128, shared_inter=128), layers=2,
                   vocab=1000, batch=3, longest=256, e4m3=e4m3)


def some_prompts(seed: int = 0) -> list[list[int]]:
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 1000, (n,), generator=g).tolist() for n in (70, 1, 33)]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--e4m3", action="store_true", help="keep the cache in 8 bits")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    prompts = some_prompts()
    model = small(a.e4m3)
    tokens, logits = model.generate(prompts, a.steps)
    for p, t in zip(prompts, tokens.tolist()):
        print(f"{len(p)} tokens ->", t)
    # the last step's logits once more, from the whole texts as prompts
    again = model.prefill([p + t[:-1] for p, t in zip(prompts, tokens.tolist())])
    print("last logits, step by step against whole prompts: largest difference %.3g (of %.3g)" %
          ((logits - again).abs().max().item(), again.abs().max().item()))


if __name__ == "__main__":
    main()
