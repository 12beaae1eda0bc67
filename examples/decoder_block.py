"""One decoder block of a serving step around the routed-expert layer, prompt and decode:

  norm (residual added)  ->  q, k, v projections  ->  cache append  ->  attention  ->  output projection
  norm (residual added, MXFP8 rows)  ->  router  ->  experts  ->  combine

Projections are plain matrix products; everything else is this package's. Run it for a prompt of ragged sequences and a few
decode steps of verification rows each:

    python examples/decoder_block.py [--mxfp8-cache] [--window 128 --sinks 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_scaled_fp8_moe_gb300 import binding as B  # noqa: E402


class PageTable:
    """Hands out a cache's pages to sequences; the table and the lengths live on the device."""

    def __init__(self, cache: B.KvCache, sequences: int, max_len: int):
        self.page_size = cache.page_size
        width = -(-max_len // cache.page_size)
        if sequences * width > cache.pages:
            raise ValueError(f"{sequences} sequences of {max_len} tokens need {sequences * width} pages")
        self.table = torch.arange(sequences * width, dtype=torch.int32, device="cuda").view(sequences, width)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.max_len = max_len

    def slots(self, seq: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
        """Where the tokens at positions `pos` of sequences `seq` are stored."""
        page = self.table[seq, pos // self.page_size]
        return (page * self.page_size + pos % self.page_size).int()


class DecoderBlock:
    def __init__(self, hidden, heads, heads_kv, dim, experts, top_k, inter, window=0, sinks=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=0.02):
            return torch.randn(*shape, generator=g, device="cuda") * std

        self.heads, self.heads_kv, self.dim, self.window, self.sinks = heads, heads_kv, dim, window, sinks
        self.norm1, self.norm2 = ((1 + normal(hidden, std=0.1)).bfloat16() for _ in range(2))
        self.w_qkv = normal(hidden, (heads + 2 * heads_kv) * dim, std=hidden ** -0.5).bfloat16()
        self.w_out = normal(heads * dim, hidden, std=(heads * dim) ** -0.5).bfloat16()
        self.moe = B.MoeLayer.from_fp32(normal(experts, hidden).bfloat16(), normal(experts, std=0.1),
                                        normal(experts, 2 * inter, hidden), normal(experts, hidden, inter), top_k)

    def _attention(self, x, residual, cache, slots, attend):
        """Norm, projections, cache and attention of rows x [T, hidden]; `attend(q, k, v)` is the attention itself."""
        y, residual, _, _ = B.moe_add_rmsnorm_mxfp8(x, self.norm1, residual, quant=False)
        qkv = (y @ self.w_qkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split((self.heads, self.heads_kv, self.heads_kv), dim=1)
        B.moe_kv_append(cache, k, v, slots)
        return attend(q, k, v).view(x.shape[0], -1) @ self.w_out, residual

    def _experts(self, x, residual, dead=None):
        """Norm with MXFP8 rows, router and experts, which read those rows."""
        y, residual, q, s = B.moe_add_rmsnorm_mxfp8(x, self.norm2, residual)
        shp = self.moe.shape(x.shape[0])
        ws = self.moe.workspace(x.shape[0])
        plan = B.moe_route_topk(shp, y, self.moe.w_router, self.moe.bias, dead, ws)
        _, _, rows = B.moe_experts_grouped(shp, q, s, self.moe.w13p, self.moe.w13sp, self.moe.w2p, self.moe.w2sp, plan, ws)
        return B.moe_combine(shp, rows, plan, ws, dead=dead), residual

    def prompt(self, x, residual, cache, slots, cu):
        """Whole prompts, packed one behind the other (bounds cu). Returns the block's output and the residual."""
        attend = lambda q, k, v: B.moe_prefill_attention(q, k, v, cu, window=self.window, sinks=self.sinks)  # noqa: E731
        return self._experts(*self._attention(x, residual, cache, slots, attend))

    def decode(self, x, residual, cache, slots, pages: PageTable, dead=None):
        """The newest rows of every sequence: x [sequences * rows, hidden]; pages.lens counts them already. Dead rows have
        slot -1 and take no expert."""
        seqs = pages.lens.numel()

        def attend(q, k, v):
            return B.moe_paged_attention(q.view(seqs, -1, self.heads, self.dim), cache, pages.table, pages.lens,
                                         pages.max_len, window=self.window, sinks=self.sinks)
        return self._experts(*self._attention(x, residual, cache, slots, attend), dead=dead)


def run(prompt_lens, rows, steps, block, cache, hidden, seed=0, on_step=None):
    """A prompt and `steps` decode steps of `rows` verification rows; of each step's rows the first two are kept."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = len(prompt_lens)
    pages = PageTable(cache, n, max(prompt_lens) + 2 * steps + rows)
    cu = torch.tensor([sum(prompt_lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(prompt_lens, device="cuda"))
    pos = torch.cat([torch.arange(m, device="cuda") for m in prompt_lens])
    x = torch.randn(sum(prompt_lens), hidden, generator=g, device="cuda").bfloat16()
    out, _ = block.prompt(x, None, cache, pages.slots(seq, pos), cu)
    pages.lens += torch.tensor(prompt_lens, dtype=torch.int32, device="cuda")
    outs = [out]
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), rows)
    for step in range(steps):
        pages.lens += rows
        pos = (pages.lens[:, None] - rows + torch.arange(rows, device="cuda")).flatten()
        x = torch.randn(n * rows, hidden, generator=g, device="cuda").bfloat16()
        out, _ = block.decode(x, None, cache, pages.slots(seq, pos), pages)
        outs.append(out)
        if on_step:
            on_step(step, pages)
        pages.lens -= rows - 2                  # two rows accepted: the next step writes over the others
    B.attention_status()
    return outs


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--mxfp8-cache", action="store_true")
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    p.add_argument("--rows", type=int, default=6)
    p.add_argument("--steps", type=int, default=8)
    a = p.parse_args()
    hidden, heads, heads_kv, dim = 4096, 32, 8, 128
    block = DecoderBlock(hidden, heads, heads_kv, dim, 64, 8, 576, a.window, a.sinks)
    cache = B.KvCache.empty(512, 16, heads_kv, dim, mxfp8=a.mxfp8_cache)
    lens = [700, 31, 1, 1200]
    stamps = []
    run(lens, a.rows, 2, block, cache, hidden)          # once for allocations
    begin = torch.cuda.Event(enable_timing=True)

    def stamp(*_):
        stamps.append(torch.cuda.Event(enable_timing=True))
        stamps[-1].record()
    begin.record()
    outs = run(lens, a.rows, a.steps, block, cache, hidden, on_step=stamp)
    torch.cuda.synchronize()
    per = (stamps[-1].elapsed_time(stamps[0]) / -(a.steps - 1)) if a.steps > 1 else float("nan")
    print(f"prompt of {sum(lens)} tokens and first step {begin.elapsed_time(stamps[0]):.2f} ms, then {per * 1e3:.0f} us a step of "
          f"{len(lens)} x {a.rows} rows; last output rms {outs[-1].float().square().mean().sqrt():.4f}")


if __name__ == "__main__":
    main()
