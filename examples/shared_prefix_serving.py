"""Serve requests that share a long prefix (a document, a system prompt) over one MXFP4 cache.

The prefix is written once, and the block table of every request begins with its pages.  A request's
prompt takes pages of its own (kv_allocate), is written (kv_insert) and attends to the prefix and to
itself (kv_slots_packed, kv_gather, prompt_attention).  Then each step writes one token of every
request and attends to the prefix, once for all of them, and to each request's own records
(kv_slots, prefix_attention).  Lengths, tables and lists stay on the GPU.

    python examples/shared_prefix_serving.py [--batch 32] [--heads 16] [--prefix 16384]
                                             [--prompt 200] [--steps 64]

The latents and queries are random, as there is no model here; a model calls SharedPrefixBatch's
methods with its own, and multiplies the outputs by its value projection.
"""
import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import gather_kv_rope_gb300 as gkr  # noqa: E402


class SharedPrefixBatch:
    """A pool of MXFP4 pages, the prefix's pages, and for each request its table and length."""

    def __init__(self, batch, prefix_kv, most, cos_sin_cache, sm_scale, block_size=64):
        """prefix_kv bf16 [tokens, 512], tokens a multiple of block_size (what is left over is part of
        every request's own prompt); most: tokens that a request can get besides."""
        dev, bs = prefix_kv.device, block_size
        if prefix_kv.shape[0] % bs:
            raise ValueError("the shared prefix must fill its pages")
        self.shared, own = prefix_kv.shape[0] // bs, -(-most // bs)
        self.block_size, self.csc, self.sm_scale = bs, cos_sin_cache, sm_scale
        self.cache = gkr.alloc_cache(self.shared + batch * own, bs, gkr.MXFP4, dev, fill=0)
        self.table = torch.full((batch, self.shared + own), -1, dtype=torch.int32, device=dev)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.free = torch.arange(self.cache.shape[0], dtype=torch.int32, device=dev)
        self.most = most
        self._append(prefix_kv[None], self.table[:1], self.lengths[:1], prefix_kv.shape[0])
        self.table[1:, :self.shared] = self.table[0, :self.shared]
        self.lengths[:] = prefix_kv.shape[0]
        self.own_first = self.lengths.clone()
        self.prefix = gkr.kv_slots(self.table[:1], self.lengths[:1], bs, prefix_kv.shape[0])[0]

    def _append(self, kv, table, lengths, tokens):
        """kv bf16 [requests, tokens, 512] behind what the requests hold; returns where each one's
        tokens begin in a packed batch."""
        added = torch.full_like(lengths, tokens)
        slots, positions, starts, taken = gkr.kv_allocate(lengths, added, table, self.free, self.block_size,
                                                          kv.shape[0] * tokens)
        gkr.kv_insert(kv.reshape(-1, 512), self.cache, slots, positions, self.csc, self.block_size)
        # the list moves on by what was taken (a rotation, so that its length stays)
        at = torch.arange(len(self.free), device=kv.device)
        self.free = self.free[(at + taken) % len(self.free)]
        lengths += tokens
        return starts

    def prompts(self, kv, q):
        """kv bf16 [batch, tokens, 512], q bf16 [batch, tokens, heads, 512] (rotated); returns the
        attention's output, q's shape."""
        batch, tokens, heads, _ = q.shape
        starts = self._append(kv, self.table, self.lengths, tokens)
        total = batch * (self.shared * self.block_size + tokens)
        idx, kv_starts = gkr.kv_slots_packed(self.table, self.lengths, self.block_size, total)
        rows = gkr.kv_gather(self.cache, idx, torch.empty(total, 512, dtype=torch.bfloat16, device=kv.device))
        out, _ = gkr.prompt_attention(q.view(-1, heads, 512), rows, starts, self.sm_scale, kv_starts=kv_starts)
        return out.view_as(q)

    def step(self, kv, q):
        """kv bf16 [batch, 512], q bf16 [batch, heads, 512] (rotated); returns the output, q's shape."""
        self._append(kv[:, None], self.table, self.lengths, 1)
        own = gkr.kv_slots(self.table, self.lengths, self.block_size, self.most, first=self.own_first)
        return gkr.prefix_attention(q, self.cache, self.prefix, own, self.sm_scale)[0]


def cos_sin(max_pos, device="cuda"):
    freq = 10000.0 ** (-torch.arange(32, device=device, dtype=torch.float64) / 32)
    angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    for name, value in (("batch", 32), ("heads", 16), ("prefix", 16384), ("prompt", 200), ("steps", 64)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    gkr.build()
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    most = a.prompt + a.steps
    c = SharedPrefixBatch(a.batch, randn(a.prefix, 512), most, cos_sin(a.prefix + most), 512 ** -0.5)
    c.prompts(randn(a.batch, a.prompt, 512), randn(a.batch, a.prompt, a.heads, 512))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    warm = min(3, a.steps - 1)
    for t in range(a.steps):
        if t == warm:
            begin.record()
        out = c.step(randn(a.batch, 512), randn(a.batch, a.heads, 512))
    end.record()
    torch.cuda.synchronize()
    print(f"{a.steps} steps of {a.batch} requests behind {a.prefix} shared tokens: "
          f"{begin.elapsed_time(end) / (a.steps - warm) * 1e3:.0f} us a step, "
          f"output norm {out.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
