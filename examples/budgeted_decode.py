"""Decode over a 4-bit KV cache that keeps a fixed number of records of each sequence.

A prompt is written as MXFP4 records (272 bytes a token, 528 in the MXFP8 cache).  Its last
queries attend to all of it and say which records matter; kv_evict keeps `keep` of them, the
`recent` newest among them.  Then each step writes the new token into the slot that the last
eviction freed, attends to the keep + 1 records and evicts one: memory and time of a step no
longer grow with the sequence.

    python examples/budgeted_decode.py [--batch 8] [--heads 32] [--prompt 4096] [--keep 2048]
                                       [--recent 256] [--steps 64]

The latents and queries are random, as there is no model here; a decode step of a model calls
BudgetedCache.step with its own, and multiplies the output by its value projection.
"""
import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import gather_kv_rope_gb300 as gkr  # noqa: E402


class BudgetedCache:
    """A pool of MXFP4 pages and, for each sequence, the list of its records, oldest first."""

    def __init__(self, batch, prompt, keep, recent, cos_sin_cache, block_size=64, device="cuda"):
        pages = -(-prompt // block_size)
        self.batch, self.keep, self.recent, self.block_size = batch, keep, recent, block_size
        self.cos_sin_cache = cos_sin_cache
        self.cache = gkr.alloc_cache(batch * pages, block_size, gkr.MXFP4, device, fill=0)
        first = torch.arange(batch, device=device)[:, None] * pages * block_size
        self.slots = first + torch.arange(prompt, device=device)            # int64 [batch, prompt]
        # list and weights of a step: what was kept, then the new token
        self.entries = torch.full((batch, keep + 1), -1, dtype=torch.int32, device=device)
        self.weights = torch.zeros(batch, keep + 1, device=device)
        self.freed = None                                                   # int64 [batch, 1]

    def _insert(self, kv, slots, positions):
        gkr.kv_insert(kv, self.cache, slots.reshape(-1), positions.reshape(-1),
                      self.cos_sin_cache, self.block_size)

    def _evict(self, entries, weights):
        kept, kept_weights, freed = gkr.kv_evict(entries, weights, self.keep, self.recent)
        self.entries[:, :self.keep] = kept
        self.weights[:, :self.keep] = kept_weights
        return freed

    def prefill(self, kv, q_last, sm_scale):
        """kv bf16 [batch, prompt, 512]; q_last bf16 [batch, window, heads, 512], rotated queries
        of the prompt's last positions."""
        batch, prompt, _ = kv.shape
        if prompt <= self.keep:
            raise ValueError("the prompt must be longer than what is kept")
        window, heads = q_last.shape[1:3]
        positions = torch.arange(prompt, device=kv.device).expand(batch, prompt).contiguous()
        self._insert(kv.reshape(-1, 512), self.slots, positions)
        entries = self.slots.to(torch.int32)
        # one row a query; a query does not see what comes after it
        rows = entries[:, None, :].expand(batch, window, prompt)
        behind = torch.arange(prompt, device=kv.device) - (prompt - window)
        rows = rows.masked_fill(behind > torch.arange(window, device=kv.device)[:, None], -1)
        weights = torch.zeros(batch * window, prompt, device=kv.device)
        gkr.sparse_attention(q_last.reshape(-1, heads, 512), self.cache,
                             rows.reshape(-1, prompt), sm_scale, weights=weights)
        freed = self._evict(entries, weights.view(batch, window, prompt).sum(1))
        self.freed = freed[:, :1].contiguous()   # the other freed slots could serve new sequences

    def step(self, kv, q, position, sm_scale):
        """kv bf16 [batch, 512], q bf16 [batch, heads, 512] (rotated), position int64 [batch];
        returns the attention's output [batch, heads, 512] over the records that are kept."""
        self._insert(kv, self.freed, position)
        self.entries[:, self.keep:] = self.freed
        self.weights[:, self.keep:] = 0
        out, _ = gkr.sparse_attention(q, self.cache, self.entries, sm_scale, weights=self.weights)
        self.freed = self._evict(self.entries, self.weights)
        return out


def cos_sin(max_pos, device="cuda"):
    freq = 10000.0 ** (-torch.arange(32, device=device, dtype=torch.float64) / 32)
    angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    for name, value in (("batch", 8), ("heads", 32), ("prompt", 4096), ("keep", 2048),
                        ("recent", 256), ("window", 16), ("steps", 64)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    gkr.build()
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    sm_scale = 512 ** -0.5
    c = BudgetedCache(a.batch, a.prompt, a.keep, a.recent, cos_sin(a.prompt + a.steps))
    c.prefill(randn(a.batch, a.prompt, 512), randn(a.batch, a.window, a.heads, 512), sm_scale)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    warm = min(3, a.steps - 1)
    for t in range(a.steps):
        if t == warm:
            begin.record()
        position = torch.full((a.batch,), a.prompt + t, device="cuda")
        out = c.step(randn(a.batch, 512), randn(a.batch, a.heads, 512), position, sm_scale)
    end.record()
    torch.cuda.synchronize()
    mib = a.batch * (a.keep + 1) * gkr.MXFP4 / 2 ** 20
    print(f"{a.steps} steps, {a.batch} sequences of {a.prompt + a.steps} tokens, {a.keep} + 1 records "
          f"each ({mib:.1f} MiB): {begin.elapsed_time(end) / (a.steps - warm) * 1e3:.0f} us a step, "
          f"output norm {out.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
