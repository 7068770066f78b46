"""The example that runs the MXFP4 cache's operators together, against plain formulas."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import plain_mxfp4 as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example(gkr):
    path = Path(__file__).resolve().parents[1] / "examples" / "budgeted_decode.py"
    spec = importlib.util.spec_from_file_location("budgeted_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("batch,prompt,keep,recent,heads", [(3, 100, 40, 8, 5), (1, 65, 64, 0, 64),
                                                            (2, 33, 1, 1, 128)])
def test_budgeted_decode(gkr, example, batch, prompt, keep, recent, heads):
    rng = np.random.default_rng(prompt)
    steps, window, sm, bs = 5, 3, 512 ** -0.5, 64

    def bf16(*shape):
        bits = plain.bf16_bits(rng.standard_normal(shape))
        return bits, torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).to(DEV)

    csc = example.cos_sin(prompt + steps)
    c = example.BudgetedCache(batch, prompt, keep, recent, csc)
    ps, slots = gkr.page_stride(272, bs), c.cache.shape[0] * bs
    c.prefill(bf16(batch, prompt, 512)[1], bf16(batch, window, heads, 512)[1], sm)
    own = c.slots.cpu().numpy()
    for b in range(batch):
        kept = c.entries[b, :keep].cpu().numpy()
        assert np.isin(kept, own[b]).all() and len(set(kept)) == keep
        assert (np.diff(kept) > 0).all()                       # oldest first
        if recent:
            assert np.array_equal(kept[keep - recent:], own[b, prompt - recent:])
        assert int(c.freed[b, 0]) in set(own[b]) - set(kept)
    for t in range(steps):
        kbits, kv = bf16(batch, 512)
        qbits, q = bf16(batch, heads, 512)
        before, w0, slot = c.entries.cpu().numpy(), c.weights.cpu().numpy(), c.freed.cpu().numpy()
        out = c.step(kv, q, torch.full((batch,), prompt + t, device=DEV), sm)
        host = gkr.cache_bytes(c.cache).cpu().numpy()
        entries = np.concatenate([before[:, :keep], slot.astype(np.int32)], 1)
        # the new records are in the freed slots
        row = csc[prompt + t].cpu().numpy()
        for b in range(batch):
            d, s = plain.encode(plain.rotate(plain.bf16(kbits[b]), row))
            got = plain.record_bytes(host, slot[b], bs, ps)
            assert np.array_equal(got[0][0], d) and np.array_equal(got[1][0], s)
        r = plain.attention(plain.bf16(qbits).astype(np.float64), host, bs, ps, slots, entries, sm)
        t_out, _, t_w = plain.tolerances(r, keep + 1)
        assert (np.abs(out.float().cpu().numpy() - r["out"]) <= t_out).all()
        # what is kept, and with which weights
        kept, kept_w = c.entries[:, :keep].cpu().numpy(), c.weights[:, :keep].cpu().numpy()
        gone = c.freed.cpu().numpy()[:, 0]
        for b in range(batch):
            assert set(kept[b]) | {gone[b]} == set(entries[b]) and gone[b] not in kept[b]
            w = r["p"][b].sum(0) + np.append(w0[b, :keep], 0.0)
            tw = t_w[b] + 2.0 ** -23 * w
            where = [int(np.flatnonzero(entries[b] == x)[0]) for x in kept[b]]
            assert (np.abs(kept_w[b] - w[where]) <= tw[where]).all()
            if recent:
                assert np.array_equal(kept[b, keep - recent:], entries[b, keep + 1 - recent:])
            g = int(np.flatnonzero(entries[b] == gone[b])[0])
            old = [x for x in where if x < keep + 1 - recent]
            assert all(w[g] - tw[g] <= w[x] + tw[x] for x in old)
