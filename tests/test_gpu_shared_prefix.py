"""The example that runs page allocation, slot lists and both attentions together, against plain
formulas over what its cache holds."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import plain_mxfp4
import plain_paged as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example(gkr):
    path = Path(__file__).resolve().parents[1] / "examples" / "shared_prefix_serving.py"
    spec = importlib.util.spec_from_file_location("shared_prefix_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("batch,prefix,prompt,heads", [(3, 128, 70, 5), (20, 1024, 3, 16), (1, 64, 1, 128)])
def test_shared_prefix(gkr, example, batch, prefix, prompt, heads):
    rng = np.random.default_rng(prefix)
    steps, sm, bs = 4, 512 ** -0.5, 64

    def bf16(*shape):
        return torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16).to(DEV)

    csc = example.cos_sin(prefix + prompt + steps)
    c = example.SharedPrefixBatch(batch, bf16(prefix, 512), prompt + steps, csc, sm)
    ps = gkr.page_stride(272, bs)

    def rows(b):
        """What request b's cache holds: its prefix and its own, every slot once."""
        n = int(c.lengths[b].item())
        pos = np.arange(n)
        slots = c.table[b].cpu().numpy()[pos // bs] * bs + pos % bs
        assert (slots >= 0).all() and len(set(slots)) == n
        host = gkr.cache_bytes(c.cache).cpu().numpy()
        return slots, plain_mxfp4.decode(*plain_mxfp4.record_bytes(host, slots, bs, ps))

    def check(out, q, keys, see):
        r = plain.attend(q.double().cpu().numpy(), keys, see, sm)
        assert (np.abs(out.float().cpu().numpy() - r["out"]) <= plain.tolerances(r, len(keys))[0]).all()

    q = 2 * bf16(batch, prompt, heads, 512)
    out = c.prompts(bf16(batch, prompt, 512), q)
    owned = []
    for b in range(batch):
        slots, keys = rows(b)
        owned.append(set(slots[prefix:]))
        assert np.array_equal(slots[:prefix], c.prefix.cpu().numpy())
        check(out[b], q[b], keys, prefix + 1 + np.arange(prompt))
    assert len(set().union(*owned)) == batch * prompt        # no request writes over another's
    for _ in range(steps):
        q = 2 * bf16(batch, heads, 512)
        out = c.step(bf16(batch, 512), q)
        for b in range(batch):
            _, keys = rows(b)
            check(out[b:b + 1], q[b:b + 1], keys, [len(keys)])
