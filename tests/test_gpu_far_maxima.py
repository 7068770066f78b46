"""GPU tests of sparse_attention, prefix_attention and prompt_attention where the maximum moves by more powers of
two than fp32 has below 1, and what came before it still shows in the result.

In the order in which the entries are read, each filling whole chunks: logits -104, then -84, then 0.  The second
ones are less than the running reference's lag (32 powers of two) above the first, so sums relative to -104 hold
terms of 2^28.9, and the third moves the reference by 150 powers of two.  In dims 32 to 511 only the second ones
have values, so the result there is their weight, 2^-121.2, times those: a normal bf16.  Tolerances are plain_paged's."""
import numpy as np
import pytest
import torch

import plain_mxfp4
import plain_paged as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
# logits as sums of an MXFP4 block's values at one scale
KINDS = {-104: (-96.0, -8.0, 0.0), -84: (-48.0, -32.0, -4.0), 0: (0.0, 0.0, 0.0)}


def row(logit):
    x = np.zeros(512, np.float32)
    x[:3] = KINDS[logit]
    if logit == -84:
        x[32:] = np.array([1, -1.5, 2, 3, -4, 6], np.float32)[np.arange(480) % 6]
    return x


def order(first, second, third):
    return np.array([-104] * first + [-84] * second + [0] * third)


def cache_of(gkr):
    """A page of 64 slots: 0, 1, 2 hold the three kinds of records."""
    ps = gkr.page_stride(272, 64)
    host = np.zeros(ps, np.uint8)
    for slot, logit in enumerate(KINDS):
        d, s = plain_mxfp4.encode(row(logit))
        at, sat = plain_mxfp4.offsets(slot, 64, ps)
        host[at:at + 256], host[sat:sat + 16] = d, s
        assert np.array_equal(plain_mxfp4.decode(d[None], s[None])[0], row(logit))
    cache = gkr.alloc_cache(1, 64, 272, DEV, page_stride_bytes=ps)
    gkr.cache_bytes(cache).copy_(torch.from_numpy(host))
    return cache


def slots_of(logits):
    return torch.tensor([list(KINDS).index(x) for x in logits], dtype=torch.int32, device=DEV)


def query(Q, H):
    q = torch.zeros(Q, H, 512, dtype=torch.bfloat16, device=DEV)
    q[..., :3] = 1.0
    return q


def check(logits, out, lse):
    """All queries and heads are alike."""
    q = np.zeros((1, 1, 512))
    q[..., :3] = 1.0
    r = plain.attend(q, np.stack([row(x) for x in logits]).astype(np.float64), [len(logits)], 1.0)
    t_out, t_lse = plain.tolerances(r, len(logits))
    assert (np.abs(r["out"][0, 0, 32:]) > 2.0 ** -126).all() and (t_out[0, 0, 32:] < 0.2 * np.abs(r["out"][0, 0, 32:])).all()
    got, l = out.double().cpu().numpy().reshape(-1, 512), lse.double().cpu().numpy().reshape(-1)
    assert (np.abs(l - r["lse"][0, 0]) <= t_lse[0, 0]).all()
    worst = np.abs(got - r["out"][0, 0]) - t_out[0, 0]
    assert (worst <= 0).all(), (got[0, 32], r["out"][0, 0, 32])


@pytest.mark.parametrize("Q,H", [(1, 1), (3, 128), (200, 20)])
def test_sparse_attention(gkr, Q, H):
    logits = order(64, 64, 64)
    lists = slots_of(logits).expand(Q, -1).contiguous()
    out, lse = gkr.sparse_attention(query(Q, H), cache_of(gkr), lists, 1.0)
    check(logits, out, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,H", [(1, 1), (1, 128), (80, 128)])
def test_prompt_attention(gkr, causal, n, H):
    logits = order(128, 128, 128)
    kv = torch.from_numpy(np.stack([row(x) for x in logits])).to(torch.bfloat16).to(DEV)
    starts = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    out, lse = gkr.prompt_attention(query(n, H), kv.repeat(n, 1), starts, 1.0, kv_starts=starts * len(logits), causal=causal)
    check(logits, out, lse)


# every list with the prefix in front; the prefix once, alone and beside own lists that the maximum is in, or all
@pytest.mark.parametrize("Q,H,parts,own", [
    (2, 16, (64, 64, 64), 64), (9000, 1, (128, 128, 128), 0), (9000, 1, (128, 128, 192), 64), (1400, 1, (65, 64, 64), 192)])
def test_prefix_attention(gkr, Q, H, parts, own):
    logits = order(*parts)
    slots = slots_of(logits)
    L = len(logits) - own
    written = gkr.prefix_attention_workspace(H, Q, L, own) == gkr.sparse_attention_workspace(H, Q, L + own)
    assert written == (Q == 2)
    lists = slots[L:].expand(Q, own).contiguous()
    out, lse = gkr.prefix_attention(query(Q, H), cache_of(gkr), slots[:L].contiguous(), lists, 1.0)
    check(logits, out, lse)
