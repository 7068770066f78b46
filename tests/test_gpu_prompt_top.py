"""GPU tests of what the rounding of the probabilities does to a row that one record dominates.

A record t has all but a share e of a head's weight, and its logit is above those before it by less
than what makes the running reference move, so its probability is no power of two.  The result is then
K[t] (1 + f), |f| <= e * 2 * max|K| / min|K| + 2^-18 (fp32 sums of at most 2^12 terms, the join of pieces),
if the probabilities are divided by their own sum, rounded as they were multiplied; the values of K lie
in [1, 2], and e is below 2^-12 (checked), so |f| < 2^-9: less than half a step of bf16 from K[t], and the
result has to be K[t] to the bit.  A sum of what was not rounded is off by up to 2^-9 and shows in
the last bit of some head's values (of 64 heads' fractions one at least is above a half of that)."""
import numpy as np
import pytest
import torch

import plain_mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
LAG = 32 * np.log(2.0)          # how far a logit may be above the reference without moving it
SM = 512 ** -0.5


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def heads(rng, K, top):
    """A query head for each record of `top`, as K[t] scaled: its logit is about 21."""
    k = K[top]
    scale = 21.0 * rng.uniform(0.98, 1.02, len(top)) / (SM * (k * k).sum(1))
    return bf16(k * scale[:, None])


def check(q, K, top, first, out, lse):
    """q [n, 512] of dominant records `top`; `first`: of the records K, how many the reference is sure to
    have come from."""
    s = SM * q.double().numpy() @ K.T
    at = s[np.arange(len(top)), top]
    assert (at - s[:, :first].max(1) < LAG - 0.1).all()
    total = np.exp(s - at[:, None]).sum(1)
    assert (total - 1 < 2.0 ** -12).all()
    assert np.abs(K).min() >= 1 and np.abs(K).max() <= 2
    assert np.array_equal(out.float().cpu().numpy(), K[top].astype(np.float32))
    assert np.abs(lse.cpu().numpy() - (at + np.log(total))).max() <= 2.0 ** -11 + 25 * 2.0 ** -22


@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("rows", [300, 3000])
def test_prompt(gkr, H, rows):
    rng = np.random.default_rng(rows + H)
    K = rng.choice([-1.0, 1.0], (rows, 512)) * bf16(rng.uniform(1, 2, (rows, 512))).double().numpy()
    n = 3
    top = rng.integers(128, rows, n * H)
    q = heads(rng, K, top)
    # three requests of one query, which share the rows
    starts = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    kv = bf16(np.concatenate([K] * n)).to(DEV)
    out, lse = gkr.prompt_attention(q.view(n, H, 512).to(DEV), kv, starts, SM, kv_starts=starts * rows)
    check(q, K, top, 128, out.view(-1, 512), lse.view(-1))


@pytest.mark.parametrize("Q,H,L,K", [(2, 64, 500, 300), (32, 32, 4000, 300), (3, 128, 0, 300), (40, 16, 2900, 0)])
@pytest.mark.parametrize("own", [False, True])
def test_prefix(gkr, Q, H, L, K, own):
    if (K if own else L) == 0:
        own = not own
    rng = np.random.default_rng(Q + own)
    bs, pages = 64, (L + K) // 64 + 1
    ps, slots = gkr.page_stride(272, bs), pages * bs
    # codes of 1, 1.5 and 2, both signs, at scale 1
    nib = rng.choice(np.array([2, 3, 4, 10, 11, 12], np.uint8), (2, pages * ps))
    host = nib[0] | nib[1] << 4
    at = np.array([plain_mxfp4.offsets(slot, bs, ps)[1] for slot in range(slots)])
    host[at[:, None] + np.arange(16)] = 127
    cache = gkr.alloc_cache(pages, bs, 272, DEV, page_stride_bytes=ps)
    gkr.cache_bytes(cache).copy_(torch.from_numpy(host))
    order = rng.permutation(slots)[:L + K].astype(np.int32)
    rows = plain_mxfp4.decode(*plain_mxfp4.record_bytes(host, order, bs, ps)).astype(np.float64)
    # the dominant record: past the first chunk of its list
    top = rng.integers(L + 128, L + K, Q * H) if own else rng.integers(128, L, Q * H)
    q = heads(rng, rows, top)
    prefix = torch.from_numpy(order[:L].copy()).to(DEV)
    indices = torch.from_numpy(order[L:].copy()).to(DEV).expand(Q, K).contiguous()
    out, lse = gkr.prefix_attention(q.view(Q, H, 512).to(DEV), cache, prefix, indices, SM)
    check(q, rows, top, 64, out.view(-1, 512), lse.view(-1))
