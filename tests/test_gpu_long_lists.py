"""sparse_attention, and prefix_attention with the prefix in front of each list, over lists that are cut over more pairs
of SMs than the device holds at once, so that no accumulator sums more than 131072 records (the tensor cores' sums are cut
off and not rounded: in one sum, a million records came out 0.4 % too small)."""
import numpy as np
import pytest
import torch

import plain_paged as plain
from test_gpu_attention_timeout import ALL_RUN_OUT, SOME_RUN_OUT, libraries  # noqa: F401
from test_gpu_prompt_timeout import check

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = 512 ** -0.5
RUN = 131072


def cache_of(gkr, rows):
    """bf16 rows [n, 512] inserted, and what is read back (double)."""
    n = len(rows)
    cache = gkr.alloc_cache(-(-n // 64), 64, 272, DEV, fill=0)
    csc = torch.cat([torch.ones(8, 32), torch.zeros(8, 32)], 1).to(DEV)
    at = torch.arange(n, device=DEV)
    gkr.kv_insert(rows, cache, at, torch.zeros_like(at), csc, 64)
    return cache, gkr.kv_gather(cache, at.int(), torch.empty(n, 512, dtype=torch.bfloat16, device=DEV)).double()


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)


def check_mean(out, lse, q, k, times):
    """Every record of k (positive values) `times` times for each query: the mean of the relative errors has no other
    reason than sums that are cut off, one last bit (2^-23) at most for each 16 records of a run, and for its first
    ones; each result's error is that and the roundings of probabilities and results."""
    s = SM * torch.einsum("nhd,md->nhm", q.double(), k)
    want = torch.softmax(s, 2) @ k
    off = (out.double() - want) / want
    assert abs(off.mean().item()) <= (RUN / 16 + 16) * 2.0 ** -23 + 2.0 ** -12
    assert off.abs().max().item() <= (RUN / 16 + 16) * 2.0 ** -23 + 2 * 2.0 ** -8 + 2.0 ** -10
    l = torch.logsumexp(s, 2) + np.log(times)
    assert (lse.double() - l).abs().max().item() <= (RUN / 64 + 200) * 2.0 ** -24 + 2.0 ** -10


# queries of one run and a bit, of several, cut anywhere; a tail of a chunk; few heads, few queries
@pytest.mark.parametrize("Q,H,K", [(80, 128, 1000000), (100, 64, 300000), (153, 5, 263000), (3, 128, 11000000), (77, 128, 132000)])
def test_sums_do_not_shrink(gkr, Q, H, K):
    rows = (randn(1000, 512, seed=1).float().abs() + 0.5).to(torch.bfloat16)
    cache, k = cache_of(gkr, rows)
    q = randn(Q, H, 512, seed=2, scale=0.1)
    lists = torch.arange(K, device=DEV, dtype=torch.int32).remainder_(1000).expand(Q, K).contiguous()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = gkr.sparse_attention(q, cache, lists, SM, err_flag=err)
    assert int(err.item()) == 0
    check_mean(out, lse, q, k, K // 1000)
    again = gkr.sparse_attention(q, cache, lists, SM)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_prefix_in_front(gkr):
    rows = (randn(1000, 512, seed=1).float().abs() + 0.5).to(torch.bfloat16)
    cache, k = cache_of(gkr, rows)
    q, L = randn(1, 128, 512, seed=3, scale=0.1), 12000000
    prefix = torch.arange(L, device=DEV, dtype=torch.int32) % 1000
    own = torch.arange(1000, device=DEV, dtype=torch.int32)[None]
    assert gkr.prefix_attention_workspace(128, 1, L, 1000) == gkr.sparse_attention_workspace(128, 1, L + 1000)
    out, lse = gkr.prefix_attention(q, cache, prefix, own, SM)
    check_mean(out, lse, q, k, L // 1000 + 1)


@pytest.mark.parametrize("weighted", [False, True])
def test_holes_and_lists_of_many_lengths(gkr, weighted):
    Q, H, K, slots = 90, 24, 400000, 6400
    cache, k = cache_of(gkr, randn(slots, 512, seed=4))
    g = torch.Generator(device=DEV).manual_seed(5)
    lists = torch.randint(0, slots, (Q, K), generator=g, device=DEV, dtype=torch.int32)
    lists[torch.rand(Q, K, generator=g, device=DEV) < 0.1] = -1
    length = (torch.rand(Q, 1, generator=g, device=DEV) ** 2 * K).long()
    length[0], length[1], length[2], length[-1] = K, 0, 1, K
    lists[torch.arange(K, device=DEV) >= length] = -1
    lists[5, :300000] = -1
    q = randn(Q, H, 512, seed=6, scale=2.0)
    weights = torch.zeros(Q, K, device=DEV) if weighted else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = gkr.sparse_attention(q, cache, lists, SM, weights=weights, err_flag=err)
    assert int(err.item()) == 0
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    for i in (0, 2, 5, 40, 41, Q - 1):
        live = lists[i] >= 0
        kk = k[lists[i][live].long()]
        if len(kk) == 0:
            assert (out[i] == 0).all() and torch.isneginf(lse[i]).all()
            continue
        s = SM * (q[i].double() @ kk.T)
        l = torch.logsumexp(s, 1)
        p = torch.exp(s - l[:, None])
        r = {"out": p @ kk, "lse": l, "mass": p @ kk.abs(), "spread": (SM * (q[i].double().abs() @ kk.abs().T)).amax(1)}
        r = {n: x.cpu().numpy()[None] for n, x in r.items()}
        t_out, t_lse = plain.tolerances(r, min(len(kk), RUN))
        assert (np.abs(out[i].double().cpu().numpy() - r["out"][0]) <= t_out[0]).all(), i
        assert (np.abs(lse[i].double().cpu().numpy() - r["lse"][0]) <= t_lse[0]).all(), i
        if weighted:
            # a term by the logit's and the lse's error, at most 128 additions
            d = np.expm1(2.0 ** -12 * r["spread"][0]).max() + t_lse.max() + 2.0 ** -16
            w = p.sum(0)
            assert ((weights[i][live].double() - w).abs() <= 2 * d * w + 1e-30).all(), i
            assert (weights[i][~live] == 0).all()


@pytest.mark.parametrize("limit", [ALL_RUN_OUT, *SOME_RUN_OUT])
def test_rows_are_right_or_not_written(gkr, libraries, limit):
    Q, H, K = 90, 16, 300000
    cache, _ = cache_of(gkr, randn(6400, 512, seed=7))
    g = torch.Generator(device=DEV).manual_seed(8)
    lists = torch.randint(-100, 6400, (Q, K), generator=g, device=DEV, dtype=torch.int32).clamp_(min=-1)
    q = randn(Q, H, 512, seed=9, scale=2.0)
    ws = torch.zeros(gkr.sparse_attention_workspace(H, Q, K), dtype=torch.uint8, device=DEV)

    def call(out, lse, err):
        gkr.sparse_attention(q, cache, lists, SM, out=out, lse=lse, workspace=ws, err_flag=err)

    def spoil():
        gkr.sparse_attention(q.flip(0).neg(), cache, lists, -SM, workspace=ws)

    check(gkr, libraries, limit, 2, call, spoil, (Q, H))
