"""prefix_attention over drawn sizes, so that it takes each of its ways (every list with the prefix in
front, whole or cut; the prefix once, with and without own lists, its tiles whole or cut), against the plain
form in 64 bits on the GPU, within the tolerances of plain_paged."""
import numpy as np
import pytest
import torch

import plain_mxfp4
import plain_paged as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEEDS = 60
BS, PAGES = 64, 50


def drawn(seed):
    rng = np.random.default_rng(1000 + seed)
    log = lambda lo, hi: int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))  # noqa: E731
    H = int(rng.choice([1, 2, 5, 16, 31, 64, 127, 128]))
    many = rng.random() < 0.6               # many queries, a prefix as long as 6e9 multiply-adds allow
    Q = log(30, 1500) if many else log(1, 1500)
    L = int(min(9000, 1.2e7 / (Q * H)) * (1 - 0.5 * rng.random())) if many else log(1, 1000)
    K = 0 if rng.random() < 0.15 else log(1, max(2, min(1500, 4e6 / Q)))
    if rng.random() < 0.1:
        L = 0
    return Q, H, L, K, rng


def test_both_ways_are_drawn(gkr):
    way = [gkr.prefix_attention_workspace(H, Q, L, K) != gkr.sparse_attention_workspace(H, Q, L + K)
           for Q, H, L, K, _ in map(drawn, range(SEEDS))]
    assert 15 <= sum(way) <= SEEDS - 15, sum(way)


@pytest.mark.parametrize("seed", range(SEEDS))
def test_drawn(gkr, seed):
    Q, H, L, K, rng = drawn(seed)
    ps, slots = gkr.page_stride(272, BS), PAGES * BS
    host = rng.integers(0, 256, PAGES * ps, dtype=np.uint8)
    at = np.array([plain_mxfp4.offsets(s, BS, ps)[1] for s in range(slots)])
    host[at[:, None] + np.arange(16)] = np.clip(127 + np.round(rng.standard_normal((slots, 16)) - 1.5), 0, 254)
    cache = gkr.alloc_cache(PAGES, BS, 272, DEV, page_stride_bytes=ps)
    gkr.cache_bytes(cache).copy_(torch.from_numpy(host))
    rows = torch.from_numpy(plain_mxfp4.decode(*plain_mxfp4.record_bytes(host, np.arange(slots), BS, ps))).to(DEV)
    holes = rng.choice([0.0, 0.1, 0.9])
    prefix = np.where(rng.random(L) < holes, -1, rng.integers(0, slots, L)).astype(np.int32)
    idx = rng.integers(0, slots, (Q, K)).astype(np.int32)
    idx[np.arange(K) >= np.ceil(rng.random((Q, 1)) ** 2 * K)] = -1      # lists of different lengths, some empty
    prefix, idx = torch.from_numpy(prefix).to(DEV), torch.from_numpy(idx).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = (2 * torch.randn(Q, H, 512, generator=g, device=DEV)).to(torch.bfloat16)
    sm = 512 ** -0.5
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = gkr.prefix_attention(q, cache, prefix, idx, sm, err_flag=err)
    assert int(err.item()) == 0
    shared = rows[prefix[prefix >= 0].long()]
    some = sorted({0, Q - 1, *rng.integers(0, Q, 40).tolist()})
    for i in some:
        k = torch.cat([shared, rows[idx[i][idx[i] >= 0].long()]])
        got, l = out[i].double().cpu().numpy(), lse[i].double().cpu().numpy()
        if len(k) == 0:
            assert (got == 0).all() and np.isneginf(l).all()
            continue
        qq = q[i].double()
        s = sm * (qq @ k.T)
        w = torch.logsumexp(s, 1)
        p = torch.exp(s - w[:, None])
        r = {"out": p @ k, "lse": w, "mass": p @ k.abs(), "spread": (sm * (qq.abs() @ k.abs().T)).amax(1)}
        r = {name: x.cpu().numpy()[None] for name, x in r.items()}
        t_out, t_lse = plain.tolerances(r, L + K)
        assert (np.abs(l - r["lse"][0]) <= t_lse[0]).all(), (Q, H, L, K, i)
        assert (np.abs(got - r["out"][0]) <= t_out[0]).all(), (Q, H, L, K, i)
