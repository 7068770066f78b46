"""prompt_attention over drawn batches: numbers and lengths of requests, heads, masks and gaps, so that tiles
are cut, left whole or empty in many ways; against the plain form in 64 bits on the GPU, within the
tolerances of plain_paged."""
import numpy as np
import pytest
import torch

import plain_paged as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def drawn(seed):
    rng = np.random.default_rng(seed)
    H = int(rng.choice([1, 2, 5, 16, 31, 64, 128, 129, 200, 500]))
    B = int(rng.choice([1, 2, 7, 31, 33, 50, 64, 65, 150, 700]))
    most = max(1, int(30000 / H / B ** 0.7))
    added = np.ceil(rng.random(B) ** 3 * most).astype(int)
    added[rng.random(B) < 0.15] = 0
    past = (rng.random(B) ** 3 * rng.choice([0, 50, 1000, 4000 if B < 50 else 300])).astype(int)
    past[rng.random(B) < 0.1] *= -1
    causal = rng.random() < 0.8
    return H, added, np.maximum(added + past, 0), bool(causal)


@pytest.mark.parametrize("seed", range(60))
def test_drawn(gkr, seed):
    H, added, keys, causal = drawn(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, N = int(added.sum()), int(keys.sum())
    q = (2 * torch.randn(T + 3, H, 512, generator=g, device=DEV)).to(torch.bfloat16)
    kv = torch.randn(N + 1, 512, generator=g, device=DEV).to(torch.bfloat16)
    kv[N] = float("nan")
    starts, kv_starts = np.concatenate([[0], added.cumsum()]), np.concatenate([[0], keys.cumsum()])
    i32 = lambda x: torch.from_numpy(x.astype(np.int32)).to(DEV)  # noqa: E731
    sm = 512 ** -0.5
    out, lse = torch.full_like(q, 7.0), torch.full((T + 3, H), 7.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    gkr.prompt_attention(q, kv, i32(starts), sm, i32(kv_starts), causal, out=out, lse=lse, err_flag=err)
    assert int(err.item()) == 0
    assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()
    for b in range(len(added)):
        n, m = int(added[b]), int(keys[b])
        if n == 0:
            continue
        k = kv[kv_starts[b]:kv_starts[b] + m].double()
        rows = torch.arange(n, device=DEV) if n * H * max(m, 1) < 4e7 else \
            torch.unique(torch.randint(0, n, (max(1, int(4e7 / H / m)),), generator=g, device=DEV))
        qq = q[starts[b] + rows].double()
        see = (m - n + 1 + rows if causal else torch.full_like(rows, m)).clamp(0, m)
        s = sm * torch.einsum("nhd,md->nhm", qq, k)
        seen = torch.arange(m, device=DEV) < see[:, None]
        s = torch.where(seen[:, None, :], s, -torch.inf)
        l = torch.logsumexp(s, 2) if m else torch.full(s.shape[:2], -torch.inf, dtype=torch.float64, device=DEV)
        p = torch.exp(s - torch.where(torch.isinf(l), 0.0, l)[..., None])
        spread = sm * torch.einsum("nhd,md->nhm", qq.abs(), k.abs()).where(seen[:, None, :], torch.zeros_like(s))
        r = {"out": p @ k, "lse": l, "mass": p @ k.abs(), "spread": spread.amax(2) if m else l.abs() * 0}
        r = {name: x.cpu().numpy() for name, x in r.items()}
        t_out, t_lse = plain.tolerances({**r, "spread": np.nan_to_num(r["spread"])}, max(m, 1))
        got, got_l = out[starts[b] + rows].double().cpu().numpy(), lse[starts[b] + rows].double().cpu().numpy()
        some = np.isfinite(r["lse"])
        assert np.array_equal(np.isneginf(got_l), ~some), (b, n, m)
        assert (got[~some] == 0).all()
        assert (np.abs(got_l[some] - r["lse"][some]) <= t_lse[some]).all(), (b, n, m)
        assert (np.abs(got - r["out"]) <= t_out).all(), (b, n, m)
