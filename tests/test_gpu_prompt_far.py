"""The paged batch's operators at their ends: many requests, rows past 4 GB, several host threads at once."""
import threading

import numpy as np
import pytest
import torch

import plain_paged as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = 512 ** -0.5


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)


def close(out, lse, q, k, see):
    r = plain.attend(q.double().cpu().numpy(), k.double().cpu().numpy(), see, SM)
    t_out, t_lse = plain.tolerances(r, len(k))
    assert (np.abs(out.float().cpu().numpy() - r["out"]) <= t_out).all()
    assert (np.abs(lse.cpu().numpy() - r["lse"]) <= t_lse).all()


@pytest.mark.parametrize("B,H", [(16384, 1), (16384, 3), (5000, 16)])
def test_many_requests(gkr, B, H):
    rng = np.random.default_rng(B)
    added = rng.integers(0, 3, B)
    keys = added + rng.integers(0, 40, B)
    starts, kv_starts = np.concatenate([[0], added.cumsum()]), np.concatenate([[0], keys.cumsum()])
    q, kv = randn(int(starts[-1]), H, 512, seed=1, scale=2.0), randn(int(kv_starts[-1]), 512, seed=2)
    out, lse = gkr.prompt_attention(q, kv, i32(starts), SM, i32(kv_starts))
    # all of them, padded: two queries, 42 rows
    at, kat = torch.arange(2, device=DEV), torch.arange(42, device=DEV)
    n, m = i32(added).long()[:, None], i32(keys).long()[:, None]
    qq = q[(i32(starts[:-1]).long()[:, None] + at).clamp(max=len(q) - 1)].double()
    kk = kv[(i32(kv_starts[:-1]).long()[:, None] + kat).clamp(max=len(kv) - 1)].double()
    s = SM * torch.einsum("bnhd,bmd->bnhm", qq, kk)
    see = kat < (m - n + at + 1)[..., None]
    s = s.masked_fill(~see[:, :, None], -torch.inf)
    live = at < n
    want_l = torch.logsumexp(s, 3)[live]
    p = torch.softmax(s, 3)
    want, mass = torch.einsum("bnhm,bmd->bnhd", p, kk)[live], torch.einsum("bnhm,bmd->bnhd", p, kk.abs())[live]
    spread = SM * torch.einsum("bnhd,bmd->bnhm", qq.abs(), kk.abs()).amax(3)[live]
    r = {"out": want, "lse": want_l, "mass": mass, "spread": spread}
    t_out, t_lse = plain.tolerances({k: v.cpu().numpy() for k, v in r.items()}, 42)
    assert (np.abs(out.float().cpu().numpy() - want.cpu().numpy()) <= t_out).all()
    assert (np.abs(lse.cpu().numpy() - want_l.cpu().numpy()) <= t_lse).all()


def test_rows_past_four_gigabytes(gkr):
    """Queries, rows and results that begin behind 2^32 bytes."""
    T, H, N, n, m = 34000, 128, (1 << 22) + 3000, 5, 700
    q = torch.empty(T, H, 512, dtype=torch.bfloat16, device=DEV)
    kv = torch.empty(N, 512, dtype=torch.bfloat16, device=DEV)
    q[T - n:], kv[N - m:] = randn(n, H, 512, seed=3, scale=2.0), randn(m, 512, seed=4)
    out, lse = torch.empty_like(q), torch.empty(T, H, device=DEV)
    out[:16], lse[:16] = 7.0, 7.0
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    gkr.prompt_attention(q, kv, i32([T - n, T]), SM, i32([N - m, N]), out=out, lse=lse, err_flag=err)
    assert int(err.item()) == 0 and (out[:16] == 7.0).all() and (lse[:16] == 7.0).all()
    close(out[T - n:], lse[T - n:], q[T - n:], kv[N - m:], m - n + 1 + np.arange(n))
    # rows far apart
    wide = torch.empty(700, 3 << 20, dtype=torch.bfloat16, device=DEV)[:, 512:1024]
    wide.copy_(kv[N - m:])
    out2, lse2 = gkr.prompt_attention(q[T - n:], wide, i32([0, n]), SM, i32([0, m]))
    assert torch.equal(out2, out[T - n:]) and torch.equal(lse2, lse[T - n:])


def test_long_prefix(gkr):
    """A prefix whose gathered rows pass 4 GB, every record listed many times: as the records once, with a
    logit of ln(times) more for each."""
    Q, H, L, S = 16, 16, (1 << 22) + 77, 64
    cache = gkr.alloc_cache(1, 64, gkr.MXFP4, DEV, fill=0)
    csc = torch.cat([torch.ones(64, 32), torch.zeros(64, 32)], 1).to(DEV)
    gkr.kv_insert(randn(S, 512, seed=5), cache, torch.arange(S, device=DEV), torch.arange(S, device=DEV), csc, 64)
    prefix = (torch.arange(L, device=DEV) % S).int()
    q, none = randn(Q, H, 512, seed=6, scale=2.0), torch.empty(Q, 0, dtype=torch.int32, device=DEV)
    out, lse = gkr.prefix_attention(q, cache, prefix, none, SM)
    k = gkr.kv_gather(cache, prefix[:S].contiguous(), torch.empty(S, 512, dtype=torch.bfloat16, device=DEV)).double()
    times = torch.full((S,), L // S, device=DEV, dtype=torch.float64)
    times[:L % S] += 1
    s = SM * torch.einsum("qhd,md->qhm", q.double(), k) + times.log()
    l, p = torch.logsumexp(s, 2), torch.softmax(s, 2)
    spread = SM * torch.einsum("qhd,md->qhm", q.double().abs(), k.abs()).amax(2)
    r = {"out": p @ k, "lse": l, "mass": p @ k.abs(), "spread": spread}
    t_out, t_lse = plain.tolerances({n: x.cpu().numpy() for n, x in r.items()}, L)
    assert (np.abs(out.float().cpu().numpy() - r["out"].cpu().numpy()) <= t_out).all()
    assert (np.abs(lse.cpu().numpy() - l.cpu().numpy()) <= t_lse).all()


def test_threads(gkr):
    """Four host threads, each with its own stream, inputs and launch options."""
    jobs = []
    for k in range(4):
        added, keys = [60 + 50 * k, 1, 7], [60 + 50 * k, 900, 300]
        q, kv = randn(sum(added), 8 << k, 512, seed=k, scale=2.0), randn(sum(keys), 512, seed=10 + k)
        args = q, kv, i32(np.concatenate([[0], np.cumsum(added)])), SM, i32(np.concatenate([[0], np.cumsum(keys)]))
        jobs.append((args, gkr.prompt_attention(*args)))
    lengths = i32([500, 3, 0, 77])
    table = torch.randperm(40, device=DEV).int().view(4, 10)
    want = gkr.kv_slots_packed(table, lengths, 64, 600)
    torch.cuda.synchronize()
    errors, barrier = [], threading.Barrier(len(jobs))

    def work(k):
        try:
            args, (o, l) = jobs[k]
            with torch.cuda.stream(torch.cuda.Stream()), gkr.launch_policy(pdl=bool(k % 2)):
                barrier.wait()
                for _ in range(20):
                    out, lse = gkr.prompt_attention(*args)
                    got = gkr.kv_slots_packed(table, lengths, 64, 600)
                    torch.cuda.current_stream().synchronize()
                    assert torch.equal(out, o) and torch.equal(lse, l)
                    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        except Exception as e:            # reported after the join
            errors.append((k, repr(e)))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not errors, errors
