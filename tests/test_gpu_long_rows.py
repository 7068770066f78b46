"""prompt_attention and prefix_attention over so many rows that a pair of SMs takes its share of a tile in runs, each
with an accumulator of its own (the tensor cores' sums are cut off and not rounded: in one sum, a million rows came
out 0.4 % too small): results, sums far apart, waits that run out, and no wait that is as long as a tile."""
import importlib
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import plain_paged as plain
from test_gpu_attention_timeout import library
from test_gpu_prompt_timeout import ALL_RUN_OUT, check

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = 512 ** -0.5
RUN = 131072                # rows of a run


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)


# whole tiles and cut ones, shares that begin a tile, end one, or lie within; fewer than 128 rows of q
@pytest.mark.parametrize("T,H,rows", [(80, 128, 1000000), (100, 128, 500000), (30, 128, 1500000), (77, 127, 1000000),
                                      (1, 5, 14000000), (600, 16, 263000)])
def test_sums_do_not_shrink(gkr, T, H, rows):
    """Positive values, each row as often as any other: the mean of the results' relative errors has no other reason
    than sums that are cut off.  One cut of the last bit (2^-23) for each 16 rows of a run, and another for its
    first ones; the roundings of probabilities and results (2^-8 at most, either way) leave less than 2^-12 of T H
    512 results' mean."""
    base = (randn(1000, 512, seed=1).float().abs() + 0.5).to(torch.bfloat16)
    q = randn(T, H, 512, seed=2, scale=0.1)
    k = base.double()
    s = SM * torch.einsum("nhd,md->nhm", q.double(), k)
    lse = torch.logsumexp(s, 2)
    want = torch.softmax(s, 2) @ k
    kv = base.repeat(rows // 1000, 1)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, l = gkr.prompt_attention(q, kv, i32(0, T), SM, kv_starts=i32(0, rows), causal=False, err_flag=err)
    assert int(err.item()) == 0
    off = (out.double() - want) / want
    assert abs(off.mean().item()) <= (RUN / 16 + 16) * 2.0 ** -23 + 2.0 ** -12
    # each result: that and the roundings; logits below 4 in magnitude, see plain_paged
    assert off.abs().max().item() <= (RUN / 16 + 16) * 2.0 ** -23 + 2 * 2.0 ** -8 + 2.0 ** -10
    assert (l.double() - lse - np.log(rows / 1000)).abs().max().item() <= (RUN / 128 + 200) * 2.0 ** -24 + 2.0 ** -10


def sampled(gkr, out, lse, q, k, see):
    """Query i of q over the first see[i] rows of k (double), within the tolerances of a run."""
    for i, m in enumerate(see):
        s = SM * (q[i].double() @ k[:m].T)
        l = torch.logsumexp(s, 1)
        p = torch.exp(s - l[:, None])
        r = {"out": p @ k[:m], "lse": l, "mass": p @ k[:m].abs(), "spread": (SM * (q[i].double().abs() @ k[:m].abs().T)).amax(1)}
        r = {name: x.cpu().numpy()[None] for name, x in r.items()}
        t_out, t_lse = plain.tolerances(r, min(m, RUN))
        assert (np.abs(out[i].double().cpu().numpy() - r["out"][0]) <= t_out[0]).all(), i
        assert (np.abs(lse[i].double().cpu().numpy() - r["lse"][0]) <= t_lse[0]).all(), i


def test_causal_requests(gkr):
    """Long and short requests in one call; what a query does not see ends within a run."""
    added, keys = [90, 1, 300, 0, 40], [400000, 270001, 300, 5, 131073]
    H = 32
    q, kv = randn(sum(added), H, 512, seed=3, scale=2.0), randn(sum(keys) + 1, 512, seed=4)
    kv[-1] = float("nan")
    starts, kv_starts = np.concatenate([[0], np.cumsum(added)]), np.concatenate([[0], np.cumsum(keys)])
    out, lse = gkr.prompt_attention(q, kv, i32(*starts.tolist()), SM, kv_starts=i32(*kv_starts.tolist()))
    for b, (n, m) in enumerate(zip(added, keys)):
        if n == 0:
            continue
        some = sorted({0, n // 2, n - 1})
        at = [int(starts[b]) + i for i in some]
        sampled(gkr, out[at], lse[at], q[at], kv[int(kv_starts[b]):int(kv_starts[b + 1])].double(), [m - n + 1 + i for i in some])


@pytest.mark.parametrize("K", [0, 70])
def test_prefix(gkr, K):
    """A long prefix with holes, whole runs of them, alone and with own lists."""
    L, Q, H, slots = 420000, 90, 32, 6400
    cache = gkr.alloc_cache(100, 64, 272, DEV, fill=0)
    csc = torch.cat([torch.ones(8, 32), torch.zeros(8, 32)], 1).to(DEV)
    at = torch.arange(slots, device=DEV)
    gkr.kv_insert(randn(slots, 512, seed=5), cache, at, torch.zeros_like(at), csc, 64)
    rows = gkr.kv_gather(cache, at.int(), torch.empty(slots, 512, dtype=torch.bfloat16, device=DEV)).double()
    g = torch.Generator(device=DEV).manual_seed(6)
    prefix = torch.randint(-300, slots, (L,), generator=g, device=DEV).clamp(min=-1).int()
    prefix[130000:270000] = -1
    own = torch.randint(-300, slots, (Q, K), generator=g, device=DEV).clamp(min=-1).int()
    q = randn(Q, H, 512, seed=7, scale=2.0)
    assert gkr.prefix_attention_workspace(H, Q, L, K) != gkr.sparse_attention_workspace(H, Q, L + K)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = gkr.prefix_attention(q, cache, prefix, own, SM, err_flag=err)
    assert int(err.item()) == 0
    shared = rows[prefix[prefix >= 0].long()]
    for i in (0, 41, Q - 1):
        k = torch.cat([shared, rows[own[i][own[i] >= 0].long()]])
        sampled(gkr, out[i:i + 1], lse[i:i + 1], q[i:i + 1], k, [len(k)])


@pytest.mark.parametrize("T,H", [(80, 128), (30, 128)])
def test_maxima_far_apart_over_runs(gkr, T, H):
    """A first run whose weight is 2^-104, and shows where the last rows have no values; and the other way round."""
    rows = 300000
    q = torch.zeros(T, H, 512, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    kv = torch.zeros(rows, 512, dtype=torch.bfloat16, device=DEV)
    kv[:, 0], kv[:, 1:] = -84.0, 1.5
    top = torch.arange(rows - 64, rows, device=DEV)
    for order in (0, 1):
        kv[top] = 0.0
        out, lse = gkr.prompt_attention(q, kv, i32(0, T), 1.0, kv_starts=i32(0, rows), causal=False)
        total = 64 + (rows - 64) * np.exp(-84.0)
        value = 1.5 * (rows - 64) * np.exp(-84.0) / total
        # a logit of 84: 2^-13 of it and the roundings in the exponent; sums cut off; bf16 twice
        d = np.expm1(2.0 ** -12 * 84) + 2 * RUN / 16 * 2.0 ** -23 + 2.0 ** -7
        assert ((out[..., 1:].double() - value).abs() <= d * value).all()
        assert (lse.double() - np.log(total)).abs().max() <= 2.0 ** -10
        kv[top, 0], kv[top, 1:] = -84.0, 1.5
        top = torch.arange(64, device=DEV)


STEADY = 5000000            # clocks: twice what a run takes, a fraction of a tile
LIMITS = [ALL_RUN_OUT, 10000, 1000000]


@pytest.fixture(scope="module")
def libraries(gkr, tmp_path_factory):
    """{limit: library}: waits of that many clocks at most."""
    b = importlib.import_module("gather_kv_rope_gb300.build")
    tmp = tmp_path_factory.mktemp("short_waits")

    def run(*args):
        subprocess.run([b.nvcc(), *b.ARCH, *map(str, args)], check=True, capture_output=True)

    def compile_one(job):
        src, limit = job
        obj = tmp / f"{src.stem}{limit}.o"
        run(*b.NVCC_FLAGS, *([] if limit is None else [f"-DGKR_WAIT_CLOCKS={limit}"]), "-c", src, "-o", obj)
        return obj

    limits = (STEADY, *LIMITS)
    jobs = [(s, x) for s in b.sources() for x in (limits if s.stem == "prompt" else (None,))]
    with ThreadPoolExecutor(8) as ex:
        objs = dict(zip(jobs, ex.map(compile_one, jobs)))
    out = {x: tmp / f"libgkr{x}.so" for x in limits}
    for x in limits:
        run("-shared", "-cudart", "static", "-o", out[x], *(o for (_, y), o in objs.items() if y in (None, x)))
    return out


@pytest.mark.parametrize("T", [30, 80])
def test_no_wait_takes_as_long_as_a_tile(gkr, libraries, T):
    """The kernels with waits of 5 million clocks; a tile takes 30 million and more."""
    rows = 2000000
    q, kv = randn(T, 128, 512, seed=8, scale=2.0), randn(1000, 512, seed=9).repeat(rows // 1000, 1)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call():
        return gkr.prompt_attention(q, kv, i32(0, T), SM, kv_starts=i32(0, rows), causal=False, err_flag=err)

    want = call()
    with library(libraries[STEADY]):
        got = call()
        torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,H", [(80, 128), (30, 128), (100, 5)])
@pytest.mark.parametrize("limit", LIMITS)
def test_rows_are_right_or_not_written(gkr, libraries, T, H, limit):
    rows = 400000
    q, kv = randn(T, H, 512, seed=10, scale=2.0), randn(rows, 512, seed=11)
    ws = torch.zeros(gkr.prompt_attention_workspace(H, T), dtype=torch.uint8, device=DEV)
    other = q.flip(0).flip(1).neg()

    def call(out, lse, err):
        gkr.prompt_attention(q, kv, i32(0, T), SM, i32(0, rows), False, out=out, lse=lse, workspace=ws, err_flag=err)

    def spoil():
        gkr.prompt_attention(other, kv, i32(0, T), -SM, i32(0, rows), False, workspace=ws)

    check(gkr, libraries, limit, 2, call, spoil, (T, H))
