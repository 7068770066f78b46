"""Calls captured into a graph and replayed with other lengths, lists and pages than they were captured with: what
a replay does is found on the device, and the same bits come out as from a call outside the graph."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = 512 ** -0.5


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)


def capture(f):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


# of one long request, many short ones, empty ones, more queries than rows: whole tiles, even cuts, no rows
@pytest.mark.parametrize("H", [1, 16, 128])
@pytest.mark.parametrize("B", [4, 40, 90])
def test_prompt_with_other_lengths(gkr, B, H):
    rng = np.random.default_rng(B + H)
    T, N = 400, 6000
    q, kv = randn(T, H, 512, seed=1, scale=2.0), randn(N, 512, seed=2)
    starts, kv_starts = i32(np.zeros(B + 1)), i32(np.zeros(B + 1))
    g, (out, lse) = capture(lambda: gkr.prompt_attention(q, kv, starts, SM, kv_starts=kv_starts))
    for kind in range(5):
        one = np.sort(rng.integers(0, T + 1, B - 1))
        two = np.sort(rng.integers(0, N + 1, B - 1))
        if kind == 1:
            one[:], two[:] = T - 1, N // 2            # nearly everything is the first request's
        if kind == 2:
            one, two = np.linspace(0, T, B + 1)[1:-1].astype(int), np.linspace(0, N, B + 1)[1:-1].astype(int)
        if kind == 3:
            two[:] = N                                # the others have no rows
        starts.copy_(i32([0, *one, T]))
        kv_starts.copy_(i32([0, *two, N]))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        want, want_lse = gkr.prompt_attention(q, kv, starts, SM, kv_starts=kv_starts)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), kind
        assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("Q,H,L,K", [(4, 16, 900, 60), (100, 16, 2000, 90), (260, 5, 700, 0)])
def test_prefix_with_other_lists(gkr, Q, H, L, K):
    cache = gkr.alloc_cache(50, 64, 272, DEV, fill=0)
    csc = torch.cat([torch.ones(8, 32), torch.zeros(8, 32)], 1).to(DEV)
    gkr.kv_insert(randn(3200, 512, seed=3), cache, torch.arange(3200, device=DEV), torch.zeros(3200, dtype=torch.int64, device=DEV),
                  csc, 64)
    q = randn(Q, H, 512, seed=4, scale=2.0)
    prefix, own = i32(np.zeros(L)), i32(np.zeros((Q, K)))
    g, (out, lse) = capture(lambda: gkr.prefix_attention(q, cache, prefix, own, SM))
    rng = np.random.default_rng(5)
    for holes in (0.0, 0.5, 1.0):
        prefix.copy_(i32(np.where(rng.random(L) < holes, -1, rng.integers(0, 3200, L))))
        own.copy_(i32(np.where(rng.random((Q, K)) < holes, -1, rng.integers(0, 3200, (Q, K)))))
        g.replay()
        want, want_lse = gkr.prefix_attention(q, cache, prefix, own, SM)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), holes
        if holes == 1.0:
            assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("batch,heads,prefix", [(3, 16, 256), (70, 16, 2048)])
def test_steps_of_a_batch(gkr, batch, heads, prefix):
    """A decode step as one graph (pages, insert, lists, attention, the lengths and the free list moved on),
    replayed over page borders, against the same steps without a graph."""
    bs, steps, first = 64, 70, 60
    csc = torch.cat([torch.ones(4096, 32), torch.zeros(4096, 32)], 1).to(DEV)
    shared, own = prefix // bs, -(-(first + steps) // bs)
    pages = shared + batch * own

    def state():
        s = {"cache": gkr.alloc_cache(pages, bs, 272, DEV, fill=0)}
        table = np.full((batch, shared + own), -1)
        table[:, :shared] = np.arange(shared)
        table[:, shared] = shared + np.arange(batch)
        s["table"], s["lengths"] = i32(table), i32(np.full(batch, prefix + first))
        s["free"] = i32(shared + batch + np.arange(pages - shared - batch))
        s["one"], s["first"] = i32(np.ones(batch)), i32(np.full(batch, prefix))
        s["kv"], s["q"] = randn(batch, 512, seed=6), randn(batch, heads, 512, seed=7, scale=2.0)
        n = shared * bs
        gkr.kv_insert(randn(n, 512, seed=8), s["cache"], torch.arange(n, device=DEV), torch.arange(n, device=DEV), csc, bs)
        s["prefix"] = i32(np.arange(n))
        return s

    def step(s):
        slots, pos, _, taken = gkr.kv_allocate(s["lengths"], s["one"], s["table"], s["free"], bs, batch)
        gkr.kv_insert(s["kv"], s["cache"], slots, pos, csc, bs)
        at = torch.arange(len(s["free"]), device=DEV)
        s["free"].copy_(s["free"][(at + taken) % len(s["free"])])
        s["lengths"] += 1
        lists = gkr.kv_slots(s["table"], s["lengths"], bs, own * bs, first=s["first"])
        return gkr.prefix_attention(s["q"], s["cache"], s["prefix"], lists, SM)

    plain, graphed = state(), state()
    start = {n: t.clone() for n, t in graphed.items() if n in ("table", "lengths", "free")}
    g, (out, lse) = capture(lambda: step(graphed))
    for n, t in start.items():                        # the captured call ran once before
        graphed[n].copy_(t)
    for i in range(steps):
        for s in (plain, graphed):
            s["kv"].copy_(randn(batch, 512, seed=100 + i))
            s["q"].copy_(randn(batch, heads, 512, seed=200 + i, scale=2.0))
        g.replay()
        want, want_lse = step(plain)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), i
        assert torch.equal(graphed["table"], plain["table"]) and torch.equal(graphed["lengths"], plain["lengths"])
    used = plain["table"][:, shared:]
    used = used[used >= 0]
    assert len(used) == batch * own and len(used.unique()) == len(used) and torch.isfinite(lse).all()
