"""GPU tests of prefix_attention where the prefix is read once for all queries: gathered to bf16 rows,
attended to by tiles of all queries' heads, joined with the queries' own lists.  A rule on sizes chooses between
that and each query's list with the prefix in front of it; every case here has to be on this side of it,
which the workspace shows: the other form takes what sparse_attention takes for the longer lists."""
import numpy as np
import pytest
import torch

import plain_mxfp4
import plain_paged as plain
from test_gpu_prefix import DEV, Case

pytestmark = pytest.mark.gpu


def shared(gkr, Q, H, L, K):
    return gkr.prefix_attention_workspace(H, Q, L, K) != gkr.sparse_attention_workspace(H, Q, L + K)


def make(gkr, Q, H, L, K, **kw):
    assert shared(gkr, Q, H, L, K)
    return Case(gkr, Q, H, L, K, **kw)


# one record, ends of tiles and chunks, no own lists, whole and cut own lists, one and many heads
@pytest.mark.parametrize("Q,H,L,K", [
    (1400, 1, 1, 64), (1000, 1, 65, 0), (1300, 2, 127, 65), (1300, 3, 129, 1), (260, 16, 700, 70),
    (100, 5, 2000, 90), (100, 1, 2000, 0), (64, 16, 4095, 100), (300, 33, 500, 0), (100, 127, 4097, 65),
    (400, 128, 1000, 130), (100, 16, 2000, 1000)])
def test_sizes(gkr, Q, H, L, K):
    make(gkr, Q, H, L, K, seed=Q + H + L + K, index_pad=3).check(gkr)


@pytest.mark.parametrize("Q,H,L,K", [(100, 5, 2000, 40), (260, 16, 700, 70), (100, 3, 2000, 0)])
@pytest.mark.parametrize("kw", [
    dict(holes=0.0), dict(holes=0.97), dict(bs=96, pad=512), dict(bs=32, pad=1536), dict(sm_scale=-0.03),
    dict(sm_scale=0.0), dict(qscale=16.0), dict(qscale=0.0), dict(spread=4.0, qscale=0.5)])
def test_kinds(gkr, Q, H, L, K, kw):
    make(gkr, Q, H, L, K, seed=3, **kw).check(gkr)


@pytest.mark.parametrize("Q,H,L,K", [(100, 4, 2000, 60), (260, 16, 700, 64)])
def test_empty_parts(gkr, Q, H, L, K):
    make(gkr, Q, H, L, K, seed=4, empty=(0, 2, Q - 1)).check(gkr)
    make(gkr, Q, H, L, K, seed=4, empty=range(Q)).check(gkr)      # no query has records of its own
    c = make(gkr, Q, H, L, K, seed=4, empty=(0, Q - 1))
    c.prefix[:] = -1                                              # a prefix of no entry
    c.upload(gkr)
    out, lse = c.check(gkr)
    for i in (0, Q - 1):
        assert (out[i] == 0).all() and torch.isneginf(lse[i]).all()
    c.idx[:] = -1                                                 # nothing at all
    c.upload(gkr)
    out, lse = c.check(gkr)
    assert (out == 0).all() and torch.isneginf(lse).all()
    c = make(gkr, 1000, 2, 130, 0, seed=4, holes=1.0)             # and no lists
    out, lse = c.check(gkr)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("only", ["first", "last"])
def test_prefix_of_one_entry(gkr, only):
    """All entries but one are holes, whole chunks of them."""
    c = make(gkr, 100, 4, 2000, 40, seed=12, empty=range(0, 100, 2))
    c.prefix[:] = -1
    c.prefix[0 if only == "first" else 1999] = 77
    c.upload(gkr)
    c.check(gkr)


@pytest.mark.parametrize("Q,H,L,K", [(100, 5, 2000, 50), (260, 16, 700, 50)])
def test_bad_indices(gkr, Q, H, L, K):
    c = make(gkr, Q, H, L, K, seed=5)
    c.prefix[[3, 200, L - 1]] = -2, c.slots, 2 ** 31 - 1
    c.upload(gkr)
    c.check(gkr)
    c.prefix[[3, 200, L - 1]] = -1
    c.idx[0, 3], c.idx[1, 49] = -2, c.slots
    c.upload(gkr)
    c.check(gkr)


@pytest.mark.parametrize("Q,H,L,K", [(100, 5, 2000, 50), (260, 16, 700, 50)])
def test_nan_record(gkr, Q, H, L, K):
    """A NaN scale reaches whoever lists the record and no one else."""
    c = make(gkr, Q, H, L, K, seed=6)
    c.prefix[c.prefix == 5] = 6
    c.idx[c.idx == 5] = 6
    c.idx[1, 7] = 5
    _, o = plain_mxfp4.offsets(5, c.bs, c.ps)
    c.host[o] = 255                                               # dims 0..31 of slot 5
    c.upload(gkr)
    out, lse = gkr.prefix_attention(*c.args)
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1].float()).all()
    rest = [i for i in range(Q) if i != 1]
    assert torch.isfinite(lse[rest]).all() and torch.isfinite(out[rest].float()).all()
    c.prefix[250] = 5
    c.upload(gkr)
    out, lse = gkr.prefix_attention(*c.args)
    assert torch.isnan(lse).all() and torch.isnan(out.float()).all()


@pytest.mark.parametrize("Q,H,L,K", [(64, 16, 4000, 100), (100, 40, 2000, 300), (260, 7, 700, 0)])
def test_equals_the_lists_written_out(gkr, Q, H, L, K):
    """The same as sparse_attention over each query's prefix and own list, within both tolerances."""
    c = make(gkr, Q, H, L, K, seed=7, pages=400)
    out, lse = c.check(gkr)
    whole = torch.cat([c.args[2].expand(Q, L), c.args[3]], 1).contiguous()
    o2, l2 = gkr.sparse_attention(c.q, c.cache, whole, c.sm)
    t_out, t_lse = plain.tolerances(c.want(), L + K)
    assert (np.abs((out.float() - o2.float()).cpu().numpy()) <= 2 * t_out).all()
    assert (np.abs((lse - l2).cpu().numpy()) <= 2 * t_lse).all()


@pytest.mark.parametrize("Q,H,L,K", [(100, 40, 2000, 300), (64, 16, 4000, 100), (100, 3, 2000, 0)])
def test_same_bits_on_streams_and_in_graphs(gkr, Q, H, L, K):
    c = make(gkr, Q, H, L, K, seed=8)
    want = c.check(gkr)
    for _ in range(3):
        again = gkr.prefix_attention(*c.args)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = gkr.prefix_attention(*c.args)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    size = gkr.prefix_attention_workspace(H, Q, L, K)
    ws = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]   # NaN, if it is read
    outs = [(torch.zeros_like(want[0]), torch.zeros_like(want[1])) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, w, (o, l) in zip(graphs, ws, outs):
        with torch.cuda.graph(g):
            gkr.prefix_attention(*c.args, out=o, lse=l, workspace=w)
    for _ in range(3):
        with torch.cuda.stream(s):                                # both at the same time
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for o, l in outs:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])
            o.zero_()
        torch.cuda.synchronize()
    with gkr.launch_policy(pdl=False):
        b = gkr.prefix_attention(*c.args)
    assert torch.equal(b[0], want[0]) and torch.equal(b[1], want[1])
    with pytest.raises(ValueError):
        gkr.prefix_attention(*c.args, workspace=ws[0][:size - 1])
