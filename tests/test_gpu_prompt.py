"""GPU tests of prompt_attention against the plain 64-bit form, within tolerances derived in
plain_paged."""
import numpy as np
import pytest
import torch

import plain_paged as plain
from plain_mxfp4 import bf16, bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


class Case:
    """Requests of `added` queries over past + added rows."""

    def __init__(self, added, past=0, H=2, seed=0, causal=True, qscale=2.0, sm_scale=512 ** -0.5, spread=1.0,
                 behind=0, kv_pad=0, rows_behind=0):
        rng = np.random.default_rng(seed)
        self.added = np.asarray(added)
        keys = np.maximum(self.added + np.asarray(past), 0)
        self.starts = np.concatenate([[0], np.cumsum(self.added)])
        self.kv_starts = np.concatenate([[0], np.cumsum(keys)])
        self.T, self.N = int(self.starts[-1]) + behind, int(self.kv_starts[-1]) + rows_behind
        self.causal, self.sm, self.H = causal, sm_scale, H
        self.qbits = bf16_bits(qscale * rng.standard_normal((self.T, H, 512)))
        self.kbits = bf16_bits(rng.standard_normal((self.N, 512)) * np.exp(spread * rng.standard_normal(512) / 2))
        self.kv_pad = kv_pad
        self.upload()

    def upload(self):
        self.q = to_bf16(self.qbits)
        wide = torch.full((self.N, 512 + self.kv_pad), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :512] = to_bf16(self.kbits)
        self.kv = wide[:, :512]

    def args(self):
        i = lambda x: torch.from_numpy(x.astype(np.int32)).to(DEV)  # noqa: E731
        return self.q, self.kv, i(self.starts), self.sm, i(self.kv_starts), self.causal

    def run(self, gkr, **kw):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full_like(self.q, 7.0)
        lse = torch.full((self.T, self.H), 7.0, device=DEV)
        gkr.prompt_attention(*self.args(), out=out, lse=lse, err_flag=err, **kw)
        torch.cuda.synchronize()
        return out, lse, int(err.item())

    def want(self):
        return plain.prompt(bf16(self.qbits).astype(np.float64), bf16(self.kbits).astype(np.float64), self.starts,
                            self.kv_starts, self.sm, self.causal)

    def check(self, gkr, **kw):
        out, lse, err = self.run(gkr, **kw)
        r = self.want()
        got, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        n = int(self.starts[-1])
        assert (got[n:] == 7.0).all() and (l[n:] == 7.0).all()
        got, l, r = got[:n], l[:n], {k: v[:n] for k, v in r.items()}
        t_out, t_lse = plain.tolerances(r, max(1, int(np.diff(self.kv_starts).max())))
        some = np.isfinite(r["lse"])
        assert np.array_equal(np.isneginf(l), ~some)
        off = np.abs(l[some] - r["lse"][some])
        assert (off <= t_lse[some]).all(), off.max()
        worst = np.abs(got - r["out"]) - t_out
        assert (worst <= 0).all(), f"out: {np.unravel_index(worst.argmax(), worst.shape)} {worst.max()}"
        assert (got[~some] == 0).all()
        assert err == 0
        return out, lse


@pytest.mark.parametrize("added,past,H", [
    ([1], 0, 1), ([1], 0, 128), ([1], 700, 128), ([1], 5000, 3), ([64], 0, 2), ([65], 0, 2), ([128], 0, 1),
    ([129], 0, 1), ([300], 0, 5), ([200], 0, 16), ([37], 91, 128), ([5], 1023, 64), ([3], 127, 130),
    ([2], 3, 300), ([1000], 0, 1), ([257], 500, 7), ([1] * 20, list(range(0, 4000, 200)), 16),
    ([0, 5, 0, 1, 130, 0, 63, 0], 0, 4), ([33, 1, 0, 200], [0, 300, 50, 129], 16), ([1] * 300, 40, 2)])
def test_sizes(gkr, added, past, H):
    Case(added, past, H, seed=sum(added) + H, behind=3, rows_behind=2).check(gkr)


@pytest.mark.parametrize("added,past,H", [([150, 20, 1], [0, 130, 260], 3), ([40, 9], [0, 300], 32)])
@pytest.mark.parametrize("kw", [
    dict(causal=False), dict(kv_pad=8), dict(kv_pad=512), dict(sm_scale=-0.03), dict(sm_scale=0.0),
    dict(qscale=16.0), dict(qscale=0.0), dict(spread=4.0, qscale=0.5), dict(qscale=1e-30, sm_scale=1.0)])
def test_kinds(gkr, added, past, H, kw):
    Case(added, past, H, seed=4, **kw).check(gkr)


@pytest.mark.parametrize("H", [1, 16, 128])
def test_more_queries_than_rows(gkr, H):
    """The first queries of such a request see no row; a request without rows; one without queries."""
    Case([10, 150, 7, 0, 3], [-4, -130, -7, 20, 0], H, seed=5).check(gkr)
    Case([10, 150, 7, 0], [-10, -150, -7, 0], H, seed=5).check(gkr)


@pytest.mark.parametrize("rising", [True, False])
def test_maximum_moves(gkr, rising):
    """Logits that climb (fall) by far along the rows, so that the running maximum is replaced again and
    again (only once)."""
    c = Case([3, 70], [900, 500], 20, seed=6, qscale=1.0, sm_scale=1.0)
    k = bf16(c.kbits).astype(np.float64)
    for b in range(2):
        a, z = c.kv_starts[b], c.kv_starts[b + 1]
        order = np.argsort(k[a:z] @ bf16(c.qbits)[c.starts[b + 1] - 1, 0].astype(np.float64), kind="stable")
        c.kbits[a:z] = c.kbits[a:z][order if rising else order[::-1]]
    c.upload()
    c.check(gkr)


@pytest.mark.parametrize("H", [1, 16, 128])
@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80])
def test_what_is_not_seen_does_not_count(gkr, H, value):
    """NaN and infinities in later rows, in the rows of other requests and behind the last; those in a
    query stay with it."""
    c = Case([100, 60, 1], [0, 70, 200], H, seed=7, rows_behind=130, behind=2)
    want_out, want_lse, _ = c.run(gkr)
    poisoned = [(0, 50), (0, 99), (1, 60)]                  # request, its row (that its query sees)
    for b, row in poisoned:
        c.kbits[c.kv_starts[b] + row, [3, 300, 511]] = value
    c.kbits[c.kv_starts[-1]:] = value
    c.qbits[20, 0] = 0x7FC0
    c.upload()
    out, lse, err = c.run(gkr)
    assert err == 0
    hit = np.zeros((c.T, H), bool)
    for b, row in poisoned:
        for i in range(c.added[b]):
            if row <= (np.diff(c.kv_starts)[b] - c.added[b]) + i:
                hit[c.starts[b] + i] = True
    hit[20, 0] = True
    hit = torch.from_numpy(hit).to(DEV)
    assert torch.equal(out[~hit], want_out[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    # a logit of -inf (three products of one sign) may take its row out of the sum; anything else shows
    if value != 0x7FC0:
        q = c.q[..., [3, 300, 511]].float() * (1.0 if value == 0x7F80 else -1.0)
        hit &= ~(q < 0).all(2)
    assert torch.isnan(lse[20, 0]) and torch.isnan(lse[hit]).all() and torch.isnan(out[hit].float()).all()


def test_starts_out_of_range(gkr):
    c = Case([20, 30], 0, 4, seed=8, behind=5, rows_behind=5)
    for starts, kv_starts in [([-3, 20, 99], [0, 20, 50]), ([0, 20, 50], [0, 2 ** 31 - 1, -7]),
                              ([20, 0, 10], [0, 10, 20]), ([2 ** 31 - 1] * 3, [-2 ** 31] * 3)]:
        d = c
        d.starts, d.kv_starts = np.array(starts), np.array(kv_starts)
        _, _, err = d.run(gkr)
        assert err == gkr.ERR_INDEX
    c = Case([20, 30], 0, 4, seed=8)
    c.check(gkr)


def test_starts_that_skip(gkr):
    """The first request begins behind some queries and rows: those are left alone."""
    c = Case([20, 30], [5, 9], 3, seed=9)
    c.starts, c.kv_starts = np.array([12, 50]), np.array([30, 64])
    out, lse, err = c.run(gkr)
    assert err == 0 and (out[:12] == 7.0).all() and (lse[:12] == 7.0).all()
    r = c.want()
    t_out, t_lse = plain.tolerances({k: v[12:] for k, v in r.items()}, 64)
    some = np.isfinite(r["lse"][12:])
    assert (np.abs(lse.cpu().numpy()[12:][some] - r["lse"][12:][some]) <= t_lse[some]).all()
    assert (np.abs(out.float().cpu().numpy()[12:] - r["out"][12:]) <= t_out).all()


def test_nothing(gkr):
    c = Case([4], 0, 2)
    e = gkr.prompt_attention(c.q[:0], c.kv, torch.zeros(1, dtype=torch.int32, device=DEV), 1.0)
    assert e[0].shape == (0, 2, 512) and e[1].shape == (0, 2)
    out, lse = torch.full_like(c.q, 7.0), torch.full((4, 2), 7.0, device=DEV)
    gkr.prompt_attention(c.q, c.kv, torch.zeros(1, dtype=torch.int32, device=DEV), 1.0, out=out, lse=lse)
    assert (out == 7.0).all() and (lse == 7.0).all()
    one = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    gkr.prompt_attention(c.q, c.kv[:0], one, 1.0, kv_starts=none, out=out, lse=lse)       # no rows at all
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_same_bits_on_streams_and_in_graphs(gkr):
    c = Case([100, 1, 260], [50, 3000, 0], 24, seed=10)
    want = c.check(gkr)
    for _ in range(3):
        again = gkr.prompt_attention(*c.args())
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = gkr.prompt_attention(*c.args())
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    size = gkr.prompt_attention_workspace(c.H, c.T)
    ws = [torch.zeros(max(size, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
    args = c.args()
    outs = [(torch.zeros_like(want[0]), torch.zeros_like(want[1])) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, w, (o, l) in zip(graphs, ws, outs):
        with torch.cuda.graph(g):
            gkr.prompt_attention(*args, out=o, lse=l, workspace=w)
    for _ in range(3):
        with torch.cuda.stream(s):                           # both at the same time
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for o, l in outs:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])
            o.zero_()
        torch.cuda.synchronize()
    with gkr.launch_policy(pdl=False):
        b = gkr.prompt_attention(*c.args())
    assert torch.equal(b[0], want[0])


def test_workspace_too_small(gkr):
    c = Case([100], 0, 24, seed=10)
    need = gkr.prompt_attention_workspace(c.H, c.T)
    if need:
        with pytest.raises(ValueError):
            gkr.prompt_attention(*c.args(), workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("added,past,H", [([2000, 700], [0, 3000], 16), ([1] * 8, 9000, 128), ([4000], 0, 8)])
def test_larger(gkr, added, past, H):
    """Against the plain form on the GPU, a sample of the queries."""
    c = Case(added, past, H, seed=11)
    out, lse, err = c.run(gkr)
    assert err == 0
    k = c.kv.double()
    rng = np.random.default_rng(1)
    for b in range(len(added)):
        n, m = int(c.added[b]), int(np.diff(c.kv_starts)[b])
        for i in sorted(set([0, n - 1, *rng.integers(0, n, 12).tolist()])):
            t = int(c.starts[b]) + i
            kk = k[int(c.kv_starts[b]):int(c.kv_starts[b]) + m - n + i + 1]
            s = c.sm * (c.q[t].double() @ kk.T)
            l = torch.logsumexp(s, 1)
            p = torch.exp(s - l[:, None])
            r = {"out": (p @ kk).cpu().numpy()[None], "lse": l.cpu().numpy()[None],
                 "mass": (p @ kk.abs()).cpu().numpy()[None],
                 "spread": (c.sm * (c.q[t].double().abs() @ kk.abs().T)).amax(1).cpu().numpy()[None]}
            t_out, t_lse = plain.tolerances(r, len(kk))
            assert (np.abs(out[t].float().cpu().numpy() - r["out"][0]) <= t_out[0]).all(), (b, i)
            assert (np.abs(lse[t].cpu().numpy() - r["lse"][0]) <= t_lse[0]).all(), (b, i)
