"""GPU tests of prefix_attention against the plain 64-bit form, within tolerances derived in
plain_paged, and of a batch's way through the cache: allocate, insert, list, gather, attend."""
import numpy as np
import pytest
import torch

import plain_mxfp4
import plain_paged as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


class Case:
    def __init__(self, gkr, Q, H, L, K, bs=64, pages=40, pad=0, seed=0, holes=0.1, qscale=2.0, spread=1.0,
                 sm_scale=512 ** -0.5, empty=(), index_pad=0):
        rng = np.random.default_rng(seed)
        self.bs, self.ps, self.slots = bs, gkr.page_stride(272, bs) + pad, pages * bs
        self.host = rng.integers(0, 256, pages * self.ps, dtype=np.uint8)
        s = np.clip(127 + np.round(spread * rng.standard_normal((self.slots, 16)) - 1.5), 0, 254)
        at = np.array([plain_mxfp4.offsets(slot, bs, self.ps)[1] for slot in range(self.slots)])
        self.host[at[:, None] + np.arange(16)] = s
        self.prefix = rng.integers(0, self.slots, L).astype(np.int32)
        self.prefix[rng.random(L) < holes] = -1
        self.idx = rng.integers(0, self.slots, (Q, K)).astype(np.int32)
        self.idx[rng.random((Q, K)) < holes] = -1
        for i in empty:
            self.idx[i] = -1
        self.sm, self.index_pad = sm_scale, index_pad
        self.qbits = plain_mxfp4.bf16_bits(qscale * rng.standard_normal((Q, H, 512)))
        self.cache = gkr.alloc_cache(pages, bs, 272, DEV, page_stride_bytes=self.ps)
        self.upload(gkr)

    def upload(self, gkr):
        self.q = to_bf16(self.qbits)
        gkr.cache_bytes(self.cache).copy_(torch.from_numpy(self.host))
        Q, K = self.idx.shape
        wide = torch.full((Q, K + self.index_pad), 7, dtype=torch.int32, device=DEV)
        wide[:, :K] = torch.from_numpy(self.idx)
        self.args = self.q, self.cache, torch.from_numpy(self.prefix).to(DEV), wide[:, :K], self.sm

    def rows(self, idx):
        idx = idx[(idx >= 0) & (idx < self.slots)]
        return plain_mxfp4.decode(*plain_mxfp4.record_bytes(self.host, idx, self.bs, self.ps))

    def want(self):
        q = plain_mxfp4.bf16(self.qbits).astype(np.float64)
        shared = self.rows(self.prefix)
        parts = []
        for i in range(len(q)):
            k = np.concatenate([shared, self.rows(self.idx[i])])
            parts.append(plain.attend(q[i:i + 1], k, [len(k)], self.sm))
        return {n: np.concatenate([p[n] for p in parts]) for n in parts[0]}

    def check(self, gkr, **kw):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, lse = gkr.prefix_attention(*self.args, err_flag=err, **kw)
        torch.cuda.synchronize()
        r = self.want()
        t_out, t_lse = plain.tolerances(r, len(self.prefix) + self.idx.shape[1])
        got, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        some = np.isfinite(r["lse"])
        assert np.array_equal(np.isneginf(l), ~some)
        off = np.abs(l[some] - r["lse"][some])
        assert (off <= t_lse[some]).all(), off.max()
        worst = np.abs(got - r["out"]) - t_out
        assert (worst <= 0).all(), f"out: {np.unravel_index(worst.argmax(), worst.shape)} {worst.max()}"
        assert (got[~some] == 0).all()
        bad = any(((x < -1) | (x >= self.slots)).any() for x in (self.prefix, self.idx))
        assert int(err.item()) == (gkr.ERR_INDEX if bad else 0)
        return out, lse


@pytest.mark.parametrize("Q,H,L,K", [
    (1, 1, 1, 1), (1, 128, 1, 0), (1, 16, 0, 31), (2, 5, 33, 3), (3, 64, 64, 64), (2, 127, 129, 65),
    (1, 128, 128, 128), (5, 33, 257, 7), (40, 16, 700, 70), (130, 3, 200, 5), (9, 128, 300, 190),
    (1, 8, 3000, 100), (64, 2, 1000, 1), (4, 16, 4095, 100), (33, 48, 63, 0), (300, 1, 130, 20)])
def test_sizes(gkr, Q, H, L, K):
    Case(gkr, Q, H, L, K, seed=Q + H + L + K, index_pad=3).check(gkr)


@pytest.mark.parametrize("Q,H,L,K", [(3, 9, 200, 40), (20, 128, 300, 70)])
@pytest.mark.parametrize("kw", [
    dict(holes=0.0), dict(holes=0.97), dict(bs=96, pad=512), dict(bs=32, pad=1536), dict(sm_scale=-0.03),
    dict(sm_scale=0.0), dict(qscale=16.0), dict(qscale=0.0), dict(spread=4.0, qscale=0.5)])
def test_kinds(gkr, Q, H, L, K, kw):
    Case(gkr, Q, H, L, K, seed=3, **kw).check(gkr)


@pytest.mark.parametrize("Q,H", [(4, 4), (12, 128)])
def test_empty_parts(gkr, Q, H):
    Case(gkr, Q, H, 200, 60, seed=4, empty=(0, 2)).check(gkr)
    c = Case(gkr, Q, H, 200, 60, seed=4, empty=(0, Q - 1))
    c.prefix[:] = -1                                         # a prefix of no entry
    c.upload(gkr)
    out, lse = c.check(gkr)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    c = Case(gkr, Q, H, 0, 0, seed=4)
    out, lse = c.check(gkr)
    assert (out == 0).all() and torch.isneginf(lse).all()
    none = gkr.prefix_attention(c.q[:0], c.cache, c.args[2], c.args[3][:0], 1.0)
    assert none[0].shape == (0, H, 512)


@pytest.mark.parametrize("Q,H", [(3, 20), (20, 128)])
def test_bad_indices(gkr, Q, H):
    c = Case(gkr, Q, H, 400, 50, seed=5)
    c.prefix[[3, 200, 399]] = -2, c.slots, 2 ** 31 - 1
    c.upload(gkr)
    c.check(gkr)
    c.prefix[[3, 200, 399]] = -1
    c.idx[0, 3], c.idx[1, 49] = -2, c.slots
    c.upload(gkr)
    c.check(gkr)


@pytest.mark.parametrize("Q,H", [(3, 8), (20, 128)])
def test_nan_record(gkr, Q, H):
    """A NaN scale reaches whoever lists the record and no one else."""
    c = Case(gkr, Q, H, 300, 50, seed=6)
    c.prefix[c.prefix == 5] = 6
    c.idx[c.idx == 5] = 6
    c.idx[1, 7] = 5
    _, o = plain_mxfp4.offsets(5, c.bs, c.ps)
    c.host[o] = 255                                          # dims 0..31 of slot 5
    c.upload(gkr)
    out, lse = gkr.prefix_attention(*c.args)
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1].float()).all()
    rest = [i for i in range(Q) if i != 1]
    assert torch.isfinite(lse[rest]).all() and torch.isfinite(out[rest].float()).all()
    c.prefix[250] = 5
    c.upload(gkr)
    out, lse = gkr.prefix_attention(*c.args)
    assert torch.isnan(lse).all() and torch.isnan(out.float()).all()


def test_equals_the_lists_written_out(gkr):
    """The same as sparse_attention over each query's prefix and own list, within both tolerances."""
    c = Case(gkr, 24, 40, 900, 100, seed=7, pages=400)
    out, lse = c.check(gkr)
    whole = torch.cat([c.args[2].expand(24, 900), c.args[3]], 1).contiguous()
    o2, l2 = gkr.sparse_attention(c.q, c.cache, whole, c.sm)
    t_out, t_lse = plain.tolerances(c.want(), 1000)
    assert (np.abs((out.float() - o2.float()).cpu().numpy()) <= 2 * t_out).all()
    assert (np.abs((lse - l2).cpu().numpy()) <= 2 * t_lse).all()


@pytest.mark.parametrize("Q,H,L,K", [(24, 40, 900, 100), (3, 16, 2000, 50)])
def test_same_bits_on_streams_and_in_graphs(gkr, Q, H, L, K):
    c = Case(gkr, Q, H, L, K, seed=8)
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
    ws = [torch.zeros(max(size, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [(torch.zeros_like(want[0]), torch.zeros_like(want[1])) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, w, (o, l) in zip(graphs, ws, outs):
        with torch.cuda.graph(g):
            gkr.prefix_attention(*c.args, out=o, lse=l, workspace=w)
    for _ in range(3):
        with torch.cuda.stream(s):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for o, l in outs:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])
            o.zero_()
        torch.cuda.synchronize()
    with gkr.launch_policy(pdl=False):
        b = gkr.prefix_attention(*c.args)
    assert torch.equal(b[0], want[0])
    if size:
        with pytest.raises(ValueError):
            gkr.prefix_attention(*c.args, workspace=ws[0][:size - 1])


@pytest.mark.parametrize("record", [272, 528, 1024])
def test_a_batch_through_the_cache(gkr, record):
    """Prompts and their continuation: pages allocated, rows inserted, listed, gathered and attended to; what
    attention sees is what was inserted, as the cache's format rounds it."""
    rng = np.random.default_rng(9)
    bs, H, sm = 64, 16, 512 ** -0.5
    csc = torch.cat([torch.ones(1024, 32), torch.zeros(1024, 32)], 1).to(DEV)     # no rotation
    cache = gkr.alloc_cache(64, bs, record, DEV, fill=0)
    free = torch.from_numpy(rng.permutation(64).astype(np.int32)).to(DEV)
    table = torch.full((3, 12), -1, dtype=torch.int32, device=DEV)
    past = torch.zeros(3, dtype=torch.int32, device=DEV)
    latents = [[], [], []]
    used = 0
    for added in ([300, 70, 0], [1, 130, 64], [1, 1, 1]):
        n = sum(added)
        kv = torch.from_numpy(rng.standard_normal((n, 512))).to(torch.bfloat16).to(DEV)
        q = torch.from_numpy(2 * rng.standard_normal((n, H, 512))).to(torch.bfloat16).to(DEV)
        add = torch.tensor(added, dtype=torch.int32, device=DEV)
        slots, pos, starts, taken = gkr.kv_allocate(past, add, table, free[used:], bs, n + 2)
        used += int(taken.item())
        gkr.kv_insert(torch.cat([kv, kv[:2]]), cache, slots, pos, csc, bs)
        past = past + add
        idx, kv_starts = gkr.kv_slots_packed(table, past, bs, int(past.sum().item()))
        assert len(set(idx.tolist())) == len(idx) and int(idx.min()) >= 0
        rows = gkr.kv_gather(cache, idx, torch.empty(len(idx), 512, dtype=torch.bfloat16, device=DEV))
        at = 0
        for b, a in enumerate(added):
            latents[b].append(kv[at:at + a])
            at += a
        held = torch.cat([torch.cat(x) for x in latents])
        # 2^-4 of the block's largest value for e4m3, a quarter of it for e2m1 (steps 1/2 .. 2 of 6)
        amax = held.float().abs().view(-1, 16, 32).amax(2, keepdim=True).expand(-1, 16, 32).reshape(-1, 512)
        bound = {272: 0.25, 528: 2.0 ** -4, 1024: 0.0}[record] * amax
        assert ((rows.float() - held.float()).abs() <= bound).all()
        out, lse = gkr.prompt_attention(q, rows, starts, sm, kv_starts=kv_starts)
        r = plain.prompt(q.double().cpu().numpy(), rows.double().cpu().numpy(), starts.tolist(),
                         kv_starts.tolist(), sm)
        t_out, t_lse = plain.tolerances(r, 400)
        assert (np.abs(out.float().cpu().numpy() - r["out"]) <= t_out).all()
        assert (np.abs(lse.cpu().numpy() - r["lse"]) <= t_lse).all()
        if record == 272 and added == [1, 1, 1]:
            lists = gkr.kv_slots(table, past, bs, 400)
            o2, l2 = gkr.sparse_attention(q, cache, lists, sm)
            # requests 1 and 2 as if request 0's records came before their own
            pre = lists[0, :int(past[0].item())].contiguous()
            o3, l3 = gkr.prefix_attention(q[1:], cache, pre, lists[1:], sm)
            assert (np.abs(o2.float().cpu().numpy() - r["out"]) <= t_out).all()
            k = rows.double().cpu().numpy()
            for b in (1, 2):
                own = k[kv_starts[b]:kv_starts[b + 1]]
                w = plain.attend(q[b:b + 1].double().cpu().numpy(), np.concatenate([k[:kv_starts[1]], own]),
                                 [1000], sm)
                t_out3, t_lse3 = plain.tolerances(w, 800)
                assert (np.abs(o3[b - 1:b].float().cpu().numpy() - w["out"]) <= t_out3).all()
                assert (np.abs(l3[b - 1:b].cpu().numpy() - w["lse"]) <= t_lse3).all()
