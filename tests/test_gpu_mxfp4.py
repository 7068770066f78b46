"""GPU tests of the MXFP4 cache operators against the plain 64-bit implementations: the record's
write and read (byte for byte), sparse attention (within tolerances derived in plain_mxfp4) and
eviction (equal)."""
import numpy as np
import pytest
import torch

import plain_mxfp4 as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def flat(gkr, cache):
    return gkr.cache_bytes(cache).cpu().numpy()


# ------------------------------------------------------------------------------ write, read

def insert_case(T, bs, pages, seed, big=False):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, 512)) * np.exp(rng.standard_normal((T, 1)) * (20 if big else 1))
    x[rng.random((T, 512)) < 0.05] = 0.0
    x[rng.random((T, 512)) < 0.01] *= -0.0
    if T > 4:
        x[1] = 0.0
        x[2, :32] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 4)        # ties, scale 1
        x[3, 32:64] = np.array([7, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5] * 4)
        x[4, 5] = np.inf
    kv = plain.bf16_bits(x)
    if T > 4:
        kv[4, 5] = 0x7F80
    slots = rng.permutation(pages * bs)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    pos = rng.integers(0, 777, T)
    ang = rng.random((777, 32)) * 7
    csc = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    return kv, slots, pos, csc


@pytest.mark.parametrize("T,bs,pad,policy", [
    (1, 64, 0, {}), (300, 32, 512, {}), (257, 96, 1024, {"insert_staged_min": 0}),
    (300, 64, 512, {"insert_stream_min": 0})])
@pytest.mark.parametrize("big", [False, True])
def test_insert_and_gather(gkr, T, bs, pad, policy, big):
    pages = T // bs + 3
    kv, slots, pos, csc = insert_case(T, bs, pages, 7 * T + big, big)
    ps = gkr.page_stride(272, bs) + pad
    cache = gkr.alloc_cache(pages, bs, 272, DEV, page_stride_bytes=ps, fill=0xA5)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    with gkr.launch_policy(**policy):
        gkr.kv_insert(to_bf16(kv), cache, torch.from_numpy(slots).to(DEV),
                      torch.from_numpy(pos).to(DEV), torch.from_numpy(csc).to(DEV), bs, 272, err)
    want = np.full(pages * ps, 0xA5, np.uint8)
    for t in range(T):
        if slots[t] >= 0:
            d, s = plain.offsets(slots[t], bs, ps)
            want[d:d + 256], want[s:s + 16] = plain.encode(plain.rotate(plain.bf16(kv[t]), csc[pos[t]]))
    assert np.array_equal(flat(gkr, cache), want)
    idx = np.concatenate([slots[slots >= 0], [-1, -1]]).astype(np.int32)
    out = torch.empty(len(idx), 512, dtype=torch.bfloat16, device=DEV)
    gkr.kv_gather(cache, torch.from_numpy(idx).to(DEV), out, err)
    v = plain.decode(*plain.record_bytes(want, idx[:-2], bs, ps))
    got = out.float().cpu().numpy()
    with np.errstate(over="ignore"):
        assert np.array_equal(got[:-2].astype(np.float64),
                              np.where(np.abs(v) > 3.39e38, np.sign(v) * np.inf, v))
    assert (np.signbit(got[:-2]) == np.signbit(v)).all() and (got[-2:] == 0).all()
    assert int(err.item()) == 0


def test_gather_every_code_and_scale(gkr):
    """All 16 codes under all 256 scale bytes (255: NaN)."""
    bs, pages = 32, 8
    rng = np.random.default_rng(5)
    data = rng.integers(0, 256, (256, 256), dtype=np.uint8)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    ps = gkr.page_stride(272, bs)
    host = np.zeros(pages * ps, np.uint8)
    for s in range(256):
        d, c = plain.offsets(s, bs, ps)
        host[d:d + 256], host[c:c + 16] = data[s], scales[s]
    cache = gkr.alloc_cache(pages, bs, 272, DEV)
    gkr.cache_bytes(cache).copy_(torch.from_numpy(host))
    out = torch.empty(256, 512, dtype=torch.bfloat16, device=DEV)
    gkr.kv_gather(cache, torch.arange(256, dtype=torch.int32, device=DEV), out)
    got = out.float().cpu().numpy()
    v = plain.decode(data, scales)
    assert np.isnan(got[255]).all()
    with np.errstate(over="ignore"):                        # values of 2^128 and more: infinity
        assert np.array_equal(got[:255], np.where(np.abs(v[:255]) >= 2.0 ** 128,
                                                  np.copysign(np.inf, v[:255]), v[:255]).astype(np.float32))


def test_insert_errors(gkr):
    kv, slots, pos, csc = insert_case(8, 32, 4, 3)
    slots[:] = np.arange(8)
    slots[2], pos[5] = 128, 777
    cache = gkr.alloc_cache(4, 32, 272, DEV, fill=0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    gkr.kv_insert(to_bf16(kv), cache, torch.from_numpy(slots).to(DEV), torch.from_numpy(pos).to(DEV),
                  torch.from_numpy(csc).to(DEV), 32, 272, err)
    assert int(err.item()) == gkr.ERR_SLOT | gkr.ERR_POS
    rows = flat(gkr, cache)[:8 * 256].reshape(8, 256)
    assert (rows[2] == 0).all() and (rows[5] == 0).all() and rows[0].any()


def test_fused_write(gkr):
    T, H, Hp, bs = 70, 3, 4, 64
    kv, slots, pos, csc = insert_case(T, bs, 3, 11)
    kv[4, 5] = 0                                            # finite rows
    q = to_bf16(plain.bf16_bits(np.random.default_rng(2).standard_normal((T, H, 512))))
    a = gkr.alloc_cache(3, bs, 272, DEV, fill=0)
    b = gkr.alloc_cache(3, bs, 272, DEV, fill=0)
    c = gkr.alloc_cache(3, bs, 528, DEV, fill=0)
    args = [torch.from_numpy(x).to(DEV) for x in (slots, pos, csc)]
    gkr.kv_insert(to_bf16(kv), a, *args, bs)
    qa = gkr.qnorm_rope_kv_insert(q, to_bf16(kv), b, *args, Hp, 1e-6, bs)
    qb = gkr.qnorm_rope_kv_insert(q, to_bf16(kv), c, *args, Hp, 1e-6, bs)
    assert torch.equal(gkr.cache_bytes(a), gkr.cache_bytes(b))
    assert torch.equal(qa, qb)


# ------------------------------------------------------------------------------ attention

class Case:
    def __init__(self, gkr, Q, H, K, bs=64, pages=40, pad=0, seed=0, holes=0.1, qscale=2.0,
                 spread=1.0, sm_scale=512 ** -0.5, empty=(), index_pad=0):
        rng = np.random.default_rng(seed)
        self.bs, self.ps, self.slots = bs, gkr.page_stride(272, bs) + pad, pages * bs
        self.host = rng.integers(0, 256, pages * self.ps, dtype=np.uint8)
        s = np.clip(127 + np.round(spread * rng.standard_normal((self.slots, 16)) - 1.5), 0, 254)
        for slot in range(self.slots):
            _, o = plain.offsets(slot, bs, self.ps)
            self.host[o:o + 16] = s[slot]
        idx = rng.integers(0, self.slots, (Q, K)).astype(np.int32)
        idx[rng.random((Q, K)) < holes] = -1
        for i in empty:
            idx[i] = -1
        self.idx, self.sm = idx, sm_scale
        self.qbits = plain.bf16_bits(qscale * rng.standard_normal((Q, H, 512)))
        self.w0 = rng.random((Q, K)).astype(np.float32)
        self.q = to_bf16(self.qbits)
        self.cache = gkr.alloc_cache(pages, bs, 272, DEV, page_stride_bytes=self.ps)
        gkr.cache_bytes(self.cache).copy_(torch.from_numpy(self.host))
        wide = torch.full((Q, K + index_pad), 7, dtype=torch.int32, device=DEV)
        wide[:, :K] = torch.from_numpy(idx)
        self.indices = wide[:, :K]
        ww = torch.full((Q, K + index_pad), 7.0, device=DEV)
        ww[:, :K] = torch.from_numpy(self.w0)
        self.weights, self.wide_weights = ww[:, :K], ww

    def want(self):
        r = plain.attention(plain.bf16(self.qbits).astype(np.float64), self.host, self.bs, self.ps,
                            self.slots, self.idx, self.sm)
        return r, plain.tolerances(r, self.idx.shape[1])

    def check(self, gkr, weights=True, **kw):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, lse = gkr.sparse_attention(self.q, self.cache, self.indices, self.sm,
                                        weights=self.weights if weights else None, err_flag=err, **kw)
        torch.cuda.synchronize()
        r, (t_out, t_lse, t_w) = self.want()
        got, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        some = np.isfinite(r["lse"])
        assert np.array_equal(np.isneginf(l), ~some)
        assert (np.abs(l - r["lse"])[some] <= t_lse[some]).all()
        worst = np.abs(got - r["out"]) - t_out
        assert (worst <= 0).all(), f"out: {np.unravel_index(worst.argmax(), worst.shape)} {worst.max()}"
        assert (got[~some] == 0).all()
        w = self.weights.cpu().numpy().astype(np.float64)
        if weights:
            want_w = self.w0 + r["p"].sum(1)
            assert (np.abs(w - want_w) <= t_w + 2.0 ** -23 * np.abs(want_w)).all()
            ok = (self.idx >= 0) & (self.idx < self.slots)
            assert np.array_equal(w[~ok], self.w0.astype(np.float64)[~ok])
        else:
            assert np.array_equal(w, self.w0.astype(np.float64))
        assert (self.wide_weights[:, self.idx.shape[1]:] == 7.0).all()
        bad = ((self.idx < -1) | (self.idx >= self.slots)).any()
        assert int(err.item()) == (gkr.ERR_INDEX if bad else 0)
        return out, lse


SIZES = [(1, 1, 1), (1, 128, 1), (1, 16, 31), (2, 5, 33), (3, 64, 64), (2, 65, 65), (1, 128, 128),
         (2, 127, 129), (5, 33, 257), (1, 8, 2047), (3, 128, 1000), (1, 128, 2049), (1, 7, 9001),
         (90, 16, 70), (170, 3, 5), (33, 128, 190)]


@pytest.mark.parametrize("Q,H,K", SIZES)
def test_attention_sizes(gkr, Q, H, K):
    Case(gkr, Q, H, K, seed=Q + H + K, index_pad=3).check(gkr)


@pytest.mark.parametrize("Q,H,K", [(2, 9, 40), (3, 128, 300)])
@pytest.mark.parametrize("kw", [
    dict(holes=0.0), dict(holes=0.97), dict(bs=96, pad=512), dict(bs=32, pad=1536),
    dict(sm_scale=-0.03), dict(sm_scale=0.0), dict(qscale=16.0), dict(qscale=0.0),
    dict(spread=4.0, qscale=0.5), dict(qscale=1e-30, sm_scale=1.0)])
def test_attention_kinds(gkr, Q, H, K, kw):
    Case(gkr, Q, H, K, seed=3, **kw).check(gkr)


def test_attention_without_weights(gkr):
    Case(gkr, 4, 32, 500, seed=8).check(gkr, weights=False)


@pytest.mark.parametrize("H", [4, 128])
def test_attention_empty_queries(gkr, H):
    Case(gkr, 4, H, 200, seed=9, empty=(0, 2)).check(gkr)
    Case(gkr, 2, H, 200, seed=9, empty=(0, 1)).check(gkr)
    c = Case(gkr, 3, H, 0, seed=9)
    out, lse = c.check(gkr)
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert gkr.sparse_attention(c.q[:0], c.cache, c.indices[:0], 1.0)[0].shape == (0, H, 512)


@pytest.mark.parametrize("lead", [64, 130, 1000])
def test_attention_first_entries_empty(gkr, lead):
    """Whole tiles without an entry before, between and after the valid ones."""
    c = Case(gkr, 2, 128, 2 * lead + 200, seed=10, holes=0.0)
    c.idx[:, :lead] = -1
    c.idx[0, lead + 3:2 * lead] = -1
    c.indices.copy_(torch.from_numpy(c.idx))
    c.check(gkr)


@pytest.mark.parametrize("rising", [True, False])
def test_attention_maximum_moves(gkr, rising):
    """Logits that climb (fall) by far over the list, so that the running maximum is replaced
    again and again (only once)."""
    c = Case(gkr, 2, 70, 700, seed=12, holes=0.0, qscale=1.0, sm_scale=1.0)
    r = plain.attention(plain.bf16(c.qbits).astype(np.float64), c.host, c.bs, c.ps, c.slots, c.idx, 1.0)
    for i in range(2):                                      # sorted by the first head's logit
        order = np.argsort(r["p"][i, 0], kind="stable")
        c.idx[i] = c.idx[i][order if rising else order[::-1]]
    c.indices.copy_(torch.from_numpy(c.idx))
    c.check(gkr)


def test_attention_bad_indices(gkr):
    c = Case(gkr, 3, 20, 150, seed=13)
    c.idx[0, 3], c.idx[1, 149], c.idx[2, 0] = -2, c.slots, 2 ** 31 - 1
    c.indices.copy_(torch.from_numpy(c.idx))
    c.check(gkr)


def test_attention_repeated_entries(gkr):
    c = Case(gkr, 2, 16, 100, seed=14)
    c.idx[0, :] = c.idx[0, 7]
    c.idx[1, 50:] = c.idx[1, :50]
    c.indices.copy_(torch.from_numpy(c.idx))
    c.check(gkr)


@pytest.mark.parametrize("H", [8, 128])
def test_attention_nan_record(gkr, H):
    """A NaN scale reaches the queries that list the record and no others, masked rows neither."""
    c = Case(gkr, 3, H, 130, seed=15)
    c.idx[c.idx == 5] = 6
    c.idx[1, 77] = 5
    c.indices.copy_(torch.from_numpy(c.idx))
    _, o = plain.offsets(5, c.bs, c.ps)
    gkr.cache_bytes(c.cache)[o] = 255                       # dims 0..31 of slot 5
    out, lse = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm)
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).all()
    assert torch.isfinite(lse[[0, 2]]).all() and torch.isfinite(out[[0, 2]].float()).all()


@pytest.mark.parametrize("byte", [0, 1, 129, 200])
def test_attention_far_scales(gkr, byte):
    """Scales at the ends of the range: subnormal values, and factors above 2 that the decode
    splits; the queries are scaled so that logits stay small."""
    c = Case(gkr, 2, 24, 90, seed=16, spread=0.0, sm_scale=2.0 ** (30 if byte > 1 else 100),
             qscale=2.0 ** ((127 - byte) - 32) if byte > 1 else 1.0)
    for slot in range(c.slots):
        _, o = plain.offsets(slot, c.bs, c.ps)
        c.host[o:o + 16] = byte
    gkr.cache_bytes(c.cache).copy_(torch.from_numpy(c.host))
    c.check(gkr)


def test_attention_same_bits_every_time(gkr):
    c = Case(gkr, 7, 128, 1500, seed=17)
    w = c.weights.clone()
    first = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, weights=w)
    for _ in range(3):
        w2 = c.weights.clone()
        again = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, weights=w2)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]) and torch.equal(w, w2)


def test_attention_streams_and_graph(gkr):
    c = Case(gkr, 6, 48, 900, seed=18)
    want = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.empty(gkr.sparse_attention_workspace(48, 6, 900), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, out=out, lse=lse, workspace=ws)
        kept = gkr.kv_evict(c.indices, c.weights, 100, 10)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    k = plain.evict(c.idx, c.weights.cpu().numpy(), 100, 10)
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(kept, k))
    with gkr.launch_policy(pdl=False):
        b = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm)
    assert torch.equal(b[0], want[0])


def test_attention_workspace_too_small(gkr):
    c = Case(gkr, 1, 128, 4000, seed=19)
    need = gkr.sparse_attention_workspace(128, 1, 4000)
    if need:
        with pytest.raises(ValueError):
            gkr.sparse_attention(c.q, c.cache, c.indices, c.sm,
                                 workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


def test_attention_far_slots(gkr):
    """Records beyond 4 GB into the cache: byte offsets past 32 bits."""
    bs, pages = 64, 270000                                  # 4.7 GB
    cache = gkr.alloc_cache(pages, bs, 272, DEV)
    slots = torch.tensor([[0, pages * bs - 1, pages * bs - 70, pages * bs // 2, 17]], dtype=torch.int32)
    rng = np.random.default_rng(4)
    kv = plain.bf16_bits(rng.standard_normal((5, 512)))
    csc = np.concatenate([np.ones((1, 32)), np.zeros((1, 32))], 1).astype(np.float32)
    gkr.kv_insert(to_bf16(kv), cache, slots[0].long().to(DEV), torch.zeros(5, dtype=torch.int64, device=DEV),
                  torch.from_numpy(csc).to(DEV), bs)
    qb = plain.bf16_bits(rng.standard_normal((1, 6, 512)))
    out, lse = gkr.sparse_attention(to_bf16(qb), cache, slots.to(DEV), 0.05)
    host = np.zeros(64 * 272, np.uint8)                     # the same five records, at slots 0..4
    for i in range(5):
        d, s = plain.offsets(i, 64, 64 * 272)
        host[d:d + 256], host[s:s + 16] = plain.encode(plain.bf16(kv[i]))
    r = plain.attention(plain.bf16(qb).astype(np.float64), host, 64, 64 * 272, 64,
                        np.arange(5, dtype=np.int32)[None], 0.05)
    t = plain.tolerances(r, 5)
    assert (np.abs(out.float().cpu().numpy() - r["out"]) <= t[0]).all()
    assert (np.abs(lse.cpu().numpy() - r["lse"]) <= t[1]).all()


# ------------------------------------------------------------------------------ eviction

def evict_check(gkr, idx, w, keep, recent, pad=0):
    B, L = idx.shape
    wi = torch.full((B, L + pad), 3, dtype=torch.int32, device=DEV)
    ww = torch.full((B, L + pad), 1e9, device=DEV)
    wi[:, :L], ww[:, :L] = torch.from_numpy(idx), torch.from_numpy(w)
    got = gkr.kv_evict(wi[:, :L], ww[:, :L], keep, recent)
    want = plain.evict(idx, w, keep, recent)
    for g, x in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), x, equal_nan=g.dtype == torch.float32), (keep, recent)


@pytest.mark.parametrize("B,L", [(1, 1), (3, 2), (2, 31), (5, 33), (2, 1000), (3, 1024), (2, 1025),
                                 (1, 4097), (4, 2049), (1, 40001), (2, 8192), (2, 8193), (1, 20000)])
def test_evict_sizes(gkr, B, L):
    rng = np.random.default_rng(B * L)
    idx = rng.permutation(B * L * 2)[:B * L].reshape(B, L).astype(np.int32)
    idx[rng.random((B, L)) < 0.1] = -1
    w = np.exp(2 * rng.standard_normal((B, L))).astype(np.float32)
    for keep, recent in {(0, 0), (L, 0), (L, L), (L // 2, 0), (L // 2, L // 4), (max(L - 1, 0), 0),
                         (min(1, L), min(1, L)), (L // 3, L // 3)}:
        evict_check(gkr, idx, w, keep, recent, pad=5)


@pytest.mark.parametrize("L", [50, 1500])
def test_evict_values(gkr, L):
    rng = np.random.default_rng(L)
    idx = np.arange(6 * L, dtype=np.int32).reshape(6, L)
    w = np.zeros((6, L), np.float32)                        # row 0: all equal
    w[1] = rng.integers(0, 3, L)                            # many ties
    w[2] = rng.choice([np.nan, -np.inf, np.inf, -1.0, 0.0, -0.0, 1e-40, 3.4e38], L)
    w[3] = -np.abs(rng.standard_normal(L))
    w[4] = 1.0 + rng.integers(0, 4, L) * 2.0 ** -23         # equal but for the last bits
    w[5] = np.nan
    for keep, recent in [(L // 2, 0), (L // 2, L // 5), (L - 1, 3), (1, 0), (3, 3)]:
        evict_check(gkr, idx, w, keep, recent)


def test_evict_sparse_rows(gkr):
    rng = np.random.default_rng(6)
    L = 3000
    idx = np.full((5, L), -1, np.int32)
    idx[1, 17] = 5
    idx[2, -1] = 6
    idx[3, ::7] = np.arange(len(idx[3, ::7]))
    idx[4, :900] = np.arange(900)
    w = rng.random((5, L)).astype(np.float32)
    w[idx < 0] = np.nan                                     # what empty entries hold is not read as weight
    for keep, recent in [(0, 0), (1, 0), (1, 1), (400, 0), (400, 399), (900, 100), (L, 50)]:
        evict_check(gkr, idx, w, keep, recent)


def test_evict_given_outputs(gkr):
    rng = np.random.default_rng(7)
    idx = rng.permutation(400).reshape(4, 100).astype(np.int32)
    w = rng.random((4, 100)).astype(np.float32)
    bufs = (torch.empty(4, 60, dtype=torch.int32, device=DEV), torch.empty(4, 60, device=DEV),
            torch.empty(4, 40, dtype=torch.int64, device=DEV))
    got = gkr.kv_evict(torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV), 60, 10, *bufs)
    assert all(a is b for a, b in zip(got, bufs))
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(got, plain.evict(idx, w, 60, 10)))


@pytest.mark.parametrize("L", [8200, 300000])
def test_evict_ties_across_parts(gkr, L):
    """Rows split over a cluster: ties, empty entries and the newest ones anywhere; and rows too long
    for their keys to be held."""
    rng = np.random.default_rng(L)
    idx = np.arange(3 * L, dtype=np.int32).reshape(3, L)
    idx[1, rng.random(L) < 0.5] = -1
    idx[2, : L // 2] = -1
    w = rng.integers(0, 3, (3, L)).astype(np.float32)
    w[2] = 1.0
    for keep, recent in [(L // 2, 0), (L // 3, L // 4), (L - 1, 7), (5, 5)]:
        evict_check(gkr, idx, w, keep, recent)


@pytest.mark.parametrize("Q,H,K,holes", [(64, 128, 700, 0.3), (200, 128, 130, 0.0), (160, 32, 130, 0.5),
                                         (5, 64, 3000, 0.6)])
def test_attention_again_and_again(gkr, Q, H, K, holes):
    """Masks that differ from chunk to chunk, and queries that follow one another on an SM: the
    first results are right, and the same bits come every time, whatever ran before."""
    c = Case(gkr, Q, H, K, holes=holes, seed=Q, pages=40)
    out, lse = c.check(gkr)
    w = c.weights.clone()
    for i in range(60):
        if i % 3 == 0:   # other work between, so that timing differs
            torch.full((1 << (18 + i % 8),), float("nan"), device=DEV)
        c.weights.copy_(torch.from_numpy(c.w0))
        o, l = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, weights=c.weights)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)), i
        assert torch.equal(l, lse) and torch.equal(c.weights, w), i


@pytest.mark.parametrize("Q,H,K", [(64, 8, 2049), (76, 128, 640)])
def test_attention_ragged_again_and_again(gkr, Q, H, K):
    """The same for lists of many lengths in a cache that is not in the L2 cache when they start."""
    c = Case(gkr, Q, H, K, seed=K, pages=1500, holes=0.05)
    rng = np.random.default_rng(Q)
    for i, n in enumerate(rng.integers(0, K + 1, Q)):
        c.idx[i, n:] = -1
    c.indices.copy_(torch.from_numpy(c.idx))
    out, lse = c.check(gkr)
    w = c.weights.clone()
    for i in range(60):
        torch.full((1 << 26,), float("nan"), device=DEV)   # 256 MB
        c.weights.copy_(torch.from_numpy(c.w0))
        o, l = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, weights=c.weights)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)), i
        assert torch.equal(l, lse) and torch.equal(c.weights, w), i
