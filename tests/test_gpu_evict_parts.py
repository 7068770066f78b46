"""kv_evict where a row's parts are of other sizes than the small cases': keys held and slots read again
(20481 to 36864 entries of a CTA), many rows (which changes the CTAs a row gets), the longest list that is
taken, and calls from several host threads at the same time."""
import threading

import numpy as np
import pytest
import torch

import plain_mxfp4 as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def by_sorting(idx, w, keep, recent):
    """plain.evict for long lists: one sort a row."""
    rows, length = idx.shape
    kept = np.full((rows, keep), -1, np.int32)
    kept_w = np.zeros((rows, keep), np.float32)
    gone = np.full((rows, length - keep), -1, np.int64)
    for r in range(rows):
        live = np.flatnonzero(idx[r] >= 0)
        cut = max(0, len(live) - recent)
        old, new = live[:cut], live[cut:]
        x = w[r, old].astype(np.float64)
        best = old[np.lexsort((old, -x, np.isnan(x)))[:keep - len(new)]]
        mine = np.sort(np.concatenate([best, new]))
        rest = np.setdiff1d(live, mine)
        kept[r, :len(mine)], kept_w[r, :len(mine)] = idx[r, mine], w[r, mine]
        gone[r, :len(rest)] = idx[r, rest]
    return kept, kept_w, gone


def rows_of(B, L, seed):
    """Rows of different kinds: weights of three values (ties across parts), spread ones, NaN and
    infinities among them, empty entries anywhere or in the first half."""
    rng = np.random.default_rng(seed)
    idx = rng.integers(0, 1 << 30, (B, L)).astype(np.int32)
    w = np.exp(2 * rng.standard_normal((B, L))).astype(np.float32)
    for r in range(B):
        if r % 3 == 0:
            w[r] = rng.integers(0, 3, L)
        if r % 3 == 1:
            idx[r, rng.random(L) < 0.3] = -1
            w[r, rng.random(L) < 0.05] = np.nan
            w[r, rng.random(L) < 0.01] = np.inf
        if r % 3 == 2:
            idx[r, :L // 2] = -7
            w[r, rng.random(L) < 0.2] = -0.0
    return idx, w


def check(gkr, idx, w, keep, recent):
    got = gkr.kv_evict(torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV), keep, recent)
    for g, x in zip(got, by_sorting(idx, w, keep, recent)):
        assert np.array_equal(g.cpu().numpy(), x, equal_nan=g.dtype == torch.float32), (keep, recent)


def test_by_sorting_is_the_plain_form():
    idx, w = rows_of(6, 57, 1)
    for keep, recent in ((0, 0), (20, 0), (20, 9), (57, 3), (41, 41)):
        for a, b in zip(by_sorting(idx, w, keep, recent), plain.evict(idx, w, keep, recent)):
            assert np.array_equal(a, b, equal_nan=a.dtype == np.float32)


# eight CTAs a row: parts of 20481.., 25000, 36864 entries; 36865: the keys no longer fit
@pytest.mark.parametrize("L", [8 * 20480, 8 * 20480 + 1, 200000, 8 * 36864, 8 * 36864 + 1])
def test_parts_of_long_rows(gkr, L):
    idx, w = rows_of(3, L, L)
    for keep, recent in ((4096, 1024), (L // 2, 0), (L - 1, 0), (L // 3, L // 3), (L // 5, 3)):
        check(gkr, idx, w, keep, recent)


# many rows get fewer CTAs each: parts of 2561 .. 36864 entries by one, two and four of them
@pytest.mark.parametrize("B,L", [(130, 2561), (65, 9000), (33, 8200), (17, 30000), (70, 21000), (64, 36864), (9, 36865),
                                 (64, 65536), (40, 73729)])
def test_many_rows(gkr, B, L):
    idx, w = rows_of(B, L, B + L)
    for keep, recent in ((L // 2, L // 8), (L - 1, 5), (min(2048, L // 3), 0)):
        check(gkr, idx, w, keep, recent)


def test_the_longest_list(gkr):
    L = 1 << 21
    idx, w = rows_of(2, L, 5)
    check(gkr, idx, w, 100000, 5000)
    check(gkr, idx, w, L - 1, 0)
    with pytest.raises(ValueError):
        gkr.kv_evict(torch.zeros(1, L + 1, dtype=torch.int32, device=DEV), torch.zeros(1, L + 1, device=DEV), 10)


def test_threads_on_separate_streams(gkr):
    """Insert, attention with weights and eviction from several host threads, each on a stream and a
    cache of its own: every result is the one that a thread alone gets."""
    sizes = [(3, 16, 700, 300), (40, 8, 130, 90), (2, 128, 1500, 800), (1, 64, 5000, 10), (17, 100, 257, 256)]
    bs = 64

    def inputs(i):
        Q, H, K, _ = sizes[i]
        g = torch.Generator(device=DEV).manual_seed(i)
        pages = -(-2 * K // bs)
        kv = torch.randn(pages * bs, 512, generator=g, device=DEV).bfloat16()
        slots = torch.randperm(pages * bs, generator=g, device=DEV)
        csc = torch.randn(pages * bs, 64, generator=g, device=DEV)
        q = torch.randn(Q, H, 512, generator=g, device=DEV).bfloat16()
        idx = torch.randint(-1, pages * bs, (Q, K), generator=g, device=DEV, dtype=torch.int32)
        return pages, kv, slots, csc, q, idx

    def run(i, x):
        pages, kv, slots, csc, q, idx = x
        cache = gkr.alloc_cache(pages, bs, gkr.MXFP4, DEV, fill=0)
        w = torch.zeros(idx.shape, device=DEV)
        gkr.kv_insert(kv, cache, slots, torch.arange(len(slots), device=DEV), csc, bs)
        for _ in range(6):
            out, lse = gkr.sparse_attention(q, cache, idx, 512 ** -0.5, weights=w)
        return (out, lse, w, *gkr.kv_evict(idx, w, sizes[i][3], 5))

    xs = [inputs(i) for i in range(len(sizes))]
    want = [run(i, x) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    got, errors, barrier = [None] * len(sizes), [], threading.Barrier(len(sizes))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                barrier.wait(timeout=60)
                for _ in range(4):
                    got[i] = run(i, xs[i])
            stream.synchronize()
        except Exception as e:            # reported after the join
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not errors, errors
    for i, (a, b) in enumerate(zip(got, want)):
        for x, y in zip(a, b):
            assert torch.equal(x, y), i
