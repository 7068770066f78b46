"""GPU tests of kv_allocate, kv_slots and kv_slots_packed against the plain form (all equal)."""
import numpy as np
import pytest
import torch

import plain_paged as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).to(DEV)


def batch(B, most_past, most_added, bs, seed, pad=0):
    """Lengths, a table with pages for what is held, a free list and how many tokens there are."""
    rng = np.random.default_rng(seed)
    past = rng.integers(0, most_past + 1, B)
    added = rng.integers(0, most_added + 1, B)
    past[rng.random(B) < 0.2] = 0
    added[rng.random(B) < 0.2] = 0
    W = max(1, int(-(-(past + added).max() // bs))) if B else 3
    table = np.full((B, W + pad), -1, np.int64)
    held = -(-past // bs)
    pool = rng.permutation(int(held.sum()) + 5)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pool[at:at + held[b]]
        at += held[b]
    need = int((-(-(past + added) // bs) - held).sum()) if B else 0
    free = len(pool) + rng.permutation(need + 7)
    return past, added, table, free, need, int(added.sum())


def check(gkr, past, added, table, W, free, bs, rows, guard=3):
    """Runs it twice; outputs behind the given rows stay as they are."""
    want = plain.allocate(past, added, table[:, :W], free, bs, rows)
    t = dev(table)
    B = len(past)
    out = [torch.full((rows + guard,), 77, dtype=torch.int64, device=DEV) for _ in range(2)]
    out += [torch.full((B + 1 + guard,), 77, dtype=torch.int32, device=DEV),
            torch.full((1 + guard,), 77, dtype=torch.int32, device=DEV)]
    sizes = (rows, rows, B + 1, 1)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(2):
        gkr.kv_allocate(dev(past), dev(added), t[:, :W], dev(free), bs, rows,
                        *(o[:n] for o, n in zip(out, sizes)), err_flag=err)
    for o, n, w in zip(out, sizes, want):
        assert np.array_equal(o[:n].cpu().numpy(), np.atleast_1d(w)), (o, w)
        assert (o[n:] == 77).all()
    got = t.cpu().numpy()
    assert np.array_equal(got[:, :W], want[4]) and np.array_equal(got[:, W:], table[:, W:])
    assert int(err.item()) == want[5]
    return want


@pytest.mark.parametrize("B,past,added,bs", [
    (1, 0, 1, 64), (1, 100, 0, 64), (3, 10, 5, 4), (64, 8192, 1, 64), (33, 300, 200, 48), (7, 50, 5000, 1),
    (512, 1000, 40, 32), (1500, 100, 30, 64), (5, 100000, 70000, 64), (4097, 20, 3, 16), (16384, 9, 2, 64)])
def test_allocate(gkr, B, past, added, bs):
    for seed in range(2):
        p, a, table, free, need, rows = batch(B, past, added, bs, 10 * B + seed, pad=seed * 3)
        want = check(gkr, p, a, table, table.shape[1] - seed * 3, free, bs, rows + 5 * seed)
        assert want[5] == 0 and want[3] == need


def test_allocate_edges(gkr):
    p, a, table, free, need, rows = batch(20, 200, 200, 16, 3)
    W = table.shape[1]
    assert check(gkr, p, a, table, W, free[:need - 3], 16, rows)[5] == plain.ERR_SLOT      # list too short
    assert check(gkr, p, a, table, W, free[:0], 16, rows)[5] == plain.ERR_SLOT
    assert check(gkr, p, a, table, W - 4, free, 16, rows)[5] == plain.ERR_SLOT             # table too narrow
    assert check(gkr, p, a, table, W, free, 16, rows - 7)[5] == plain.ERR_SLOT             # too few rows
    assert check(gkr, p, a, table, W, free, 16, 0)[5] == plain.ERR_SLOT
    table[3, 0], p[3], a[3] = -1, 5, 2                                                     # a page is missing
    assert check(gkr, p, a, table, W, free, 16, int(a.sum()))[5] == plain.ERR_SLOT
    p[7], a[9] = -3, -4
    assert check(gkr, p, a, table, W, free, 16, rows)[5] & plain.ERR_POS
    empty = np.zeros(0, np.int64)
    got = check(gkr, empty, empty, np.zeros((0, 3), np.int64), 3, free, 16, 6)             # no request
    assert got[3] == 0 and (got[0] == -1).all()
    check(gkr, p, a, np.zeros((20, 0), np.int64), 0, free, 16, rows)


def test_allocate_far(gkr):
    """Positions and slots past 32 bits, and sums that end at 2^31 - 1."""
    big = 2 ** 31 - 5
    table = np.full((2, 4), 2 ** 30, np.int64)
    want = check(gkr, np.array([big, 3]), np.array([10, 4]), table, 4, np.arange(9), 2 ** 30, 14)
    assert want[1].max() == big + 9 and want[0].max() >= 2 ** 60
    past, added = np.zeros(3, np.int64), np.array([2 ** 31 - 1, 2 ** 31 - 1, 5])
    out = gkr.kv_allocate(dev(past), dev(added), dev(np.full((3, 2), -1)), dev(np.arange(3)), 64, 200)
    assert out[2].tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert out[0][:64].tolist() == list(range(64)) and (out[0][128:] == -1).all()
    assert out[1].tolist() == list(range(200)) and int(out[3].item()) == 3


def tables(B, lengths, bs, seed, pad=0):
    rng = np.random.default_rng(seed)
    W = max(1, int(-(-max(lengths) // bs))) if B else 1
    return rng.permutation(B * W).reshape(B, W) if B else np.zeros((0, 1), np.int64), W


@pytest.mark.parametrize("B,length,bs", [(1, 1, 64), (3, 7, 4), (64, 8191, 64), (5, 70000, 48), (700, 33, 16),
                                         (5000, 5, 64), (1, 300000, 32)])
@pytest.mark.parametrize("window", [None, 20])
def test_slots(gkr, B, length, bs, window):
    rng = np.random.default_rng(B + length)
    n = rng.integers(0, length + 1, B)
    n[rng.random(B) < 0.2] = 0
    n[0] = length
    first = None if window is None else np.maximum(n - window, 0)
    table, W = tables(B, n, bs, 1)
    wide = np.concatenate([table, np.full((B, 3), 12345)], 1)
    rows, bits = plain.slots(table, n, bs, first)
    assert bits == 0
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    width = max(len(r) for r in rows) + 2
    f = None if first is None else dev(first)
    got = gkr.kv_slots(dev(wide)[:, :W], dev(n), bs, width, f, err_flag=err).cpu().numpy()
    want = np.full((B, width), -1, np.int64)
    for b, r in enumerate(rows):
        want[b, :len(r)] = r
    assert np.array_equal(got, want)
    flat = np.concatenate([np.asarray(r, np.int64) for r in rows])
    for extra in (0, 9):
        idx, starts = gkr.kv_slots_packed(dev(wide)[:, :W], dev(n), bs, len(flat) + extra, f, err_flag=err)
        assert np.array_equal(idx.cpu().numpy(), np.concatenate([flat, np.full(extra, -1)]))
        assert np.array_equal(starts.cpu().numpy(), np.concatenate([[0], np.cumsum([len(r) for r in rows])]))
    assert int(err.item()) == 0


def test_slots_errors(gkr):
    table = np.array([[3, -1], [2 ** 31 - 1, 0], [0, 1]])

    def run(lengths, width, first=None, bs=4):
        err = torch.zeros(2, dtype=torch.int32, device=DEV)
        f = None if first is None else dev(first)
        a = gkr.kv_slots(dev(table), dev(lengths), bs, width, f, err_flag=err)
        b = gkr.kv_slots_packed(dev(table), dev(lengths), bs, 3 * width, f, err_flag=err[1:])
        assert err[0] == err[1]
        return a.tolist(), b[0].tolist(), b[1].tolist(), int(err[0].item())

    a, b, s, bits = run([4, 0, 3], 4)
    assert a == [[12, 13, 14, 15], [-1] * 4, [0, 1, 2, -1]] and bits == 0
    assert b == [12, 13, 14, 15, 0, 1, 2] + [-1] * 5 and s == [0, 4, 4, 7]
    a, b, s, bits = run([5, 2, 9], 12)                       # no page; no int32; past the table
    assert a[0][4] == -1 and a[1][:2] == [-1, -1] and a[2][7:] == [7, -1, -1, -1, -1]
    assert bits == gkr.ERR_INDEX and s == [0, 5, 7, 16]
    assert run([-2, 0, 1], 4)[3] == gkr.ERR_INDEX
    assert run([2, 0, 1], 4, first=[-1, 5, 0])[3] == gkr.ERR_INDEX
    assert run([2, 0, 1], 4, first=[1, 5, 0])[0] == [[13, -1, -1, -1], [-1] * 4, [0, -1, -1, -1]]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert gkr.kv_slots(dev(table), dev([3, 0, 1]), 4, 2, err_flag=err).tolist() == [[12, 13], [-1, -1], [0, -1]]
    assert int(err.item()) == gkr.ERR_INDEX                  # a row is too short
    err.zero_()
    got, s = gkr.kv_slots_packed(dev(table), dev([3, 0, 1]), 4, 2, err_flag=err)
    assert got.tolist() == [12, 13] and s.tolist() == [0, 3, 3, 4] and int(err.item()) == gkr.ERR_INDEX
    # nothing to do
    assert gkr.kv_slots(dev(table)[:0], dev([]), 4, 5).shape == (0, 5)
    got, s = gkr.kv_slots_packed(dev(table)[:0], dev([]), 4, 3)
    assert got.tolist() == [-1] * 3 and s.tolist() == [0]


def test_plan_on_another_stream_and_in_a_graph(gkr):
    p, a, table, free, need, rows = batch(40, 300, 50, 64, 5)
    want = plain.allocate(p, a, table, free, 64, rows + 3)
    args = dev(p), dev(a), dev(table), dev(free)
    lists, _ = plain.slots(want[4], p + a, 64)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gkr.kv_allocate(*args, 64, rows + 3)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        out = gkr.kv_allocate(*args, 64, rows + 3)
        # in the same graph: the lists over what the table then holds
        idx, starts = gkr.kv_slots_packed(args[2], args[0] + args[1], 64, int((p + a).sum()))
    for _ in range(2):
        for o in (*out, idx, starts):
            o.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(out, want):
            assert np.array_equal(o.cpu().numpy(), np.atleast_1d(w))
        assert np.array_equal(idx.cpu().numpy(), np.concatenate([np.asarray(r, np.int64) for r in lists]))
