"""CPU tests of the operators of a batch's way through a paged cache: the plain forms pinned by
hand, the refusals of the C entries (fake pointers never reach a kernel: every call fails a host
check or enqueues nothing) and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import plain_paged as plain

A, B = 0x10000, 0x20000000          # fake pointers, 16-byte aligned and far apart


def test_plain_allocate_pin():
    # 3 requests, pages of 4: 5 held + 4 (pages 7, 2 -> third page 30), 0 + 0, 8 + 1
    table = np.array([[7, 2, -1], [-1, -1, -1], [9, 8, -1]])
    slots, pos, starts, taken, out, bits = plain.allocate([5, 0, 8], [4, 0, 1], table, [30, 31, 32], 4, 7)
    assert slots.tolist() == [9, 10, 11, 120, 124, -1, -1]
    assert pos.tolist() == [5, 6, 7, 8, 8, 0, 0] and starts.tolist() == [0, 4, 4, 5]
    assert taken == 2 and out.tolist() == [[7, 2, 30], [-1, -1, -1], [9, 8, 31]] and bits == 0
    # the list is one short
    slots, _, _, taken, out, bits = plain.allocate([5, 0, 8], [4, 0, 1], table, [30], 4, 5)
    assert slots.tolist() == [9, 10, 11, 120, -1] and taken == 1 and bits == plain.ERR_SLOT
    assert out[2].tolist() == [9, 8, -1]


def test_plain_slots_pin():
    rows, bits = plain.slots([[3, 1], [5, -1]], [3, 1], 2)
    assert rows == [[6, 7, 2], [10]] and bits == 0
    rows, bits = plain.slots([[3, 1], [5, -1]], [3, 3], 2, first=[1, 1])
    assert rows == [[7, 2], [11, -1]] and bits == plain.ERR_INDEX


def test_plain_prompt_pin():
    # one dim of 512 is used: two rows with values 1 and 3, logits 0 and ln 3 -> weights 1/4, 3/4
    q, kv = np.zeros((2, 1, 512)), np.zeros((3, 512))
    q[:, 0, 0] = np.log(3.0)
    kv[:3, 0], kv[:3, 1] = [0.0, 1.0, 0.0], [1.0, 3.0, 100.0]
    r = plain.prompt(q, kv[:2], [0, 2], [0, 2], 1.0)
    assert np.allclose(r["out"][0, 0, 1], 1.0) and np.allclose(r["out"][1, 0, 1], 2.5)
    assert np.allclose(r["lse"][:, 0], [0.0, np.log(4.0)])
    assert np.allclose(plain.prompt(q, kv[:2], [0, 2], [0, 2], 1.0, causal=False)["out"][:, 0, 1], 2.5)
    # one row for two queries: the first sees none
    r = plain.prompt(q, kv[:1], [0, 2], [0, 1], 1.0)
    assert np.isneginf(r["lse"][0, 0]) and (r["out"][0] == 0).all() and r["out"][1, 0, 1] == 1.0


def allocate(gkr, past=A, added=A, n=2, table=A, stride=8, width=8, free=A, num_free=4, bs=64, tokens=5,
             slots=A, pos=A, starts=A, taken=A, err=None, opts=None):
    return gkr.lib().gkr_kv_allocate(past, added, n, table, stride, width, free, num_free, bs, tokens, slots,
                                     pos, starts, taken, err, opts, None)


def slots(gkr, table=A, stride=8, width=8, lengths=A, first=None, n=2, bs=64, out=16, idx=A, starts=None,
          err=None, opts=None):
    return gkr.lib().gkr_kv_slots(table, stride, width, lengths, first, n, bs, out, idx, starts, err, opts, None)


def prompt(gkr, q=A, H=2, T=4, kv=A, stride=512, rows=4, starts=A, kstarts=A, n=1, causal=1, scale=1.0, out=B,
           lse=A, ws=A, bytes_=1 << 40, err=None, opts=None):
    return gkr.lib().gkr_prompt_attention(q, H, T, kv, stride, rows, starts, kstarts, n, causal, scale, out, lse,
                                          ws, bytes_, err, opts, None)


def prefix(gkr, d=(272, 64, 4), q=A, H=2, cache=A, pre=A, L=8, idx=A, stride=8, Q=2, K=8, scale=1.0, out=B,
           lse=A, ws=A, bytes_=1 << 40, err=None, opts=None, ps=None):
    d = None if d is None else gkr.CacheDesc(*d, gkr.page_stride(d[0], d[1]) if ps is None else ps)
    return gkr.lib().gkr_prefix_attention(q, H, cache, None if d is None else ctypes.byref(d), pre, L, idx,
                                          stride, Q, K, scale, out, lse, ws, bytes_, err, opts, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=16385), dict(width=-1), dict(stride=7), dict(num_free=-1), dict(num_free=1 << 31),
    dict(bs=0), dict(bs=-64), dict(tokens=-1), dict(tokens=1 << 31), dict(past=None), dict(added=None),
    dict(table=None), dict(free=None), dict(slots=None), dict(pos=None), dict(starts=None), dict(taken=None)])
def test_allocate_refusals(gkr, bad):
    assert allocate(gkr, **bad) == 1


@pytest.mark.parametrize("bad", ["past", "added", "table", "free", "slots", "pos", "starts", "taken", "err"])
def test_allocate_alignment(gkr, bad):
    assert allocate(gkr, **{bad: A + (4 if bad in ("slots", "pos") else 2)}) == 4


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=16385, starts=A), dict(width=-1), dict(stride=7), dict(bs=0), dict(out=-1),
    dict(out=1 << 31), dict(table=None), dict(lengths=None), dict(idx=None),
    dict(n=(1 << 31) - 1, out=1 << 20)])
def test_slots_refusals(gkr, bad):
    assert slots(gkr, **bad) == 1


def test_slots_alignment_and_nothing(gkr):
    for bad in ("table", "lengths", "first", "idx", "starts", "err"):
        assert slots(gkr, **{bad: A + 2}) == 4, bad
    assert slots(gkr, n=0, table=None, lengths=None, idx=None) == 0
    assert slots(gkr, out=0, idx=None) == 0


@pytest.mark.parametrize("bad", [
    dict(H=0), dict(H=4097), dict(T=-1), dict(T=1 << 31), dict(H=4096, T=1 << 20), dict(rows=-1),
    dict(rows=1 << 31), dict(stride=511), dict(stride=516), dict(n=-1), dict(n=16385), dict(causal=2),
    dict(causal=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(q=None), dict(kv=None),
    dict(starts=None), dict(kstarts=None), dict(out=None), dict(lse=None), dict(out=A), dict(out=A + 4096),
    dict(kv=B), dict(kv=B - 1024, rows=2)])
def test_prompt_refusals(gkr, bad):
    assert prompt(gkr, **bad) == 1


def test_prompt_alignment_and_nothing(gkr):
    for bad in ("q", "kv", "starts", "kstarts", "lse", "err"):
        assert prompt(gkr, **{bad: A + 2}) == 4, bad
    assert prompt(gkr, out=B + 8) == 4
    assert prompt(gkr, T=0, q=None, kv=None, starts=None, kstarts=None, out=None, lse=None, ws=None, bytes_=0) == 0
    assert prompt(gkr, n=0, q=None, kv=None, starts=None, kstarts=None, out=None, lse=None, ws=None, bytes_=0) == 0
    n = ctypes.c_int64(7)
    ws = gkr.lib().gkr_prompt_attention_workspace
    assert ws(0, 1, ctypes.byref(n)) == 1 and ws(4, 1 << 31, ctypes.byref(n)) == 1 and ws(4, 4, None) == 1
    assert ws(4, 0, ctypes.byref(n)) == 0 and n.value == 0


@pytest.mark.parametrize("bad", [
    dict(H=0), dict(H=129), dict(Q=-1), dict(Q=(1 << 24) + 1), dict(L=-1), dict(L=(1 << 24) + 1), dict(K=-1),
    dict(K=(1 << 24) + 1, stride=1 << 25), dict(stride=7), dict(scale=float("inf")), dict(q=None),
    dict(cache=None), dict(pre=None), dict(idx=None), dict(out=None), dict(lse=None), dict(out=A),
    dict(Q=1 << 20, K=1 << 20, stride=1 << 20), dict(d=None), dict(H=128, Q=1 << 24)])
def test_prefix_refusals(gkr, bad):
    assert prefix(gkr, **bad) == 1


def test_prefix_formats_alignment_and_nothing(gkr):
    for rec in (528, 584, 512, 1024):
        assert prefix(gkr, d=(rec, 64, 4)) == 2
    assert prefix(gkr, ps=64 * 272 - 512) == 3
    for bad in ("q", "cache", "pre", "idx", "lse", "err"):
        assert prefix(gkr, **{bad: A + 2}) == 4, bad
    assert prefix(gkr, out=B + 8) == 4
    assert prefix(gkr, Q=0, q=None, cache=None, pre=None, idx=None, out=None, lse=None, ws=None, bytes_=0) == 0
    n = ctypes.c_int64(7)
    ws = gkr.lib().gkr_prefix_attention_workspace
    assert ws(129, 1, 1, 1, ctypes.byref(n)) == 1 and ws(4, -1, 1, 1, ctypes.byref(n)) == 1
    assert ws(4, 1, 1, 1, None) == 1 and ws(4, 0, 1, 1, ctypes.byref(n)) == 0 and n.value == 0


def test_launch_options_are_checked(gkr):
    bad = ctypes.byref(gkr.LaunchOpts())
    bad._obj.pdl = 2
    assert allocate(gkr, opts=bad) == 1 and slots(gkr, opts=bad) == 1
    assert prompt(gkr, opts=bad) == 1 and prefix(gkr, opts=bad) == 1


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_rejects_bad_tensors(gkr):
    ok = (i32(2), i32(2), i32(2, 8), i32(4), 64, 5)

    def but(args, at, value):
        return tuple(value if i == at else a for i, a in enumerate(args))

    cases = [
        (gkr.kv_allocate, but(ok, 0, i32(2, 1)), "past"), (gkr.kv_allocate, but(ok, 1, i32(3)), "added"),
        (gkr.kv_allocate, but(ok, 1, i32(2).long()), "added"),
        (gkr.kv_allocate, but(ok, 2, i32(3, 8)), "row for each"),
        (gkr.kv_allocate, but(ok, 2, i32(2, 8).long()), "block_table"),
        (gkr.kv_allocate, but(ok, 2, i32(8, 2).T), "block_table"),
        (gkr.kv_allocate, but(ok, 3, i32(4, 1)), "free_pages"),
        (gkr.kv_allocate, but(ok, 5, -1), "num_tokens"), (gkr.kv_allocate, but(ok, 5, 1 << 31), "num_tokens"),
        (gkr.kv_allocate, ok, "CUDA"),
        (gkr.kv_slots, (i32(2, 8), i32(3), 64, 5), "row for each"),
        (gkr.kv_slots, (i32(2, 8), i32(2), 64, -1), "width"),
        (gkr.kv_slots, (i32(2, 8), i32(2), 64, 5, i32(3)), "first"),
        (gkr.kv_slots, (i32(2, 8), i32(2), 64, 5), "CUDA"),
        (gkr.kv_slots_packed, (i32(2, 8), i32(2).float(), 64, 5), "lengths"),
        (gkr.kv_slots_packed, (i32(2, 8), i32(2), 64, 1 << 31), "total"),
        (gkr.prompt_attention, (bf16(4, 2, 512).float(), bf16(4, 512), i32(2), 1.0), "q must"),
        (gkr.prompt_attention, (bf16(4, 2, 256), bf16(4, 512), i32(2), 1.0), "q must"),
        (gkr.prompt_attention, (bf16(4, 2, 512), bf16(4, 256), i32(2), 1.0), "kv must"),
        (gkr.prompt_attention, (bf16(4, 2, 512), bf16(4, 516)[:, :512], i32(2), 1.0), "kv must"),
        (gkr.prompt_attention, (bf16(4, 2, 512), bf16(4, 512), i32(0), 1.0), "starts"),
        (gkr.prompt_attention, (bf16(4, 2, 512), bf16(4, 512), i32(2), 1.0, i32(3)), "kv_starts"),
        (gkr.prompt_attention, (bf16(4, 2, 512), bf16(4, 512), i32(2), 1.0), "CUDA"),
        (gkr.prefix_attention, (bf16(2, 2, 512), torch.zeros(4, 64, 528, dtype=torch.uint8), i32(3), i32(2, 3),
                                1.0), "MXFP4"),
        (gkr.prefix_attention, (bf16(2, 2, 512), torch.zeros(4, 64, 272, dtype=torch.uint8), i32(3, 1), i32(2, 3),
                                1.0), "prefix"),
        (gkr.prefix_attention, (bf16(2, 2, 512), torch.zeros(4, 64, 272, dtype=torch.uint8), i32(3), i32(3, 3),
                                1.0), "row for each"),
        (gkr.prefix_attention, (bf16(2, 129, 512), torch.zeros(4, 64, 272, dtype=torch.uint8), i32(3), i32(2, 3),
                                1.0), "128 heads"),
        (gkr.prefix_attention, (bf16(2, 2, 512), torch.zeros(4, 64, 272, dtype=torch.uint8), i32(3), i32(2, 3),
                                1.0), "CUDA"),
    ]
    for fn, args, what in cases:
        with pytest.raises(ValueError, match=what):
            fn(*args)
    for kw in (dict(out=bf16(4, 2, 256)), dict(lse=torch.zeros(4, 3)), dict(err_flag=i32(1).long())):
        with pytest.raises(ValueError):
            gkr.prompt_attention(bf16(4, 2, 512), bf16(4, 512), i32(2), 1.0, **kw)
    for kw in (dict(slot_mapping=i32(5)), dict(positions=torch.zeros(4, dtype=torch.int64)),
               dict(starts=i32(2)), dict(taken=i32(2))):
        with pytest.raises(ValueError):
            gkr.kv_allocate(*ok, **kw)
    with pytest.raises(ValueError):
        gkr.kv_slots(i32(2, 8), i32(2), 64, 5, indices=i32(2, 6))


@pytest.mark.parametrize("wrapped", [2 ** 32 + 64, 2 ** 31, 0, -64])
def test_binding_refuses_sizes_past_32_bits(gkr, wrapped):
    """What C takes as int32 is checked before it could be cut to its low bits (2^32 + 64: 64)."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)   # noqa: E731
    with pytest.raises(ValueError, match="block_size"):
        gkr.kv_allocate(i32(2), i32(2), i32(2, 8), i32(4), wrapped, 5)
    with pytest.raises(ValueError, match="block_size"):
        gkr.kv_slots(i32(2, 8), i32(2), wrapped, 5)
    with pytest.raises(ValueError, match="block_size"):
        gkr.kv_slots_packed(i32(2, 8), i32(2), wrapped, 5)
    with pytest.raises(ValueError, match="num_heads"):
        gkr.prompt_attention_workspace(wrapped, 4, "cuda:0")
    with pytest.raises(ValueError, match="num_heads"):
        gkr.prefix_attention_workspace(wrapped, 4, 5, 6, "cuda:0")
