"""CPU checks of the MXFP4 operators: hand-derived pins of the plain record encoder that the GPU
tests compare with, and the C ABI's and the binding's refusals (no GPU needed: every call fails
in the host checks)."""
import ctypes

import numpy as np
import pytest
import torch

import plain_mxfp4 as plain

A = 0x7F0000000000       # plausible aligned device addresses, never dereferenced
B = A + (1 << 30)


def desc(gkr, record=272, bs=64, pages=8, ps=None):
    return gkr.CacheDesc(record, bs, pages, (bs * record + 511) // 512 * 512 if ps is None else ps)


def attend(gkr, d, q=A, H=8, cache=B, idx=A, istride=64, Q=2, topk=64, scale=1.0, out=A, lse=A,
           weights=None, wstride=0, ws=A, ws_bytes=1 << 30, err=None, opts=None):
    return gkr.lib().gkr_sparse_attention(q, H, cache, None if d is None else ctypes.byref(d), idx,
                                          istride, Q, topk, scale, out, lse, weights, wstride, ws,
                                          ws_bytes, err,
                                          None if opts is None else ctypes.byref(opts), None)


def evict(gkr, idx=A, istride=16, w=A, wstride=16, rows=2, length=16, keep=8, recent=2, kept=A,
          kept_w=A, gone=A, opts=None):
    return gkr.lib().gkr_kv_evict(idx, istride, w, wstride, rows, length, keep, recent, kept,
                                  kept_w, gone, None if opts is None else ctypes.byref(opts), None)


def test_plain_encoder_pins():
    x = np.zeros(512, np.float32)
    x[:8] = [6.0, 0.25, 0.75, -5.0, 2.5, 3.5, -0.0, 1.25]   # every tie of the e2m1 levels
    x[32] = 7.0                                             # above 6: the next power of two
    x[64] = 6.0 * 2.0 ** -100
    data, scale = plain.encode(x)
    # codes: 6.0 = 7; ties 0.25 -> 0, 0.75 -> 1.0 (2), -5 -> -4 (e), 2.5 -> 2 (4), 3.5 -> 4 (6),
    # -0 (8), 1.25 -> 1 (2); dims 0, 2, 4, 6 in nibbles 0..3, dims 1, 3, 5, 7 in nibbles 4..7
    assert data[:4].tolist() == [0x27, 0x84, 0xE0, 0x26]
    assert scale[:3].tolist() == [127, 128, 27] and (scale[3:] == 0).all()
    assert data[16] & 15 == 6                               # 7 / 2 = 3.5: a tie, to 4
    v = plain.decode(data[None], scale[None])[0]
    assert v[:8].tolist() == [6, 0, 1, -4, 2, 4, 0, 1] and np.signbit(v[6])
    assert v[32] == 8.0 and v[64] == 6.0 * 2.0 ** -100


def test_plain_encoder_is_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal(512).astype(np.float32)
    data, scale = plain.encode(x)
    v = plain.decode(data[None], scale[None])[0]
    step = 2.0 ** (scale.astype(int).repeat(32) - 127)
    assert (np.abs(v - x) <= step).all()                    # widest spacing 2: half of it
    assert (np.abs(x).reshape(16, 32).max(1) <= 6 * 2.0 ** (scale.astype(int) - 127)).all()
    assert (np.abs(x).reshape(16, 32).max(1) > 3 * 2.0 ** (scale.astype(int) - 127)).all()


def test_plain_evict_pin():
    idx = np.array([[5, -1, 3, 9, 7, 1]], np.int32)
    w = np.array([[2.0, 99.0, 1.0, 2.0, 0.5, np.nan]], np.float32)
    kept, kw, gone = plain.evict(idx, w, 3, 1)
    assert kept.tolist() == [[5, 9, 1]] and gone.tolist() == [[3, 7, -1]]
    assert kw[0, :2].tolist() == [2.0, 2.0] and np.isnan(kw[0, 2])


def test_geometry(gkr):
    assert gkr.page_stride(272, 64) == 64 * 272
    assert gkr.page_stride(272, 32) == 8704                 # 8704 = 17 * 512
    assert gkr.page_stride(272, 96) == 96 * 272
    assert gkr.page_stride(272, 48) == -1                   # packed: a multiple of 32
    assert gkr.record_rows(272) == (256, 16, 512)
    c = gkr.alloc_cache(3, 64, 272, "cpu", page_stride_bytes=64 * 272 + 512)
    assert tuple(c.shape) == (3, 64, 272) and c.stride(0) == 64 * 272 + 512


def test_record_272_is_refused_where_it_is_not_read(gkr):
    d = desc(gkr)
    lib = gkr.lib()
    assert lib.gkr_sparse_logits(A, 8, B, ctypes.byref(d), A, 2, 64, 1.0, None, A, None, None,
                                 None) == 2
    assert lib.gkr_rope_quant_insert(A, 8, B, ctypes.byref(d), A, A, A, 16, 4, 0, None, None,
                                     None) == 2


@pytest.mark.parametrize("record", [528, 584, 512, 1024, 500])
def test_attention_reads_mxfp4_only(gkr, record):
    ps = {528: 33792, 584: 37440}.get(record, 64 * record)
    assert attend(gkr, desc(gkr, record, ps=ps)) == 2


def test_attention_refusals(gkr):
    d = desc(gkr)
    assert attend(gkr, None) == 1
    assert attend(gkr, desc(gkr, bs=48)) == 1
    assert attend(gkr, desc(gkr, ps=64 * 272 - 512)) == 3
    assert attend(gkr, desc(gkr, ps=64 * 272 + 256)) == 3
    assert attend(gkr, d, Q=0, q=None, cache=None, idx=None, out=None, lse=None) == 0
    for bad in (dict(H=0), dict(H=129), dict(Q=-1), dict(Q=(1 << 24) + 1), dict(topk=-1),
                dict(topk=(1 << 24) + 1, istride=1 << 25), dict(istride=63),
                dict(Q=1 << 24, topk=1 << 20, istride=1 << 20),
                dict(weights=A, wstride=63), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(q=None), dict(cache=None), dict(idx=None), dict(out=None), dict(lse=None),
                dict(opts=gkr.LaunchOpts())):
        if "opts" in bad:
            bad["opts"].pdl = 2
        assert attend(gkr, d, **bad) == 1, bad
    for bad in (dict(q=A + 8), dict(cache=B + 4), dict(out=A + 8), dict(idx=A + 2), dict(lse=A + 2),
                dict(weights=A + 2, wstride=64), dict(err=A + 2)):
        assert attend(gkr, d, **bad) == 4, bad


def test_workspace_refusals(gkr):
    f = gkr.lib().gkr_sparse_attention_workspace
    n = ctypes.c_int64(-7)
    assert f(8, 2, 64, None) == 1
    for bad in ((0, 2, 64), (129, 2, 64), (8, -1, 64), (8, 2, -1), (8, (1 << 24) + 1, 64)):
        assert f(*bad, ctypes.byref(n)) == 1, bad
    assert f(8, 0, 64, ctypes.byref(n)) == 0 and n.value == 0


def test_evict_refusals(gkr):
    assert evict(gkr, rows=0, idx=None, w=None, kept=None, kept_w=None, gone=None) == 0
    assert evict(gkr, length=0, keep=0, recent=0, idx=None, w=None, kept=None, kept_w=None,
                 gone=None) == 0
    for bad in (dict(rows=-1), dict(length=-1), dict(keep=17), dict(keep=-1, recent=-1),
                dict(recent=9), dict(recent=-1), dict(istride=15), dict(wstride=15),
                dict(length=(1 << 24) + 1, istride=1 << 25, wstride=1 << 25), dict(idx=None),
                dict(w=None), dict(kept=None), dict(kept_w=None), dict(gone=None),
                dict(opts=gkr.LaunchOpts())):
        if "opts" in bad:
            bad["opts"].early_metadata = 5
        assert evict(gkr, **bad) == 1, bad
    for bad in (dict(idx=A + 2), dict(w=A + 1), dict(kept=A + 2), dict(kept_w=A + 2),
                dict(gone=A + 4)):
        assert evict(gkr, **bad) == 4, bad


def test_binding_refusals(gkr):
    q = torch.zeros(2, 4, 512, dtype=torch.bfloat16)
    idx = torch.zeros(2, 8, dtype=torch.int32)
    cache = gkr.alloc_cache(2, 64, 272, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        gkr.sparse_attention(q, cache, idx, 1.0)
    with pytest.raises(ValueError, match="272"):
        gkr.sparse_attention(q, gkr.alloc_cache(2, 64, 528, "cpu"), idx, 1.0)
    for bad in (dict(q=q.float()), dict(q=q[:, ::2]), dict(q=q[:1]), dict(idx=idx.long()),
                dict(idx=idx.t()), dict(q=torch.zeros(2, 129, 512, dtype=torch.bfloat16)),
                dict(q=torch.zeros(2, 0, 512, dtype=torch.bfloat16)),
                dict(out=q.float()), dict(lse=torch.zeros(2, 3)),
                dict(weights=torch.zeros(2, 7)), dict(weights=torch.zeros(2, 8, dtype=torch.float64)),
                dict(err_flag=torch.zeros(1))):
        kw = {"q": q, "k_cache": cache, "indices": idx, "sm_scale": 1.0}
        kw.update({"indices" if k == "idx" else k: v for k, v in bad.items()})
        with pytest.raises(ValueError):
            gkr.sparse_attention(**kw)
    w = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gkr.kv_evict(idx, w, 4)
    for bad in (dict(keep=9), dict(keep=-1), dict(keep=4, recent=5), dict(keep=4, recent=-1),
                dict(keep=4, weights=w.double()), dict(keep=4, weights=w[:, :7]),
                dict(keep=4, indices=idx.long()),
                dict(keep=4, kept=torch.zeros(2, 5, dtype=torch.int32)),
                dict(keep=4, evicted=torch.zeros(2, 4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            gkr.kv_evict(**{"indices": idx, "weights": w, **bad})


def test_evict_list_limit(gkr):
    """2^21 entries of a list at most: the words of a longer one would outgrow shared memory."""
    n = (1 << 21) + 1
    assert evict(gkr, length=n, istride=n, wstride=n) == 1
    assert evict(gkr, length=n, istride=n, wstride=n, keep=n, recent=0) == 1
    # at the limit the lengths pass, and the pointers are looked at next
    assert evict(gkr, length=n - 1, istride=n - 1, wstride=n - 1, idx=A + 2) == 4
