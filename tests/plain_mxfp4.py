"""Plain implementations, in 64 bits, of the MXFP4 cache operators: the record's encode and
decode, sparse attention and eviction.  Written from the definitions; no code of the library."""
from __future__ import annotations

import numpy as np

D, DATA, SCALES = 512, 256, 16
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def byte_and_shift(d):
    """Byte of the data row, and shift within it, of dim d's code."""
    w, i = d // 8, d % 8
    nibble = i // 2 + 4 * (i % 2)
    return 4 * w + nibble // 2, 4 * (nibble % 2)


BYTE, SHIFT = (np.array(x) for x in zip(*(byte_and_shift(d) for d in range(D))))


def bf16(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def bf16_bits(x):
    """Round to bf16, nearest even (finite values)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def rotate(row, csc):
    """fp32 row with dims 448..511 turned by a cos/sin row, every step rounded to fp32."""
    x = np.array(row, np.float32)
    c, s = csc[:32], csc[32:]
    e, o = x[448::2].copy(), x[449::2].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        x[448::2] = e * c - o * s
        x[449::2] = o * c + e * s
    return x


def encode(row):
    """fp32 row [512] -> (data bytes [256], scale bytes [16])."""
    data, scale = np.zeros(DATA, np.uint8), np.zeros(SCALES, np.uint8)
    x = np.asarray(row, np.float64)
    for b in range(SCALES):
        v = x[32 * b:32 * b + 32]
        amax = np.abs(v).max()
        if amax == 0:
            e = -127
        elif np.isinf(amax):
            e = 127
        else:
            m, ex = np.frexp(amax)                # amax = m 2^ex, m in [0.5, 1); 6 = 0.75 * 2^3
            e = int(np.clip(ex - 3 + (1 if m > 0.75 else 0), -127, 127))
        scale[b] = e + 127
        for i, y in enumerate(v):
            d = 32 * b + i
            a = min(abs(y) / 2.0 ** e, 6.0)
            dist = np.abs(LEVELS - a)
            best = np.flatnonzero(dist == dist.min())
            code = int(best[best % 2 == 0][0]) if len(best) > 1 else int(best[0])
            code |= 8 if np.signbit(y) else 0
            data[BYTE[d]] |= code << SHIFT[d]
    return data, scale


def offsets(slot, block_size, page_stride):
    page, row = divmod(int(slot), block_size)
    base = page * page_stride
    return base + row * DATA, base + block_size * DATA + row * SCALES


def record_bytes(cache, slots, block_size, page_stride):
    """(data [n, 256], scales [n, 16]) of the records at `slots` in the flat cache."""
    slots = np.asarray(slots, np.int64)
    page, row = slots // block_size, slots % block_size
    base = page * page_stride
    d = cache[(base + row * DATA)[:, None] + np.arange(DATA)]
    s = cache[(base + block_size * DATA + row * SCALES)[:, None] + np.arange(SCALES)]
    return d, s


def decode(data, scales):
    """(bytes [n, 256], [n, 16]) -> fp64 values [n, 512] (scale byte 255: NaN)."""
    code = (data[:, BYTE] >> SHIFT) & 15
    v = LEVELS[code & 7] * np.where(code >= 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, 32, 1)


def attention(q, cache, block_size, page_stride, num_slots, indices, sm_scale):
    """q fp64 [Q, H, 512], indices [Q, K] -> dict of fp64: out, lse, p [Q, H, K] and, for the
    tolerances, mass = sum p |K| and spread = the largest sum_d |q_d K_d| of a valid entry."""
    Q, H, _ = q.shape
    K = indices.shape[1]
    r = {"out": np.zeros((Q, H, D)), "lse": np.full((Q, H), -np.inf), "p": np.zeros((Q, H, K)),
         "mass": np.zeros((Q, H, D)), "spread": np.zeros((Q, H))}
    for i in range(Q):
        ok = np.flatnonzero((indices[i] >= 0) & (indices[i] < num_slots))
        if not len(ok):
            continue
        k = decode(*record_bytes(cache, indices[i][ok], block_size, page_stride))
        s = sm_scale * (q[i] @ k.T)
        m = s.max(1, keepdims=True)
        e = np.exp(s - m)
        r["lse"][i] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
        p = e / e.sum(1, keepdims=True)
        r["out"][i] = p @ k
        r["mass"][i] = p @ np.abs(k)
        r["p"][i][:, ok] = p
        r["spread"][i] = (abs(sm_scale) * (np.abs(q[i]) @ np.abs(k).T)).max(1)
    return r


def tolerances(r, K):
    """How far fp32 sums and bf16 probabilities may take the results of attention() (finfo(t).eps / 2
    a rounding, relative to the value: bf16 2^-8, fp32 2^-24).

    A logit: 512 exact products summed in fp32 in some order, at most 2^-13 of the sum of
    their magnitudes (`spread`), and five roundings (two scalings, the difference to the
    maximum, the exponent's approximation 2^-22) on values up to 2 * spread: below 2^-13 * spread
    more.  So a term exp(s - m) is off by a factor of at most 1 + d, d = expm1(2^-12 * spread)
    + 2^-21.  lse: the sum's terms by d, its at most K + 64 fp32 additions, its own rounding.
    out: numerator and denominator by d each, the probability's rounding 2^-8 in the numerator,
    K / 16 + 16 additions of fp32 (one a matrix instruction, 2^-23: sums may be truncated), the
    output's rounding.  A weight: its terms by 2 d, at most 128 additions."""
    adds = (K + 64) * 2.0 ** -24
    d = np.expm1(2.0 ** -12 * r["spread"]) + 2.0 ** -21
    with np.errstate(invalid="ignore"):
        lse = d + adds + 2.0 ** -22 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0.0)) + 2.0 ** -20
    rel = (2.0 ** -8 + 2 * d + adds + (K / 16 + 16) * 2.0 ** -23)[:, :, None]
    err = rel * r["mass"]
    out = err + 2.0 ** -8 * (np.abs(r["out"]) + err) + 2.0 ** -133
    w = (r["p"] * (2 * (d + lse) + 2.0 ** -17)[:, :, None]).sum(1)
    return out, lse, w


def evict(indices, weights, keep, recent):
    """Lists in, (kept, kept_weights, evicted) out; the weights are only compared."""
    rows, length = indices.shape
    kept = np.full((rows, keep), -1, np.int32)
    kept_w = np.zeros((rows, keep), np.float32)
    gone = np.full((rows, length - keep), -1, np.int64)
    for r in range(rows):
        live = [p for p in range(length) if indices[r, p] >= 0]
        cut = max(0, len(live) - recent)
        old, new = live[:cut], live[cut:]

        def rank(p):
            w = float(weights[r, p])
            return (1, 0.0, p) if np.isnan(w) else (0, -w + 0.0, p)
        best = sorted(old, key=rank)[:keep - len(new)]
        mine = sorted(best + new)
        rest = sorted(set(live) - set(mine))
        kept[r, :len(mine)], kept_w[r, :len(mine)] = indices[r, mine], weights[r, mine]
        gone[r, :len(rest)] = indices[r, rest]
    return kept, kept_w, gone
