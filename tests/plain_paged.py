"""Plain implementations, in 64 bits, of a batch's way through a paged cache: page allocation,
slot lists, attention of packed prompts and attention behind a shared prefix.  Written from the
definitions; no code of the library."""
from __future__ import annotations

import numpy as np

ERR_SLOT, ERR_POS, ERR_INDEX = 1, 2, 4
TOP = 2 ** 31 - 1


def allocate(past, added, table, free, block_size, num_tokens):
    """(slots, positions, starts, taken, table, error bits)."""
    table = np.array(table, np.int64)
    B, W = table.shape
    slots, pos = np.full(num_tokens, -1, np.int64), np.zeros(num_tokens, np.int64)
    starts, taken, bits, row = [0], 0, 0, 0
    for b in range(B):
        p, a = max(int(past[b]), 0), max(int(added[b]), 0)
        bits |= ERR_POS if past[b] < 0 or added[b] < 0 else 0
        for col in range(min(-(-p // block_size), W), min(-(-(p + a) // block_size), W)):
            if taken < len(free):
                table[b, col] = free[taken]
            else:
                bits |= ERR_SLOT
            taken += 1
        held, end = min(-(-p // block_size), W), min(-(-(p + a) // block_size), W)
        first_free = taken - (end - held)                 # in the list, of this request
        for i in range(a):
            if row + i >= num_tokens:
                bits |= ERR_SLOT
                break
            page, at = divmod(p + i, block_size)
            there = page < W and (page < held or first_free + page - held < len(free))
            if there and table[b, page] >= 0:
                slots[row + i] = table[b, page] * block_size + at
            else:
                bits |= ERR_SLOT
            pos[row + i] = p + i
        row += a
        starts.append(min(row, TOP))
    return slots, pos, np.array(starts, np.int64), min(taken, len(free)), table, bits


def slots(table, lengths, block_size, first=None):
    """One list of slots (int64) per request, and error bits."""
    out, bits = [], 0
    for b, n in enumerate(lengths):
        f = 0 if first is None else int(first[b])
        if n < 0 or f < 0:
            bits |= ERR_INDEX
        row = []
        for p in range(max(f, 0), int(n)):
            page, at = divmod(p, block_size)
            s = int(table[b][page]) * block_size + at if page < len(table[b]) and table[b][page] >= 0 else -1
            if s < 0 or s > TOP:
                s, bits = -1, bits | ERR_INDEX
            row.append(s)
        out.append(row)
    return out, bits


def attend(q, k, see, sm_scale):
    """q fp64 [n, H, 512] over k fp64 [m, 512], query i over the first see[i] rows ->
    out, lse and, for the tolerances, mass = sum p |k|, spread = the largest sum_d |q_d k_d|."""
    n, H, D = q.shape
    r = {"out": np.zeros((n, H, D)), "lse": np.full((n, H), -np.inf), "mass": np.zeros((n, H, D)),
         "spread": np.zeros((n, H))}
    for i in range(n):
        m = min(max(int(see[i]), 0), len(k))
        if m == 0:
            continue
        s = sm_scale * (q[i] @ k[:m].T)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        total = e.sum(1, keepdims=True)
        r["lse"][i] = (top + np.log(total))[:, 0]
        r["out"][i] = e @ k[:m] / total
        r["mass"][i] = e @ np.abs(k[:m]) / total
        r["spread"][i] = (abs(sm_scale) * (np.abs(q[i]) @ np.abs(k[:m]).T)).max(1)
    return r


def prompt(q, kv, starts, kv_starts, sm_scale, causal=True):
    """Packed requests; queries of no request keep out NaN and lse NaN."""
    T, H, D = q.shape
    r = {"out": np.full((T, H, D), np.nan), "lse": np.full((T, H), np.nan),
         "mass": np.zeros((T, H, D)), "spread": np.zeros((T, H))}
    for b in range(len(starts) - 1):
        a, z = int(starts[b]), int(starts[b + 1])
        k = kv[int(kv_starts[b]):int(kv_starts[b + 1])]
        n, m = z - a, len(k)
        see = m - n + 1 + np.arange(n) if causal else np.full(n, m)
        one = attend(q[a:z], k, see, sm_scale)
        for name in r:
            r[name][a:z] = one[name]
    return r


def tolerances(r, keys):
    """(out, lse): how far results with fp32 sums and bf16 probabilities may be off.

    A logit: 512 exact products summed in fp32 in some order, at most 2^-13 of the sum of
    their magnitudes (`spread`), and five roundings (two scalings, the difference to the
    maximum, the exponent's approximation 2^-22) on values up to 2 * spread: below 2^-13 * spread
    more.  A term exp(s - m) is then off by a factor of at most 1 + d, d = expm1(2^-12 spread) +
    2^-21.  lse: the terms by d, at most keys + 64 fp32 additions, its own roundings.  out:
    numerator and denominator by d each, the probability's rounding 2^-8 (twice the half step,
    which leaves room for the pieces' weights, 2^-21 each), keys / 16 + 16 additions of fp32
    in the matrix unit (2^-23: sums may be truncated), the output's rounding 2^-8 (half a step of
    bf16 is 2^-9 of the power of two below, 2^-8 of the value at most)."""
    adds = (keys + 64) * 2.0 ** -24
    d = np.expm1(2.0 ** -12 * r["spread"]) + 2.0 ** -21
    lse = d + adds + 2.0 ** -22 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0.0)) + 2.0 ** -20
    rel = (2.0 ** -8 + 2 * d + adds + (keys / 16 + 16) * 2.0 ** -23)[:, :, None]
    err = rel * r["mass"]
    return err + 2.0 ** -8 * (np.abs(r["out"]) + err) + 2.0 ** -133, lse
