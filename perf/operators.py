"""The 4-bit cache operators as they are measured: their cases, inputs and plain forms.

Operators (DeepSeek-V4 style latent attention: one 512-dim row per token is key and value
of every query head):

  write      kv_insert of T latent rows into a cache of 272-byte MXFP4 records (RoPE on dims
             448..511, e2m1 codes, one UE8M0 scale per 32 dims), read back with kv_gather
  gather     kv_gather of listed 272-byte records to bf16 rows
  attention  sparse_attention: decode attention of each query over its listed records,
             output rows and log-sum-exp, with accumulate=True also the attention weight of
             every listed record summed over the heads and added to a running total
  evict      kv_evict: the records of each sequence that its budget keeps, by accumulated
             attention weight with the newest protected, and the slots it frees

A record: 64 little-endian 32-bit words of eight e2m1 codes, then (in the page's scale region)
16 UE8M0 bytes.  Word w holds dims 8w .. 8w+7: the even ones in nibbles 0..3, the odd ones in
nibbles 4..7.  A page holds its block_size data rows of 256 bytes, then its scale rows.

`own` False: the plain forms below, in elementary torch operations; True: the framework's
calls.  Both take prepare()'s state.
"""
import math

import numpy as np
import torch

own = False

D = 512                      # dims of a row
ROPE0, PAIRS = 448, 32       # rotated dims 448..511
DATA, SCALES = 256, 16       # bytes of a record's data and scale rows
BLOCK = 64                   # slots of a page
SM_SCALE = D ** -0.5
EPS_COS = 10000.0            # RoPE base of the cos/sin table


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step writes one token of each of 64 sequences: latency
        {"name": "write decode 64", "op": "write", "tokens": 64, "pages": 2048},
        # a prefill chunk of 16384 tokens
        {"name": "write prefill 16384", "op": "write", "tokens": 16384, "pages": 512},
        # one query's 2048 selected records, odd by one entry
        {"name": "gather 2047", "op": "gather", "entries": 2047, "pages": 1024},
        # 128 queries x 2048 selected records of a 1M-token cache
        {"name": "gather 262144 of 1M", "op": "gather", "entries": 262144, "pages": 16384},
        # a single query with all 128 heads over 2048 selected records: latency
        {"name": "attend 1x128 top 2048", "op": "attention", "queries": 1, "heads": 128,
         "topk": 2048, "pages": 1024, "ragged": False, "accumulate": False},
        # 37 sequences on one of eight ranks (16 heads each), lists of very different lengths,
        # one of them empty
        {"name": "attend 37x16 ragged 1531", "op": "attention", "queries": 37, "heads": 16,
         "topk": 1531, "pages": 4096, "ragged": True, "accumulate": False},
        # the sparse-decode batch: 128 queries x 128 heads x 2048 records of a 1M-token cache
        {"name": "attend 128x128 top 2048", "op": "attention", "queries": 128, "heads": 128,
         "topk": 2048, "pages": 16384, "ragged": False, "accumulate": False},
        # two long sequences attended in full on one of two ranks (64 heads)
        {"name": "attend 2x64 full 100000", "op": "attention", "queries": 2, "heads": 64,
         "topk": 100000, "pages": 4096, "ragged": False, "accumulate": False},
        # a budgeted cache: 8 sequences, 32 heads, budget 2048 plus the new token, weights kept
        {"name": "attend+weights 8x32 of 2049", "op": "attention", "queries": 8, "heads": 32,
         "topk": 2049, "pages": 512, "ragged": False, "accumulate": True},
        # the same for a batch of 64 with all 128 heads, lists of different lengths
        {"name": "attend+weights 64x128 of 2049", "op": "attention", "queries": 64, "heads": 128,
         "topk": 2049, "pages": 4096, "ragged": True, "accumulate": True},
        # each decode step of 128 sequences frees one record of a full budget
        {"name": "evict 128x2049 to 2048", "op": "evict", "rows": 128, "length": 2049,
         "keep": 2048, "recent": 256, "ragged": False},
        # four prompts of up to 131071 tokens cut to a budget of 4096 after prefill
        {"name": "evict 4x131071 to 4096", "op": "evict", "rows": 4, "length": 131071,
         "keep": 4096, "recent": 1024, "ragged": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "gather", "attention", "attention", "attention", "evict"])
    if op == "write":
        t = _log(rng, 1, 16384)
        return {"op": op, "tokens": t, "pages": max(8, -(-t // BLOCK)) + _log(rng, 1, 1024)}
    if op == "gather":
        return {"op": op, "entries": _log(rng, 1, 262144), "pages": _log(rng, 64, 16384)}
    if op == "attention":
        q = _log(rng, 1, 128)
        k = _log(rng, 1, 262144 // q)
        h = rng.choice([8, 16, 32, 64, 128, rng.randint(1, 128)])
        return {"op": op, "queries": q, "heads": h, "topk": k,
                "pages": max(16, -(-k // BLOCK)) + _log(rng, 1, 8192),
                "ragged": rng.random() < 0.5, "accumulate": rng.random() < 0.4}
    rows = _log(rng, 1, 128)
    length = _log(rng, 2, 524288 // rows)
    keep = rng.randint(1, length)
    return {"op": op, "rows": rows, "length": length, "keep": keep,
            "recent": rng.randint(0, keep), "ragged": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op == "write":     # bf16 row, slot, position, cos/sin row in; record out; record and
        t = case["tokens"]                               # index in, bf16 row out
        return {"bytes": t * (1024 + 16 + 256 + 272) + t * (4 + 272 + 1024), "flops": t * D * 4}
    if op == "gather":
        n = case["entries"]
        return {"bytes": n * (4 + 1024) + min(n, case["pages"] * BLOCK) * 272, "flops": n * D}
    if op == "attention":
        q, h, k = case["queries"], case["heads"], case["topk"]
        live = q * k * (0.6 if case["ragged"] else 1.0)  # ragged lists: mean share of entries
        b = q * h * (1024 + 1024 + 4) + q * k * 4 + min(live, case["pages"] * BLOCK) * 272
        if case["accumulate"]:
            b += q * k * 8
        return {"bytes": b, "flops": 4 * live * h * D}
    n, keep = case["rows"] * case["length"], case["rows"] * case["keep"]
    return {"bytes": n * 8 + keep * 8 + (n - keep) * 8, "flops": n}


# ------------------------------------------------------------------------------ the inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _views(flat, pages):
    """The pages' data rows (64 words) and scale rows (4 words) in the flat bytes."""
    words = flat.view(torch.int32)
    step = BLOCK * (DATA + SCALES) // 4
    data = words.as_strided((pages, BLOCK, 64), (step, 64, 1))
    scales = words.as_strided((pages, BLOCK, 4), (step, 4, 1), BLOCK * DATA // 4)
    return data, scales


def _latents(g, n, spread):
    """Latent rows: normal values with a scale of their own for each dim, and outliers."""
    x = torch.randn(n, D, generator=g, device="cuda") * spread
    x *= torch.where(torch.rand(n, D, generator=g, device="cuda") < 0.002, 8.0, 1.0)
    return x.to(torch.bfloat16)


def _filled_cache(g, pages):
    """A cache whose every slot holds the record of a random latent row."""
    flat = torch.zeros(pages * BLOCK * (DATA + SCALES), dtype=torch.uint8, device="cuda")
    data, scales = _views(flat, pages)
    spread = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    step = 1024
    for p in range(0, pages, step):
        n = min(step, pages - p)
        w, s = _encode(_latents(g, n * BLOCK, spread).float())
        data[p:p + n] = w.view(n, BLOCK, 64)
        scales[p:p + n] = s.view(n, BLOCK, SCALES).view(torch.int32)
    return flat, spread


def _lists(g, rows, length, slots, ragged):
    """Index rows of distinct slots; ragged: rows of different lengths padded with -1, a few
    -1 entries inside, and the last of several rows empty."""
    perm = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    start = torch.randint(0, slots, (rows, 1), generator=g, device="cuda")
    at = torch.arange(length, device="cuda")
    idx = perm[(start + at) % slots]
    if ragged:
        share = 0.2 + 0.8 * torch.rand(rows, 1, generator=g, device="cuda")
        if rows > 2:
            share[-1] = 0.0
        hole = torch.rand(rows, length, generator=g, device="cuda") < 0.01
        idx = torch.where((at < torch.ceil(share * length)) & ~hole, idx, -1)
    return idx.contiguous()


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    s["level"] = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                              device="cuda")     # the e2m1 codes' values, for the plain forms
    if op in ("write", "gather", "attention"):
        pages = case["pages"]
        s["flat"], spread = _filled_cache(g, pages)
        # the paged view that the framework takes: [pages, block, record], stride(0) the page
        s["cache"] = s["flat"].as_strided((pages, BLOCK, DATA + SCALES),
                                          (BLOCK * (DATA + SCALES), DATA + SCALES, 1))
    if op == "write":
        t = case["tokens"]
        s["kv"] = _latents(g, t, spread)
        perm = torch.randperm(pages * BLOCK, generator=g, device="cuda")
        s["slots"] = perm[:t].contiguous()
        s["indices"] = s["slots"].to(torch.int32)
        max_pos = 65536
        s["positions"] = torch.randint(0, max_pos, (t,), generator=g, device="cuda")
        inv = EPS_COS ** (-torch.arange(PAIRS, device="cuda", dtype=torch.float64) / PAIRS)
        ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * inv
        s["csc"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["out"] = torch.empty(t, D, dtype=torch.bfloat16, device="cuda")
    elif op == "gather":
        n = case["entries"]
        idx = torch.randint(0, pages * BLOCK, (n,), generator=g, device="cuda", dtype=torch.int32)
        pad = torch.rand(n, generator=g, device="cuda") < 0.02   # -1 pads the lists of short queries
        s["indices"] = torch.where(pad, -1, idx).contiguous()
        s["out"] = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    elif op == "attention":
        q, h, k = case["queries"], case["heads"], case["topk"]
        # queries of logits with a spread of about 2.5, as trained heads have
        s["q"] = (2.0 * torch.randn(q, h, D, generator=g, device="cuda")).to(torch.bfloat16)
        s["indices"] = _lists(g, q, k, pages * BLOCK, case["ragged"])
        if case["accumulate"]:   # what earlier steps have added up
            s["weights"] = 4.0 * torch.rand(q, k, generator=g, device="cuda")
    else:
        rows, length = case["rows"], case["length"]
        s["indices"] = _lists(g, rows, length, 4 * length, case["ragged"])
        w = torch.exp(2.0 * torch.randn(rows, length, generator=g, device="cuda"))
        never = torch.rand(rows, length, generator=g, device="cuda") < 0.1  # ties: never attended
        s["weights"] = torch.where(never, 0.0, w)
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    return {"write": _write, "gather": _gather, "attention": _attention, "evict": _evict}[case["op"]](s)


def _write(s):
    if own:
        import gather_kv_rope_gb300 as gkr
        gkr.kv_insert(s["kv"], s["cache"], s["slots"], s["positions"], s["csc"], BLOCK)
        return gkr.kv_gather(s["cache"], s["indices"], s["out"])
    x = s["kv"].float()
    row = s["csc"][s["positions"]]
    c, n = row[:, :PAIRS], row[:, PAIRS:]
    e, o = x[:, ROPE0::2], x[:, ROPE0 + 1::2]
    turned = torch.stack([e * c - o * n, o * c + e * n], -1).flatten(1)
    w, sc = _encode(torch.cat([x[:, :ROPE0], turned], 1))
    data, scales = _views(s["flat"], case_pages(s))
    page, at = s["slots"] // BLOCK, s["slots"] % BLOCK
    data[page, at] = w
    scales[page, at] = sc.view(torch.int32)
    return _rows(s, s["indices"]).to(torch.bfloat16)


def _gather(s):
    if own:
        import gather_kv_rope_gb300 as gkr
        return gkr.kv_gather(s["cache"], s["indices"], s["out"])
    return _rows(s, s["indices"]).to(torch.bfloat16)


def _attention(s):
    if own:
        import gather_kv_rope_gb300 as gkr
        out, lse = gkr.sparse_attention(s["q"], s["cache"], s["indices"], SM_SCALE,
                                        weights=s.get("weights"))
    else:
        k = _rows(s, s["indices"])                                       # [Q, K, 512]
        live = (s["indices"] >= 0)[:, None, :]
        x = torch.where(live, torch.matmul(s["q"].float(), k.transpose(1, 2)) * SM_SCALE, -math.inf)
        top = x.amax(2, keepdim=True)
        p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        total = p.sum(2, keepdim=True)
        p = p / torch.where(total == 0.0, 1.0, total)
        out = torch.matmul(p, k).to(torch.bfloat16)
        lse = (top + torch.log(total)).squeeze(2)
        if "weights" in s:
            s["weights"] += p.sum(1)
    return {"out": out, "lse": lse, **({"weights": s["weights"]} if "weights" in s else {})}


def _evict(s):
    case = s["case"]
    keep, recent = case["keep"], case["recent"]
    if own:
        import gather_kv_rope_gb300 as gkr
        kept, kept_w, freed = gkr.kv_evict(s["indices"], s["weights"], keep, recent)
        return {"kept": kept, "kept_weights": kept_w, "evicted": freed}
    idx, w = s["indices"], s["weights"]
    length = idx.shape[1]
    at = torch.arange(length, device=idx.device)
    live = idx >= 0
    newer = live.flip(1).cumsum(1).flip(1)               # live entries from here to the end
    new = live & (newer <= recent)
    bits = (w + 0.0).view(torch.int32).to(torch.int64)   # + 0.0: -0 counts as 0
    rank = torch.where(bits < 0, -2147483648 - bits, bits) + (1 << 31)   # in the order of the values
    rank = torch.where(torch.isnan(w), 0, rank)
    rank = torch.where(new, 1 << 33, rank)
    rank = torch.where(live, rank * (1 << 24) + (length - 1 - at), -1)   # ties: the lowest entry
    best = torch.sort(rank, 1, descending=True).indices[:, :keep]
    chosen = torch.zeros_like(live).scatter(1, best, True) & live

    def pack(mask, n):
        order = torch.sort(torch.where(mask, at, length), 1).values[:, :n]
        return order.clamp(max=length - 1), order < length

    i, ok = pack(chosen, keep)
    kept = torch.where(ok, idx.gather(1, i), -1)
    kept_w = torch.where(ok, w.gather(1, i), 0.0)
    i, ok = pack(live & ~chosen, length - keep)
    freed = torch.where(ok, idx.gather(1, i).to(torch.int64), -1)
    return {"kept": kept, "kept_weights": kept_w, "evicted": freed}


# ------------------------------------------------------------------------------ plain parts

def case_pages(s):
    return s["case"]["pages"]


def _encode(x):
    """fp32 rows [n, 512] -> words int32 [n, 64] and UE8M0 bytes uint8 [n, 16].  A block's scale
    is the smallest power of two with amax / scale <= 6, a code the nearest of 0, .5, 1, 1.5, 2,
    3, 4, 6 (halfway: the even code), the sign in its bit 3."""
    n = x.shape[0]
    b = x.reshape(n, SCALES, 32)
    bits = b.abs().amax(2).view(torch.int32)
    e = ((bits >> 23) - 2 + ((bits & 0x7FFFFF) > 0x400000)).clamp(0, 254)   # 6 = 1.5 * 2^2
    inv = ((254 - e).clamp(min=1) << 23).view(torch.float32)                # 2^(127 - e)
    y = (b * inv[:, :, None]).abs()
    code = ((y > 0.25).to(torch.int32) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5)
            + (y >= 3.5) + (y > 5.0))
    code = code + 8 * torch.signbit(b)
    code = code.reshape(n, 64, 4, 2).transpose(2, 3).reshape(n, 64, 8).to(torch.int32)
    shift = 4 * torch.arange(8, device=x.device, dtype=torch.int32)
    return (code << shift).sum(2, dtype=torch.int32), e.to(torch.uint8)


def _rows(s, indices):
    """The listed records' values in fp32 [*, 512]; zeros for index -1."""
    data, scales = _views(s["flat"], case_pages(s))
    live = indices >= 0
    slot = indices.clamp(min=0)
    page, at = slot // BLOCK, slot % BLOCK
    w = data[page, at]
    e = scales[page, at].view(torch.uint8).to(torch.int32)
    shift = 4 * torch.arange(8, device=w.device, dtype=torch.int32)
    code = (w[..., None] >> shift) & 15
    code = code.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3)          # dims in order
    scale = torch.where(e == 0, 0x400000, e << 23).view(torch.float32)
    x = s["level"][code].unflatten(-1, (SCALES, 32)) * scale[..., None]
    return torch.where(live[..., None], x.flatten(-2), 0.0)


# ------------------------------------------------------------------------------ 64 bits

def _exact_rows(flat, pages, slots):
    """Values of the records at `slots` (a flat index tensor, all valid) in fp64."""
    base = slots // BLOCK * (BLOCK * (DATA + SCALES))
    at = slots % BLOCK
    d = torch.arange(D, device=flat.device)
    byte = d // 8 * 4 + (d % 2) * 2 + d % 8 // 4          # odd dims in a word's upper half
    raw = flat[(base + at * DATA)[:, None] + byte].to(torch.int64)
    nib = (raw >> (d // 2 % 2 * 4)) & 15                   # two nibbles of a byte: dims d, d + 2
    ex, man = (nib >> 1) & 3, nib & 1
    mag = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2((ex - 1).double()))
    e = flat[(base + BLOCK * DATA + at * SCALES)[:, None] + d // 32].double() - 127.0
    return torch.where(nib >= 8, -mag.double(), mag.double()) * torch.exp2(e)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "write":
        t = case["tokens"]
        x = s["kv"].double()
        row = s["csc"].double()[s["positions"]]
        c, n = row[:, :PAIRS], row[:, PAIRS:]
        e, o = x[:, ROPE0::2].clone(), x[:, ROPE0 + 1::2].clone()
        single = lambda v: v.float().double()  # noqa: E731  the rotation is defined in fp32 steps
        x[:, ROPE0::2] = single(single(e * c) - single(o * n))
        x[:, ROPE0 + 1::2] = single(single(o * c) + single(e * n))
        b = x.view(t, SCALES, 32)
        m, ex = torch.frexp(b.abs().amax(2))               # 6 = 0.75 * 2^3
        ex = torch.clamp(ex - 3 + (m > 0.75).int(), -127, 127).double()
        y = b / torch.exp2(ex)[:, :, None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1.0)   # 1/2, 1, 2
        return (torch.round(y / step) * step * torch.exp2(ex)[:, :, None]).view(t, D)
    if op == "gather":
        idx = s["indices"].long()
        x = _exact_rows(s["flat"], case["pages"], idx.clamp(min=0))
        return torch.where((idx >= 0)[:, None], x, 0.0)
    if op == "attention":
        outs, lses, sums = [], [], []
        for i in range(case["queries"]):
            idx = s["indices"][i].long()
            live = idx >= 0
            k = _exact_rows(s["flat"], case["pages"], idx[live])
            x = s["q"][i].double() @ k.T * SM_SCALE
            lse = torch.logsumexp(x, 1) if k.shape[0] else torch.full((case["heads"],), -math.inf,
                                                                      dtype=torch.float64, device="cuda")
            p = torch.exp(x - lse[:, None])
            outs.append(p @ k)
            lses.append(lse)
            if case["accumulate"]:
                total = s["weights"][i].double()
                total[live] += p.sum(0)
                sums.append(total)
        r = {"out": torch.stack(outs), "lse": torch.stack(lses)}
        return {**r, "weights": torch.stack(sums)} if case["accumulate"] else r
    idx, w = s["indices"].cpu().numpy(), s["weights"].cpu().numpy().astype(np.float64)
    rows, length = idx.shape
    keep, recent = case["keep"], case["recent"]
    kept = np.full((rows, keep), -1, np.int32)
    kept_w = np.zeros((rows, keep))
    freed = np.full((rows, length - keep), -1, np.int64)
    for r in range(rows):
        live = np.flatnonzero(idx[r] >= 0)
        new = live[len(live) - min(recent, len(live)):]
        old = live[:len(live) - len(new)]
        room = min(keep - len(new), len(old))
        best = old[np.lexsort((old, -w[r, old]))[:room]]
        mine = np.sort(np.concatenate([best, new]))
        gone = np.setdiff1d(live, mine)
        kept[r, :len(mine)], kept_w[r, :len(mine)] = idx[r, mine], w[r, mine]
        freed[r, :len(gone)] = idx[r, gone]
    return {"kept": kept, "kept_weights": kept_w, "evicted": freed}
