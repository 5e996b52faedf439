"""Serving a batch from a paged packed cache: the operators, what a pass of each costs at least, and
their plain forms.

  rope     queries or keys rotated by position, the frequency blocks shared out over one or several axes
  append   new keys and values of a ragged batch rotated, quantized and packed into the pages of a pool
  decode   one query token per sequence attends over its own pages
  prefix   the same, where the whole batch also attends over one shared prefix

A pool is a header and n_pages pages; a page holds, per KV head, page_tokens / 32 tile records: the K
bit streams of 32 tokens (word-planar, widths per frequency block), 32 fp16 K norms, 32 fp16 V norms,
the V bit streams per dim.
"""
import math
import random
from functools import lru_cache

import numpy as np
import torch

own = False

D, H2, TILE = 128, 64, 32
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's queries, rotated before attention: the smallest call
        {"name": "rope step", "op": "rope", "tokens": 32, "heads": 16, "dtype": "bf16", "axes": 1, "positions": 131072,
         "mix": 1},
        # the queries of a prompt of images and text, three position axes
        {"name": "rope 3 axes prompt", "op": "rope", "tokens": 16384, "heads": 32, "dtype": "bf16", "axes": 3,
         "positions": 32768, "mix": 2},
        # one new token for each of 64 sequences of a running batch
        {"name": "append step", "op": "append", "new_lo": 1, "new_hi": 1, "batch": 64, "len_lo": 100, "len_hi": 8000,
         "hkv": 8, "bits_k": 4, "bits_v": 4, "page": 64, "dtype": "bf16", "axes": 1, "mix": 3},
        # chunks of six prompts with images, starting inside tiles
        {"name": "append chunks", "op": "append", "new_lo": 200, "new_hi": 1500, "batch": 6, "len_lo": 1, "len_hi": 5000,
         "hkv": 8, "bits_k": 2, "bits_v": 2, "page": 128, "dtype": "f16", "axes": 3, "mix": 4},
        # a whole long prompt
        {"name": "append long prompt", "op": "append", "new_lo": 131072, "new_hi": 131072, "batch": 1, "len_lo": 0,
         "len_hi": 0, "hkv": 2, "bits_k": 3, "bits_v": 3, "page": 256, "dtype": "bf16", "axes": 1, "mix": 5},
        # a few short conversations
        {"name": "decode short", "op": "decode", "batch": 4, "len_lo": 60, "len_hi": 700, "hq": 16, "hkv": 2, "bits_k": 3,
         "bits_v": 3, "page": 32, "prefix": 0, "dtype": "bf16", "out": "f32", "mix": 6},
        # a running batch of very different lengths
        {"name": "decode ragged batch", "op": "decode", "batch": 32, "len_lo": 64, "len_hi": 16384, "hq": 32, "hkv": 8,
         "bits_k": 4, "bits_v": 4, "page": 64, "prefix": 0, "dtype": "bf16", "out": "bf16", "mix": 7},
        # one long context
        {"name": "decode long", "op": "decode", "batch": 1, "len_lo": 131072, "len_hi": 131072, "hq": 16, "hkv": 2,
         "bits_k": 3, "bits_v": 3, "page": 256, "prefix": 0, "dtype": "bf16", "out": "f32", "mix": 8},
        # four samples of one prompt
        {"name": "prefix small", "op": "prefix", "batch": 4, "len_lo": 1, "len_hi": 100, "hq": 16, "hkv": 2, "bits_k": 3,
         "bits_v": 3, "page": 32, "prefix": 2000, "dtype": "bf16", "out": "f32", "mix": 9},
        # 16 questions about one document
        {"name": "prefix 16 users", "op": "prefix", "batch": 16, "len_lo": 16, "len_hi": 900, "hq": 32, "hkv": 8,
         "bits_k": 2, "bits_v": 2, "page": 64, "prefix": 32749, "dtype": "f16", "out": "f16", "mix": 10},
        # 64 users behind one long system prompt
        {"name": "prefix 64 users", "op": "prefix", "batch": 64, "len_lo": 100, "len_hi": 2000, "hq": 16, "hkv": 2,
         "bits_k": 3, "bits_v": 3, "page": 128, "prefix": 65536, "dtype": "bf16", "out": "bf16", "mix": 11},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "prefix"])
    mix = rng.randrange(1 << 20)
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": rng.choice([1, 2, 5, 8, 16, 32]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "axes": rng.choice([1, 2, 3, 4]),
                "positions": rng.choice([4096, 32768, 131072]), "mix": mix}
    hkv = rng.choice([1, 2, 4, 8])
    base = {"hkv": hkv, "bits_k": rng.choice([1, 2, 3, 4, 5, 8]), "bits_v": rng.choice([1, 2, 3, 4, 5, 6, 7, 8]),
            "page": rng.choice([32, 64, 128, 256]), "mix": mix}
    if op == "append":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 262144 // (batch * hkv))
        dtype = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "batch": batch, "new_lo": rng.choice([0, 1, hi]), "new_hi": hi, "len_lo": 0,
                "len_hi": _log_int(rng, 1, 4000), "dtype": dtype, "axes": rng.choice([0, 1, 3]), **base}
    batch = _log_int(rng, 1, 48)
    hi = _log_int(rng, 1, min(131072, 2097152 // (batch * hkv)))
    return {"op": op, "batch": batch, "len_lo": rng.choice([0, 1, hi]), "len_hi": hi, "hq": hkv * rng.choice([1, 2, 3, 4, 7, 8]),
            "prefix": 0 if op == "decode" else _log_int(rng, 1, min(65536, 131072 // hkv)), "dtype": rng.choice(["bf16", "f16"]),
            "out": rng.choice(["f32", "bf16", "f16"]), **base}


def _spread(case, lo, hi, salt):
    """The batch's counts between lo and hi, spread over their logarithm; the first is hi."""
    rng = random.Random(case["mix"] * 7 + salt)
    got = [hi] + [lo if lo >= hi else _log_int(rng, max(lo, 1), hi) for _ in range(case["batch"] - 1)]
    if lo == 0 and case["batch"] > 1:
        got[-1] = 0                                          # a row of the batch that holds no sequence
    return got


def _lens(case):
    return _spread(case, case["len_lo"], case["len_hi"], 1)


def _new(case):
    return _spread(case, case["new_lo"], case["new_hi"], 2)


def work(case):
    e = DTYPES[case["dtype"]].itemsize
    if case["op"] == "rope":
        n = case["tokens"]
        return {"bytes": 2 * n * case["heads"] * D * e + n * (8 * H2 + 4 * case["axes"]), "flops": 6 * n * case["heads"] * H2}
    stored = 16 * (case["bits_k"] + case["bits_v"]) + 4       # bytes of a token and KV head
    if case["op"] == "append":
        n = sum(_new(case))
        table = n * (8 * H2 + 4 * case["axes"]) if case["axes"] else 0
        return {"bytes": n * case["hkv"] * (2 * D * e + stored) + table, "flops": n * case["hkv"] * 14 * D}
    own_tokens = sum(_lens(case))
    b, hq = case["batch"], case["hq"]
    return {"bytes": (case["prefix"] + own_tokens) * case["hkv"] * stored + b * hq * D * (e + DTYPES[case["out"]].itemsize),
            "flops": 4 * D * hq * (b * case["prefix"] + own_tokens)}


# ------------------------------------------------------------------------------ tables and allocation

def _mass(a, b):
    sf = lambda x: 0.5 * torch.special.erfc(x / math.sqrt(2.0))  # noqa: E731
    return torch.where(a >= 0, sf(a) - sf(b), sf(-b) - sf(-a))


@lru_cache(maxsize=None)
def _codebook(w):
    """Centroids (fp16) and thresholds (fp32) of the 2^w-level quantizer of N(0, 1) with the least
    square error, and that error: centroids at their cells' means, thresholds midway."""
    n = 1 << w
    i = torch.arange(n, dtype=torch.float64)
    c = math.sqrt(3.0) * torch.special.ndtri((i + 0.5) / n)
    inf = torch.tensor([math.inf], dtype=torch.float64)
    phi = lambda x: torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)  # noqa: E731
    for step in range(260):
        t = 0.5 * (c[:-1] + c[1:])
        a, b = torch.cat([-inf, t]), torch.cat([t, inf])
        p = _mass(a, b)
        m = (phi(a) - phi(b)) / p
        if step < 240:
            c = m
            continue
        da = torch.where(a.isfinite(), phi(a) * (m - a) / p, 0.0)   # Newton on c = m(c)
        db = torch.where(b.isfinite(), phi(b) * (b - m) / p, 0.0)
        da, db = da.nan_to_num(), db.nan_to_num()
        jac = torch.eye(n, dtype=torch.float64) - 0.5 * torch.diag(da + db)
        jac = jac - 0.5 * torch.diag(da[1:], -1) - 0.5 * torch.diag(db[:-1], 1)
        c = c - torch.linalg.solve(jac, c - m)
    c = 0.5 * (c - c.flip(0))
    c16 = c.to(torch.float16)
    t32 = (0.5 * (c16[:-1].double() + c16[1:].double())).float()
    t, c = t32.double(), c16.double()
    a, b = torch.cat([-inf, t]), torch.cat([t, inf])
    edge = lambda x: torch.where(x.isfinite(), x * phi(x), 0.0).nan_to_num()  # noqa: E731
    m0 = _mass(a, b)
    err = (m0 + edge(a) - edge(b) - 2 * c * (phi(a) - phi(b)) + c * c * m0).sum()
    return c16, t32, float(err.float())


def _widths(E, bits):
    """bits * 64 single bits, each to the block that gains most by it, ties to the lowest block."""
    delta = np.array([1.0] + [_codebook(w)[2] for w in range(1, 9)])
    gain = E[:, None] * (delta[:-1] - delta[1:])[None, :]
    b, k = np.divmod(np.arange(gain.size), 8)
    first = np.lexsort((k, b, -gain.reshape(-1)))[:bits * H2]
    return np.bincount(b[first], minlength=H2)


def _mix64(z):
    m = (1 << 64) - 1
    z = (z + 0x9E3779B97F4A7C15) & m
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
    return z ^ (z >> 31)


RECORD = np.dtype([("energy", "<f8", 64), ("gain", "<f4", 64), ("dequant", "<f4", 64), ("bit_off", "<i2", 64),
                   ("width", "u1", 64), ("stream_block", "u1", 64), ("class_bit", "<u2", 8), ("class_width", "u1", 8),
                   ("class_first", "u1", 8), ("class_blocks", "u1", 8), ("pad0", "u1", 56), ("head_dim", "<i4"),
                   ("bits_k", "<i4"), ("w_max", "<i4"), ("mode", "<i4"), ("n_classes", "<i4"), ("k_words", "<i4"),
                   ("n_blocks", "<i4"), ("pad1", "<i4"), ("plan_slot", "<u4", 24), ("plan_col_block", "i1", 96),
                   ("plan_n_slots", "<i4"), ("plan_k_cols", "<i4"), ("digest", "<u8"), ("pad2", "u1", 432)])


def _allocation(E, bits):
    """Allocation record of one KV head with block energies E: widths, gains, the order of the K
    stream (widths descending, blocks ascending) and the plan of slots of four block pairs."""
    r = np.zeros((), RECORD)
    w = _widths(E, bits)
    total = 0.0
    for e in E.tolist():
        total += e
    g = np.sqrt(2.0 * total / (D * E)).astype(np.float32)
    order = np.lexsort((np.arange(H2), -w))
    order = order[w[order] > 0]
    off = np.full(H2, -1)
    off[order] = np.concatenate([[0], np.cumsum(2 * w[order])[:-1]])
    r["energy"], r["gain"], r["dequant"] = E, g, (1.0 / (math.sqrt(D) * g.astype(np.float64))).astype(np.float32)
    r["bit_off"], r["width"] = off, w
    r["stream_block"][:], r["plan_col_block"][:] = 255, -1
    r["stream_block"][:len(order)] = order
    r["head_dim"], r["bits_k"], r["w_max"], r["mode"] = D, bits, 8, 0
    slot = 0
    widths = sorted(set(w[order].tolist()), reverse=True)
    for c, cw in enumerate(widths):
        mine = [i for i, b in enumerate(order) if w[b] == cw]
        r["class_width"][c], r["class_first"][c], r["class_blocks"][c] = cw, mine[0], len(mine)
        r["class_bit"][c] = off[order[mine[0]]]
        for i in range(0, len(mine), 4):
            cols = order[mine[i:i + 4]]
            r["plan_slot"][slot] = cw | int(off[cols[0]]) << 8
            r["plan_col_block"][4 * slot:4 * slot + len(cols)] = cols
            slot += 1
    r["n_classes"], r["k_words"], r["n_blocks"] = len(widths), bits * D, len(order)
    r["plan_n_slots"], r["plan_k_cols"] = slot, -(-4 * slot // 8) * 8
    bitsg = g.view(np.uint32)
    r["digest"] = sum(_mix64(b << 40 | int(w[b]) << 32 | int(bitsg[b])) for b in range(H2)) & ((1 << 64) - 1)
    return r


def _record_bytes(case):
    return 4 * D * (case["bits_k"] + case["bits_v"]) + 4 * TILE


def _header(case, n_pages, records):
    """The pool's header: layout, shapes, widths, one allocation digest per KV head."""
    h = np.zeros(-(-(64 + 8 * case["hkv"]) // 128) * 128, np.uint8)
    u = h.view("<u4")
    u[0], u[1], u[2] = 0x5051564B, 1 | D << 16, case["bits_k"] | case["bits_v"] << 8 | 8 << 16
    u[4], u[5], u[6], u[7] = n_pages, case["hkv"], case["page"], _record_bytes(case)
    h[64:64 + 8 * case["hkv"]] = np.array([r["digest"] for r in records], "<u8").view(np.uint8)
    return torch.from_numpy(h)


# ------------------------------------------------------------------------------ plain forms

def _rotate(x, table, positions, axis):
    """x [tokens][heads][128] rotated: block b by the angle of axis[b]'s position, rounded once."""
    cs = table[positions[axis.long()].long(), torch.arange(H2, device=x.device)[:, None]]   # [64][tokens][2]
    c, s = (cs[..., i].t()[:, None, :] for i in (0, 1))
    x1, x2 = x[..., :H2].float(), x[..., H2:].float()
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1).to(x.dtype)


def _row_codes(x, gain, widths):
    """fp16 norm and codes of rows x [..., 128]: the sum of squares as eight partial sums over the
    dims of one residue, codes as the number of thresholds below sqrt(128) x / norm * gain."""
    x = x.float()
    sq = (x * x).unflatten(-1, (16, 8))
    s = sq[..., 0, :]
    for j in range(1, 16):                                    # this order of the sum is the definition
        s = s + sq[..., j, :]
    s = s[..., 0::2] + s[..., 1::2]
    s = s[..., 0::2] + s[..., 1::2]
    norm = torch.sqrt(s[..., 0] + s[..., 1]).half()
    n32 = norm.float()
    a = torch.where(n32 == 0, 0.0, torch.full_like(n32, math.sqrt(D)) / n32)
    y = (x * a[..., None]) * gain
    codes = torch.zeros(y.shape, dtype=torch.int32, device=y.device)
    for w in sorted(set(widths.tolist()) - {0}):
        dims = torch.from_numpy(np.flatnonzero(widths == w)).to(y.device)
        codes[..., dims] = torch.bucketize(y[..., dims].contiguous(), _codebook(w)[1].to(y.device), out_int32=True)
    return norm, codes


def _bits(codes, offsets, widths, words):
    """Codes [..., n] as little-endian bit streams of `words` 32-bit words, code i at offsets[i]."""
    live = np.flatnonzero(widths)
    off = torch.from_numpy(offsets[live].astype(np.int64)).to(codes.device)
    v = codes[..., torch.from_numpy(live).to(codes.device)].long() << (off & 31)
    out = torch.zeros(codes.shape[:-1] + (words + 1,), dtype=torch.int64, device=codes.device)
    out.index_add_(-1, off >> 5, v & 0xffffffff)
    out.index_add_(-1, (off >> 5) + 1, v >> 32)
    return out[..., :words].to(torch.int32)                   # the low 32 bits


def _stream(r):
    """Bit offset and width of every dim's code in the K stream."""
    w = r["width"].astype(np.int64)
    off = r["bit_off"].astype(np.int64)
    return np.concatenate([off, off + w]), np.concatenate([w, w])


def _records(K, V, case, records):
    """Tile records of rows K, V [tiles][32][heads][128]: int32 [tiles][heads][words of a record]."""
    n, h = K.shape[0], case["hkv"]
    bk, bv = case["bits_k"], case["bits_v"]
    out = torch.empty((n, h, _record_bytes(case) // 4), dtype=torch.int32, device=K.device)
    for i, r in enumerate(records):
        off, w = _stream(r)
        gain = torch.from_numpy(np.concatenate([r["gain"], r["gain"]])).to(K.device)
        norm, codes = _row_codes(K[:, :, i], gain, w)
        out[:, i, :D * bk] = _bits(codes, off, w, 4 * bk).transpose(1, 2).reshape(n, -1)
        vn, codes = _row_codes(V[:, :, i], 1.0, np.full(D, bv))
        out[:, i, D * bk:D * bk + TILE] = torch.cat([norm, vn], 1).contiguous().view(torch.int32)
        words = _bits(codes.transpose(1, 2), bv * np.arange(TILE), np.full(TILE, bv), bv)    # [tiles][128][bv]
        out[:, i, D * bk + TILE:] = words.transpose(1, 2).reshape(n, -1)
    return out


def _unpack(rec, case, records):
    """Keys and values that records int32 [..., tiles][heads][words] stand for, fp32 [heads][..., tokens][128]."""
    bk, bv = case["bits_k"], case["bits_v"]
    dev = rec.device
    token = torch.arange(TILE, device=dev)
    ks, vs = [], []
    for i, r in enumerate(records):
        one = rec[..., i, :]
        norm = one[..., D * bk:D * bk + TILE].contiguous().view(torch.float16).float()       # 32 K norms, 32 V norms
        off, w = _stream(r)
        dims = np.flatnonzero(w)
        o, wd = (torch.from_numpy(a[dims]).to(dev) for a in (off, w))
        first = torch.cat([_codebook(x)[0] for x in range(1, 9)]).float().to(dev)            # width x at 2^x - 2
        at = (o >> 5) * TILE + token[:, None]                                                # [32][dims]
        lo = one[..., at].long() & 0xffffffff
        hi = one[..., torch.clamp(at + TILE, max=D * bk + TILE - 1)].long() & 0xffffffff     # the last word's next is unused
        code = ((lo | hi << 32) >> (o & 31)) & ((1 << wd) - 1)
        f = torch.from_numpy(np.concatenate([r["dequant"], r["dequant"]])[dims]).to(dev)
        k = torch.zeros(one.shape[:-1] + (TILE, D), device=dev)
        k[..., torch.from_numpy(dims).to(dev)] = first[(1 << wd) - 2 + code] * f * norm[..., :TILE, None]
        words = one[..., D * bk + TILE:].unflatten(-1, (bv, D)).long() & 0xffffffff
        words = torch.cat([words, torch.zeros_like(words[..., :1, :])], -2)
        bit = bv * token
        code = ((words[..., bit >> 5, :] | words[..., (bit >> 5) + 1, :] << 32) >> (bit & 31)[:, None]) & ((1 << bv) - 1)
        v = _codebook(bv)[0].float().to(dev)[code] * (norm[..., TILE:, None] / math.sqrt(D))
        ks.append(k.flatten(-3, -2))
        vs.append(v.flatten(-3, -2))
    return torch.stack(ks), torch.stack(vs)


def _pages(s):
    """The pool's records as int32 [pages][tiles of a page][heads][words] (stored head first)."""
    c = s["case"]
    body = s["pool"][s["header"]:].view(torch.int32)
    return body.view(s["n_pages"], c["hkv"], c["page"] // TILE, -1).transpose(1, 2)


def _plain_append(s):
    c, dev = s["case"], s["K"].device
    k = _rotate(s["K"], s["table"], s["positions"], s["axis"]) if c["axes"] else s["K"]
    # every tile that gets a token: its stored tokens stay, tokens past the last one are zeroed
    lens, new = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    first, end = lens // TILE, (lens + new + TILE - 1) // TILE
    count = torch.where(new > 0, end - first, 0)
    seq = torch.repeat_interleave(torch.arange(c["batch"], device=dev), count)
    if not len(seq):
        return s["pool"]
    tile = first[seq] + torch.arange(len(seq), device=dev) - (torch.cumsum(count, 0) - count)[seq]
    pos = tile[:, None] * TILE + torch.arange(TILE, device=dev)
    row = s["cu"][:-1].long()[seq][:, None] + pos - lens[seq][:, None]
    old, past = pos < lens[seq][:, None], pos >= (lens + new)[seq][:, None]
    row = torch.where(old | past, len(k), row)
    pad = lambda x: torch.cat([x, torch.zeros_like(x[:1])])[row]  # noqa: E731
    rec = _records(pad(k), pad(s["V"]), c, s["records"])
    page = s["block_table"][seq, tile // (c["page"] // TILE)].long()
    # a zero row has zero norms and, by the rule for tokens that are not there, zero codes
    bk, bv = c["bits_k"], c["bits_v"]
    kw, vw = rec[..., :D * bk].unflatten(-1, (-1, TILE)), rec[..., D * bk + TILE:].unflatten(-1, (bv, D))
    kw.masked_fill_((old | past)[:, None, None, :], 0)
    ones = torch.full((len(seq), TILE), (1 << bv) - 1, dtype=torch.int32, device=dev)
    span = lambda m: _bits(torch.where(m, ones, 0), bv * np.arange(TILE), np.full(TILE, bv), bv)[:, None, :, None]  # noqa: E731
    vw &= span(~(old | past))
    pages, slot = _pages(s), tile % (c["page"] // TILE)
    was = pages[page, slot]
    kw += was[..., :D * bk].unflatten(-1, (-1, TILE)) * old[:, None, None, :]
    vw |= was[..., D * bk + TILE:].unflatten(-1, (bv, D)) & span(old)
    norms = rec[..., D * bk:D * bk + TILE].view(torch.int16).unflatten(-1, (2, TILE))
    norms += was[..., D * bk:D * bk + TILE].contiguous().view(torch.int16).unflatten(-1, (2, TILE)) * old[:, None, None, :]
    pages[page, slot] = rec
    return s["pool"]


def _plain_attention(s):
    c = s["case"]
    hkv, b = c["hkv"], c["batch"]
    q = s["q"].float().unflatten(1, (hkv, -1)) / math.sqrt(D)                               # [batch][heads][group][128]
    pages, tiles = _pages(s), c["page"] // TILE
    longest = int(max(_lens(c)))
    seen = torch.arange(longest, device=q.device) < s["lens"][:, None]
    parts = []
    if longest:
        at = torch.where(seen[:, ::c["page"]], s["block_table"][:, :-(-longest // c["page"])], 0)
        k, v = _unpack(pages[at.long()].flatten(1, 2), c, s["records"])                     # [heads][batch][tokens][128]
        z = torch.einsum("bhgd,hbtd->bhgt", q, k[:, :, :longest]).masked_fill(~seen[:, None, None, :], -math.inf)
        parts.append((z, v[:, :, :longest], "bhgt,hbtd->bhgd"))
    if c["prefix"]:
        k, v = _unpack(pages[s["prefix_pages"].long()].flatten(0, 1), c, s["records"])      # [heads][tokens][128]
        z = torch.einsum("bhgd,htd->bhgt", q, k[:, :c["prefix"]])
        parts.append((z, v[:, :c["prefix"]], "bhgt,htd->bhgd"))
    if not parts:
        return torch.zeros((b, c["hq"], D), dtype=DTYPES[c["out"]], device=q.device)
    m = torch.stack([z.amax(-1) for z, _, _ in parts]).amax(0)[..., None]
    m = torch.where(m.isinf(), 0.0, m)                                                      # nothing to attend to
    o, total = 0.0, 0.0
    for z, v, rule in parts:
        p = torch.exp(z - m)
        o, total = o + torch.einsum(rule, p, v), total + p.sum(-1, keepdim=True)
    return torch.where(total > 0, o / total, 0.0).flatten(1, 2).to(DTYPES[c["out"]])


# ------------------------------------------------------------------------------ measured calls

def _table(n, dev):
    """cos and sin of position p's angle in block b, p * 1e6^(-b / 64), from 64 bits."""
    b = torch.arange(H2, dtype=torch.float64, device=dev)
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * torch.pow(1e6, -b / H2)
    return torch.stack([torch.cos(a), torch.sin(a)], -1).float()


def _axes(case, dev):
    """Which axis turns a block: sections of 16, 24 and 24 blocks for three, interleaved otherwise."""
    b = np.arange(H2)
    axis = np.minimum((b + 8) // 24, 2) if case["axes"] == 3 else b % max(1, case["axes"])
    return torch.from_numpy(axis.astype(np.int32)).to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = np.random.RandomState(seed % (1 << 31))
    dt = DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    whole = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    s = {"case": dict(case)}
    if case["op"] == "rope":
        n = case["tokens"]
        start = host.randint(0, case["positions"] - min(n, case["positions"]) + 1)
        s |= {"x": normal(n, case["heads"], D).to(dt), "table": _table(case["positions"], dev), "axis": _axes(case, dev)}
        line = start + np.arange(n) if n > 64 else host.randint(0, case["positions"], n)     # a prompt, or a batch's steps
        s["positions"] = whole([(line // (1 + 7 * a * a)) % case["positions"] for a in range(case["axes"])])
        return s
    h, page = case["hkv"], case["page"]
    # block energies as keys have them: log-normal scales and two blocks far above the others
    sigma = np.exp(host.randn(h, H2))
    sigma[:, host.permutation(H2)[:2]] *= 20.0
    records = [_allocation(2.0 * sigma[i] ** 2, case["bits_k"]) for i in range(h)]
    scale = torch.from_numpy(np.concatenate([sigma, sigma], 1)).float().to(dev)
    lens = np.array(_lens(case))
    new = np.array(_new(case)) if case["op"] == "append" else np.zeros_like(lens)
    need = -(-(lens + new) // page)
    shared = -(-case.get("prefix", 0) // page)
    n_pages = int(need.sum() + shared + 3)
    ids = host.permutation(n_pages)
    table = np.full((case["batch"], int(need.max()) + 1), -1)
    starts = np.concatenate([[0], np.cumsum(need)])
    for i, n in enumerate(need):
        table[i, :n] = ids[starts[i]:starts[i + 1]]
    header = _header(case, n_pages, records)
    pool = torch.empty(len(header) + n_pages * h * (page // TILE) * _record_bytes(case), dtype=torch.uint8, device=dev)
    pool[:len(header)] = header.to(dev)
    s |= {"pool": pool, "header": len(header), "n_pages": n_pages, "records": records, "block_table": whole(table),
          "lens": whole(lens), "alloc": torch.from_numpy(np.frombuffer(b"".join(r.tobytes() for r in records), np.uint8).copy()).to(dev)}
    pages = _pages(s)
    at_once = max(1, (1 << 18) // (h * page))                # pages filled at a time
    for p in range(0, n_pages, at_once):
        n = min(at_once, n_pages - p) * (page // TILE)
        k, v = normal(n, TILE, h, D) * scale, normal(n, TILE, h, D)
        pages[p:p + at_once] = _records(k.to(dt), v.to(dt), case, records).view(-1, page // TILE, h, _record_bytes(case) // 4)
    if case["op"] == "append":
        n = int(new.sum())
        s |= {"K": (normal(n, h, D) * scale).to(dt), "V": normal(n, h, D).to(dt), "cu": whole(np.concatenate([[0], np.cumsum(new)]))}
        if case["axes"]:
            pos = np.concatenate([np.arange(m) + l for m, l in zip(new, lens)] + [np.zeros(0, np.int64)])
            s |= {"table": _table(int((lens + new).max()) + 1, dev), "axis": _axes(case, dev),
                  "positions": whole([pos // (1 + 7 * a * a) for a in range(case["axes"])])}
    else:
        s |= {"q": normal(case["batch"], case["hq"], D).to(dt), "prefix_pages": whole(ids[starts[-1]:starts[-1] + shared])}
    return s


def _own(s):
    from packed_cache_attention_b200 import kvq
    c = s["case"]
    rope = None
    if c.get("axes"):
        if "axis_list" not in s:
            s["axis_list"] = s["axis"].tolist()
        rope = kvq.rope_desc(s["table"], s["positions"], s["axis_list"])
    if c["op"] == "rope":
        return kvq.kvq_rope(s["x"], rope)
    desc = kvq.paged_desc(s["n_pages"], c["page"], c["hkv"], c["bits_k"], c["bits_v"])
    if c["op"] == "append":
        return kvq.kvq_paged_append(s["K"], s["V"], s["alloc"], desc, s["block_table"], s["lens"], s["cu"], s["pool"], rope=rope)
    if "ws" not in s:
        s["ws"] = kvq.kvq_paged_decode_workspace(desc, c["batch"], c["hq"], c["prefix"])
    return kvq.kvq_paged_decode_attn(s["q"], s["pool"], s["alloc"], desc, s["block_table"], s["lens"],
                                     prefix_pages=s["prefix_pages"] if c["prefix"] else None, prefix_len=c["prefix"],
                                     out_dtype=DTYPES[c["out"]], ws=s["ws"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _rotate(state["x"], state["table"], state["positions"], state["axis"])
    return _plain_append(state) if op == "append" else _plain_attention(state)


# ------------------------------------------------------------------------------ in 64 bits

def _bit_values(words, order):
    """Numbers from the bits of int32 words [..., n]: order lists, per number, its bits' places."""
    bits = (words[..., None] >> torch.arange(32, device=words.device)) & 1
    bits = torch.cat([bits.flatten(-2), torch.zeros_like(bits[..., 0, :1])], -1)              # a last bit, 0, for places of none
    return (bits[..., order].double() * (2.0 ** torch.arange(order.shape[-1], device=words.device).double())).sum(-1).long()


def _places(first, width):
    """Places of `width[i]` bits from `first[i]`, -1 (the zero bit) past them."""
    k = np.arange(8)[None, :]
    return np.where(k < np.asarray(width)[:, None], np.asarray(first)[:, None] + k, -1)


def _exact_kv(s, pages, count, head):
    """Keys and values of the first `count` tokens of `pages` for one head, 64 bits."""
    c, r = s["case"], s["records"][head]
    bk, bv = c["bits_k"], c["bits_v"]
    per = _record_bytes(c) * (c["page"] // TILE)
    base = s["pool"][s["header"]:].view(s["n_pages"], c["hkv"], per)[pages.long(), head].reshape(-1, _record_bytes(c)).contiguous()
    words = base.view(torch.int32)
    dev = words.device
    k = torch.zeros((len(words), TILE, D), dtype=torch.float64, device=dev)
    v = torch.zeros_like(k)
    norms = words[:, D * bk:D * bk + TILE].contiguous().view(torch.float16).double()
    kw = words[:, :D * bk].reshape(-1, 4 * bk, TILE).transpose(1, 2)
    for b in range(H2):
        w, at = int(r["width"][b]), int(r["bit_off"][b])
        if w:
            near = kw[..., at // 32:at // 32 + 2]
            code = _bit_values(near, torch.from_numpy(_places([at % 32, at % 32 + w], [w, w])).to(dev))
            k[..., [b, b + H2]] = _codebook(w)[0].double().to(dev)[code] * norms[:, :TILE, None] * float(r["dequant"][b])
    vw = words[:, D * bk + TILE:].reshape(-1, bv, D).transpose(1, 2)
    code = _bit_values(vw, torch.from_numpy(_places(bv * np.arange(TILE), [bv] * TILE)).to(dev)).transpose(1, 2)
    v = _codebook(bv)[0].double().to(dev)[code] * norms[:, TILE:, None] / math.sqrt(D)
    return k.reshape(-1, D)[:count], v.reshape(-1, D)[:count]


def exact(case, seed):
    if case["op"] == "append":
        return None                                           # packed bits: whole numbers, no values in between
    s = prepare(case, seed)
    if case["op"] == "rope":
        x, out = s["x"].double(), torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for b in range(H2):
            angle = s["table"][s["positions"][int(s["axis"][b])].long(), b].double()[:, None, :]
            z = torch.complex(x[..., b], x[..., b + H2]) * torch.view_as_complex(angle.contiguous())
            out[..., b], out[..., b + H2] = z.real, z.imag
        return out
    tokens = case["hkv"] * (case["prefix"] + sum(_lens(case)))
    if tokens > 1 << 21:
        return None
    group = case["hq"] // case["hkv"]
    out = torch.zeros((case["batch"], case["hq"], D), dtype=torch.float64, device="cuda")
    for h in range(case["hkv"]):
        pk, pv = _exact_kv(s, s["prefix_pages"], case["prefix"], h)
        for i, n in enumerate(_lens(case)):
            k, v = _exact_kv(s, s["block_table"][i, :-(-n // case["page"])], n, h)
            k, v = torch.cat([pk, k]), torch.cat([pv, v])
            if len(k):
                rows = slice(h * group, h * group + group)
                out[i, rows] = torch.softmax(s["q"][i, rows].double() @ k.T / math.sqrt(D), -1) @ v
    return out
