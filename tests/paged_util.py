"""Shared helpers of the paged-cache tests: a pool with its batch, and plain forms in 64 bits."""
import math

import numpy as np

from oracle import blockgtq as bg
from packed_cache_attention_b200 import kvq
from tests.parity_util import host_f32

LOG2E = 1.4426950408889634


def angle_table(n, base=1e6):
    """cos and sin of position p's angle in block b, p * base^(-b / 64), fp32 [n][64][2] from 64 bits."""
    a = np.arange(n, dtype=np.float64)[:, None] * np.power(base, -np.arange(64) / 64.0)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate_f32(x, table, positions, axis):
    """Plain rotation of host fp32 rows [tokens][heads][128], every operation rounded to fp32."""
    cs = table[positions[axis], np.arange(64)[:, None]]                   # [64][tokens][2]
    c, s = (cs[..., i].T[:, None, :] for i in (0, 1))
    x1, x2 = x[..., :64], x[..., 64:]
    return np.concatenate([x1 * c - x2 * s, x2 * c + x1 * s], -1)


class Paged:
    """A pool, its allocation and the pages of a batch, every page id different and out of order."""

    def __init__(self, dev, seed, hkv, bits_k, bits_v, page, lens_max, prefix=0, spare=2, profile_tokens=300):
        import torch
        self.torch, self.dev, self.page, self.hkv, self.bits_k, self.bits_v = torch, dev, page, hkv, bits_k, bits_v
        self.rng = np.random.default_rng(seed)
        self.sigma = np.exp(self.rng.standard_normal((hkv, 64)))
        self.sigma[:, self.rng.permutation(64)[:2]] *= 20.0
        self.scale = torch.from_numpy(np.concatenate([self.sigma, self.sigma], 1)).float().to(dev)
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        keys = torch.randn((1, hkv, profile_tokens, 128), generator=self.gen, device=dev) * self.scale[None, :, None]
        self.alloc = kvq.kvq_calibrate(keys, bits_k)
        self.ref = bg.calibrate(host_f32(keys), bits_k)
        need = [-(-n // page) for n in lens_max]
        shared = -(-prefix // page)
        n_pages = sum(need) + shared + spare
        ids = self.rng.permutation(n_pages).astype(np.int32)
        self.desc = kvq.paged_desc(n_pages, page, hkv, bits_k, bits_v)
        table = np.full((len(need), max(max(need), 1)), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table_np, self.prefix_np, self.unused = table, ids[at:at + shared], ids[at + shared:]
        self.table, self.prefix_pages = (torch.from_numpy(x).to(dev) for x in (table, self.prefix_np))
        # whatever a page held before must not matter: random bytes, NaN and infinite norms among them
        self.pool = torch.randint(0, 256, (kvq.kvq_paged_bytes(self.desc),), generator=self.gen, device=dev, dtype=torch.uint8)
        kvq.kvq_paged_init(self.alloc, self.desc, self.pool)
        self.hdr, self.rec = bg.header_bytes(hkv), bg.tile_record_bytes(128, bits_k, bits_v)

    def ints(self, a):
        return self.torch.from_numpy(np.asarray(a, np.int32)).to(self.dev)

    def rows(self, n, dtype):
        """New keys and values [n][hkv][128]."""
        torch = self.torch
        k = torch.randn((n, self.hkv, 128), generator=self.gen, device=self.dev) * self.scale[None]
        v = torch.randn((n, self.hkv, 128), generator=self.gen, device=self.dev)
        return k.to(dtype), v.to(dtype)

    def append(self, K, V, lens, cu, table=None, rope=None, **kw):
        return kvq.kvq_paged_append(K, V, self.alloc, self.desc, self.table if table is None else table, self.ints(lens),
                                    self.ints(cu), self.pool, rope=rope, **kw)

    def records(self, pages):
        """Host copy of pages' records in order: uint8 [1][hkv][tiles][record]."""
        body = self.pool[self.hdr:].cpu().numpy().reshape(self.desc.n_pages, self.hkv, self.page // 32, self.rec)
        return np.concatenate([body[p] for p in pages], 1)[None]

    def kv(self, pages, n):
        """Keys and values of the first n positions of `pages`, fp64 [hkv][n][128]."""
        if n == 0:
            return (np.zeros((self.hkv, 0, 128)),) * 2
        u = bg.unpack_cache(self.records(pages[:-(-n // self.page)]), self.ref, self.bits_v, n)
        return (bg.dequantize_keys(u["Kc"], u["Kn"], self.ref)[0], bg.dequantize_values(u["Vc"], u["Vn"], self.bits_v)[0])

    def fill(self, lens, dtype, prefix=0, at_prefix=None):
        """Appends random tokens up to `lens` (and to the prefix pages)."""
        cu = np.concatenate([[0], np.cumsum(lens)])
        if cu[-1]:
            K, V = self.rows(int(cu[-1]), dtype)
            self.append(K, V, [0] * len(lens), cu)
        if prefix:
            K, V = self.rows(prefix, dtype)
            self.append(K, V, [0], [0, prefix], table=self.prefix_pages[None].contiguous())
        assert kvq.kvq_packed_status(self.pool) == 0

    def decode(self, q, lens, prefix=0, **kw):
        return kvq.kvq_paged_decode_attn(q, self.pool, self.alloc, self.desc, self.table, self.ints(lens),
                                         prefix_pages=self.prefix_pages if prefix else None, prefix_len=prefix, **kw)

    def attention(self, q, lens, prefix=0, out=None):
        """(rows in 64 bits, bound of an fp32 kernel's error) for q [B][Hq][128].

        The bound counts the kernel's roundings at their worst. A logit is q' . k over at most 24
        products of 16 terms, high and low parts (each at most 2^-22 off the sum of magnitudes A,
        the split of q' 2^-22 more): A 2^-17 in log2 units. p is off by that times ln 2, in the
        numerator and in the sum; sums over up to 2^12 tokens in at most 2^8 + 2^8 steps of 2^-22, and
        the exponential, the splits of p and the merges, are together below 2^-12. A weighted mean
        of the values then moves by at most that share of the largest value. For bf16 outputs (`out`) a prefix's
        shares are rounded to fp16, 2^-11 more."""
        import torch
        shares = 2.0 ** -12 + (2.0 ** -11 if prefix and out == torch.bfloat16 else 0.0)
        q = host_f32(q).astype(np.float64)
        B, Hq, _ = q.shape
        G = Hq // self.hkv
        out, bound = np.zeros(q.shape), np.zeros((B, Hq, 1))
        pk, pv = self.kv(self.prefix_np, prefix)
        for b, n in enumerate(lens):
            k, v = self.kv(self.table_np[b], n)
            k, v = np.concatenate([pk, k], 1), np.concatenate([pv, v], 1)
            if k.shape[1] == 0:
                continue
            for h in range(Hq):
                kk, vv = k[h // G], v[h // G]
                z = kk @ q[b, h] / math.sqrt(128.0)
                p = np.exp(z - z.max())
                out[b, h] = (p @ vv) / p.sum()
                A = (np.abs(kk) @ np.abs(q[b, h])).max() / math.sqrt(128.0) * LOG2E
                bound[b, h] = (2 * math.log(2) * A * 2.0 ** -17 + shares) * np.abs(vv).max()
        return out, bound


def check_rows(got, want, bound, dtype):
    """got [B][Hq][128] within the kernel's bound and half a step of its type of `want`."""
    import torch
    half = torch.finfo(dtype).eps / 2
    g = host_f32(got).astype(np.float64)
    assert np.isfinite(g).all()
    err = np.abs(g - want)
    lim = bound * (1 + half) + half * np.abs(want) + torch.finfo(dtype).tiny
    assert (err <= lim).all(), (float((err / lim).max()), float(err.max()))


def rows_and_bound(k, v, q):
    """softmax(q . k / sqrt(128)) . v in 64 bits for q [heads][128], and a bound of an fp32 kernel's error,
    element by element, for one KV head and at most 148 * 128 positions (a share of the kernels is then one chunk).

    A softmax weight is off by a relative e, in the numerator and in the sum, so an output by at most 2 e of
    the weighted mean of |v|. e is: the logit's error times ln 2, with A the sum of |q k| in log2 units: the
    pair of a query 2^-22 of each product, fp32 sums of 24 products cut off at 2^-23, the products with the
    norm and the scale, 2^-24 each of A: below 2^-18 A (high and low sums one after the other: 2^-17 A); the
    pair of a share 2^-22; a chunk's 16 products cut off at 2^-23: 2^-19; 2^x and row sums of a chunk 2^-19;
    the merge of at most 148 shares by 16 warps and of those 2^-18: together below 2^-17. Shares below fp16's
    normal range are off by 2^-38 of the largest share, times a centroid below 5."""
    z = (k @ q.T).T / math.sqrt(128.0)                                    # [heads][tokens]
    p = np.exp(z - z.max(1, keepdims=True))
    total = p.sum(1, keepdims=True)
    A = (np.abs(k) @ np.abs(q.T)).T.max(1) / math.sqrt(128.0) * LOG2E
    e = A * math.log(2) * 2.0 ** -17 + 2.0 ** -17
    largest = (p * np.abs(v).max(1)).max(1, keepdims=True)
    return p @ v / total, 2 * e[:, None] * (p @ np.abs(v)) / total + 5 * p.shape[1] * 2.0 ** -38 * largest / total


def check_close(got, want, bound, dtype):
    """got within the bound and half a step of its type of `want`."""
    import torch
    f = torch.finfo(dtype)
    g = host_f32(got).astype(np.float64)
    assert np.isfinite(g).all()
    lim = bound * (1 + f.eps) + f.eps / 2 * np.abs(want) + f.tiny * f.eps
    err = np.abs(g - want)
    assert (err <= lim).all(), (float((err / lim).max()), float(err.max()))
