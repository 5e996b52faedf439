"""Rotary positions and the paged cache without a GPU: struct layouts, sizes, and the calls that
are refused before anything is launched."""
import ctypes
import math

import numpy as np
import pytest

from oracle import blockgtq as bg
from oracle import rope as orope
from packed_cache_attention_b200 import kvq
from tests import test_c_client as cc
from tests.paged_util import angle_table, check_close, rotate_f32, rows_and_bound
from tests.test_abi import L, WS_BYTES, _t4, buf  # noqa: F401

ARG, SHAPE, DTYPE, RANGE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 5, 6, 9


def test_structs_have_the_headers_layout(tmp_path, monkeypatch):
    structs = [("kvq_rope_desc", kvq.RopeDesc), ("kvq_paged_desc", kvq.PagedDesc), ("kvq_page_table", kvq.PageTable),
               ("kvq_prefix", kvq.Prefix)]
    monkeypatch.setattr(cc, "STRUCTS", structs)
    cc.test_binding_structs_have_the_headers_layout(tmp_path)


def test_sizes_follow_the_layout(L):
    for (n, page, h, bk, bv) in [(1, 32, 1, 1, 1), (10, 64, 2, 3, 3), (7, 256, 8, 4, 5), (3, 65536, 9, 8, 8)]:
        want = bg.header_bytes(h) + n * h * (page // 32) * bg.tile_record_bytes(128, bk, bv)
        assert kvq.kvq_paged_bytes(kvq.paged_desc(n, page, h, bk, bv)) == want
        assert kvq._pool_bytes(kvq.paged_desc(n, page, h, bk, bv)) == want
    for bad in [(0, 64, 2, 3, 3), (4, 33, 2, 3, 3), (4, 0, 2, 3, 3), (4, 65568, 2, 3, 3), (4, 64, 0, 3, 3), (4, 64, 2, 0, 3),
                (4, 64, 2, 9, 3), (4, 64, 2, 3, 0), (4, 64, 2, 3, 9), (4, 64, 2, 3, 3, 64)]:
        assert kvq.kvq_paged_bytes(kvq.paged_desc(*bad)) == 0, bad
    d = kvq.paged_desc(100, 64, 2, 3, 3)
    ws = lambda *a: kvq.kvq_paged_decode_workspace_bytes(d, *a)  # noqa: E731
    assert ws(4, 16, 100) > ws(4, 16, 0) > 0
    assert ws(4, 16, 1) == ws(4, 16, 131072)                              # any length
    for bad in [(0, 16, 0), (1025, 16, 0), (4, 15, 0), (4, 18, 0), (4, 0, 0), (4, 16, -1)]:
        assert ws(*bad) == 0, bad
    assert ws(1024, 16, 100) > 0
    with pytest.raises(ValueError):
        kvq.kvq_paged_decode_workspace(d, 0, 16, 0, "cpu")


def test_plain_rotation_is_the_rotation_of_the_formula():
    """The tests' fp32 rotation against the complex rotation in 64 bits, three axes."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((9, 3, 128)).astype(np.float32)
    axis = np.minimum((np.arange(64) + 8) // 24, 2)
    pos = rng.integers(0, 500, (3, 9))
    got = rotate_f32(x, angle_table(500), pos, axis)
    for t in range(9):
        for h in range(3):
            for a in range(3):
                r = orope.rotate(x[t, h], float(pos[a, t]), 1e6)
                dims = np.concatenate([np.flatnonzero(axis == a), np.flatnonzero(axis == a) + 64])
                scale = np.abs(x[t, h]).max()
                assert np.abs(got[t, h, dims] - r[dims]).max() <= 8 * 2.0 ** -24 * scale


def _rope(mem, n_pos=16, n_axes=1, stride=64, **kw):
    r = kvq.RopeDesc(mem, mem, stride, n_pos, n_axes)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_rope_refusals(L):
    mem = buf()
    out = buf()
    call = lambda xd, r, od=None, o=None, x=None: L.kvq_rope(  # noqa: E731
        mem if x is None else x, ctypes.byref(xd), ctypes.byref(r) if r else None, out if o is None else o,
        ctypes.byref(xd if od is None else od), None)
    x = _t4(T=8)
    assert call(x, None) == ARG
    assert call(_t4(T=0), _rope(mem)) == SHAPE
    assert call(_t4(T=8, d=64), _rope(mem)) == SHAPE
    assert call(_t4(T=8, dtype=5), _rope(mem)) == DTYPE
    assert call(x, _rope(mem), od=_t4(T=8, dtype=kvq.KVQ_F16)) == DTYPE
    assert call(x, _rope(mem), od=_t4(T=8, H=1)) == SHAPE
    assert call(x, _rope(mem), o=out + 8) == ARG                           # misaligned
    assert call(x, _rope(mem), od=_t4(T=8, sh=0)) == ARG                   # two heads written to one place
    assert call(x, _rope(mem), od=_t4(T=8, sh=64)) == ARG                  # rows overlap
    assert call(x, _rope(mem), od=_t4(T=8, st=256, sh=128), o=mem) == ARG  # in place with other strides
    assert call(x, _rope(0)) == ARG
    assert call(x, _rope(mem, table=mem + 8)) == ARG
    assert call(x, _rope(mem, n_pos=0)) == SHAPE
    assert call(x, _rope(mem, n_axes=0)) == SHAPE
    assert call(x, _rope(mem, n_axes=5)) == SHAPE
    assert call(x, _rope(mem, n_axes=2, stride=7)) == ARG                  # axes' positions overlap
    r = _rope(mem)
    r.axis[63] = 1
    assert call(x, r) == ARG                                               # axis 1 of one


def _pages(mem, batch=2, max_pages=4, stride=None, **kw):
    t = kvq.PageTable(mem, mem, max_pages if stride is None else stride, batch, max_pages)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


D = kvq.paged_desc(8, 64, 2, 3, 3)


def test_init_refusals(L):
    mem = buf()
    init = lambda a, d, p: L.kvq_paged_init(a, ctypes.byref(d) if d else None, p, None)  # noqa: E731
    assert init(mem, None, mem) == ARG
    assert init(mem, kvq.paged_desc(8, 48, 2, 3, 3), mem) == ARG
    assert init(None, D, mem) == ARG
    assert init(mem, D, None) == ARG
    assert init(mem, D, mem + 8) == ARG


def test_append_refusals(L):
    mem = buf()

    def call(kd=None, vd=None, rope=None, d=D, seqs=None, cu=mem, pool=mem, alloc=mem, K=mem):
        kd = _t4(T=10) if kd is None else kd
        vd = kd if vd is None else vd
        seqs = _pages(mem) if seqs is None else seqs
        return L.kvq_paged_append(K, ctypes.byref(kd), mem, ctypes.byref(vd), ctypes.byref(rope) if rope else None, alloc,
                                  ctypes.byref(d), ctypes.byref(seqs), cu, pool, None)
    assert call(K=None) == ARG
    assert call(kd=_t4(T=0)) == SHAPE
    assert call(kd=_t4(T=10, B=2)) == SHAPE
    assert call(kd=_t4(T=10, H=3)) == SHAPE
    assert call(vd=_t4(T=9)) == SHAPE
    assert call(vd=_t4(T=10, dtype=kvq.KVQ_F16)) == DTYPE
    assert call(kd=_t4(T=10, st=132)) == ARG
    assert call(cu=None) == ARG and call(pool=None) == ARG and call(alloc=None) == ARG
    assert call(pool=mem + 4) == ARG
    assert call(d=kvq.paged_desc(8, 64, 2, 3, 0)) == ARG
    for bad in (dict(batch=0), dict(batch=1025), dict(max_pages=0)):
        assert call(seqs=_pages(mem, **bad)) == SHAPE
    assert call(seqs=_pages(mem, stride=3)) == ARG                        # table rows overlap
    assert call(seqs=_pages(mem, batch=1, max_pages=1 << 26)) == RANGE    # positions are 32-bit
    assert call(seqs=_pages(mem, block_table=None)) == ARG
    assert call(seqs=_pages(mem, seq_lens=None)) == ARG
    assert call(rope=_rope(mem, n_axes=3, stride=9)) == ARG
    assert call(rope=_rope(mem, n_pos=0)) == SHAPE


def test_decode_refusals(L):
    mem, ws = buf(), buf(WS_BYTES)

    def call(qd=None, d=D, seqs=None, prefix=None, out=mem, dtype=0, w=ws, wsb=WS_BYTES, pool=mem):
        qd = kvq.Tensor4(2, 16, 1, 128, 2048, 128, 128, kvq.KVQ_BF16, 0) if qd is None else qd
        seqs = _pages(mem) if seqs is None else seqs
        return L.kvq_paged_decode_attn(mem, ctypes.byref(qd), pool, mem, ctypes.byref(d), ctypes.byref(seqs),
                                       ctypes.byref(prefix) if prefix else None, out, dtype, w, wsb, None)
    assert call(qd=kvq.Tensor4(3, 16, 1, 128, 2048, 128, 128, 2, 0)) == SHAPE       # another batch
    assert call(qd=kvq.Tensor4(2, 16, 2, 128, 4096, 256, 128, 2, 0)) == SHAPE       # two tokens
    assert call(qd=kvq.Tensor4(2, 15, 1, 128, 2048, 128, 128, 2, 0)) == UNSUPPORTED
    assert call(qd=kvq.Tensor4(2, 18, 1, 128, 2304, 128, 128, 2, 0)) == UNSUPPORTED  # 9 heads a KV head
    assert call(pool=None) == ARG and call(out=None) == ARG and call(out=mem + 4) == ARG
    assert call(dtype=3) == DTYPE and call(dtype=-1) == DTYPE
    assert call(d=kvq.paged_desc(8, 64, 2, 3, 0)) == ARG
    assert call(seqs=_pages(mem, batch=0)) == SHAPE
    assert call(prefix=kvq.Prefix(mem, 2, -1)) == RANGE
    assert call(prefix=kvq.Prefix(mem, 2, 129)) == RANGE                            # longer than its pages
    assert call(prefix=kvq.Prefix(mem, 1 << 30, 2 ** 31 - 1)) == RANGE              # no room to round up
    assert call(prefix=kvq.Prefix(None, 2, 100)) == ARG
    assert call(w=None) == WORKSPACE and call(wsb=1 << 10) == WORKSPACE
    need = kvq.kvq_paged_decode_workspace_bytes(D, 2, 16, 100)
    assert call(prefix=kvq.Prefix(mem, 2, 100), wsb=need - 1) == WORKSPACE


def test_binding_refuses_host_tensors_and_wrong_arguments(L):
    import torch
    table = torch.from_numpy(angle_table(16))
    pos = torch.zeros(4, dtype=torch.int32)
    r = kvq.rope_desc(table, pos)
    with pytest.raises(ValueError, match="device"):
        kvq.kvq_rope(torch.zeros(4, 2, 128), r)
    with pytest.raises(ValueError):
        kvq.rope_desc(table.double(), pos)
    with pytest.raises(ValueError):
        kvq.rope_desc(table, pos.long())
    with pytest.raises(ValueError):
        kvq.rope_desc(table, pos, [0] * 63)
    with pytest.raises(ValueError):
        kvq.rope_desc(table.transpose(1, 2), pos)
    with pytest.raises(ValueError):
        kvq._ints(torch.zeros(3, 8, dtype=torch.int32)[:, ::2], "block_table", 3, None)
    with pytest.raises(ValueError):
        kvq._bytes(torch.zeros(10, dtype=torch.uint8), "pool", 11)
    with pytest.raises(ValueError):
        kvq._rows(torch.zeros(4, 128))
    with pytest.raises(ValueError):
        kvq._rope_tokens(r, 5)
    z = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvq.kvq_paged_decode_attn(torch.zeros(2, 16, 128), torch.zeros(8, dtype=torch.uint8),
                                  torch.zeros(8, dtype=torch.uint8), D, z, z[:, 0])


def test_every_split_rule_covers_the_batch():
    """The rule that shares a ragged batch out: for any lengths the rounds it settles on fit the slots, no
    sequence's split is empty, and no CTA gets more rounds than the longest sequence needs alone."""
    rng = np.random.default_rng(1)
    for _ in range(300):
        n = int(rng.integers(1, 70))
        chunks = rng.integers(0, int(rng.integers(1, 2000)), n)
        slots = max(n, int(rng.integers(1, 148)))
        least = max(1, -(-int(chunks.sum()) // (4 * slots)))
        most = max(1, -(-int(chunks.max()) // 4))
        tries = [least + -(-least * w // 8) for w in range(19)] + [most]
        fits = [p for p in tries if sum(-(-int(c) // (4 * p)) for c in chunks) <= slots]
        best = min(fits)
        splits = [-(-int(c) // (4 * best)) for c in chunks]
        assert sum(splits) <= slots and best <= max(most, least * 4)
        for c, s in zip(chunks, splits):
            assert (s == 0) == (c == 0)
            for i in range(s):
                assert (i + 1) * int(c) // s > i * int(c) // s
        assert math.isfinite(best)


def test_axis_maps_of_every_kind_are_their_numbers():
    """Lists, tuples, bytes, numpy and torch integers of any width, strided ones: the same 64 bytes."""
    import array

    import torch
    table, pos = torch.from_numpy(angle_table(4)), torch.zeros((4, 5), dtype=torch.int32)
    want = np.minimum((np.arange(64) + 8) // 24, 2)
    kinds = [want.tolist(), tuple(want.tolist()), bytes(want.tolist()), bytearray(want.tolist()), [np.int32(a) for a in want],
             array.array("i", want.tolist()), array.array("q", want.tolist()), range(64)]
    kinds += [want.astype(t) for t in (np.uint8, np.int8, np.int16, np.int32, np.int64, np.uint64)]
    kinds += [np.repeat(want.astype(np.int32), 2)[::2], torch.from_numpy(want), torch.from_numpy(want).int(), torch.from_numpy(want).to(torch.uint8)]
    for axis in kinds:
        r = kvq.rope_desc(table, pos, axis)
        assert bytes(r.axis) == bytes(range(64)) if isinstance(axis, range) else list(r.axis) == want.tolist(), type(axis)
    for bad in (want.astype(np.float32), want[:63], [0] * 65, [-1] * 64, [256] * 64, [[0]] * 64, "0" * 64, want.reshape(64, 1),
                torch.from_numpy(want).float()):
        with pytest.raises(ValueError):
            kvq.rope_desc(table, pos, bad)


@pytest.mark.parametrize("batch,max_pages", [(1024, (1 << 19) + 1), (17, (1 << 25) - 65), (2, 1 << 25)])
def test_batches_whose_tiles_do_not_fit_32_bits_are_refused(L, batch, max_pages):
    """max_pages * 64 * batch past 2^35 (or a sequence past 2^31 - 4096 positions), by append and decode."""
    mem, ws = buf(), buf(WS_BYTES)
    seqs = _pages(mem, batch=batch, max_pages=max_pages)
    kd = _t4(T=10)
    assert L.kvq_paged_append(mem, ctypes.byref(kd), mem, ctypes.byref(kd), None, mem, ctypes.byref(D), ctypes.byref(seqs), mem, mem,
                              None) == RANGE
    qd = kvq.Tensor4(batch, 16, 1, 128, 2048, 128, 128, kvq.KVQ_BF16, 0)
    assert L.kvq_paged_decode_attn(mem, ctypes.byref(qd), mem, mem, ctypes.byref(D), ctypes.byref(seqs), None, mem, 0, ws, WS_BYTES,
                                   None) == RANGE


SPLIT_SOURCE = r"""
#include "paged_split.h"
#include <vector>
using namespace kvq;

// One head's decode of a list (cs: chunk offsets of the sequences): every share it leaves, as the
// kernel's warpgroups walk their ranges, in `put(entry, sequence, first chunk, chunks)`; then the shares that the
// merge reads for every sequence. Returns 0, or the number of the first thing that does not fit.
extern "C" int split(int batch, const int* cs, int ctas, long long* shares) {
  const int chunks = cs[batch], entries = 4 * ctas + batch;
  const Shares sh(chunks, ctas);
  struct Left { int b, n, times; };
  std::vector<Left> left(entries, Left{-1, 0, 0});
  int walked = 0;
  for (int cta = 0; cta < ctas; ++cta) {
    const CtaShare c(sh, cs, batch, cta);
    if (c.w_end - c.w > 4) return 1;                        // a warpgroup has one range
    for (int g = 0; g < 4 && g < sh.per_cta; ++g) {
      const int w = c.w + g;
      int x = w < sh.workers ? sh.first(w) : 0;
      const int x1 = w < sh.workers ? sh.first(w + 1) : 0;
      if (w < sh.workers && x1 <= x) return 2;              // an empty range
      if (x1 - x > sh.per) return 3;
      int b = x1 > x ? find_span(cs, batch, x) : 0;
      while (x < x1) {
        const int n = (x1 < cs[b + 1] ? x1 : cs[b + 1]) - x;
        if (n <= 0 || x < cs[b]) return 4;
        const int e = c.joint ? c.w + c.b : w + b;
        if (c.joint && b != c.b) return 5;
        if (e < 0 || e >= entries) return 6;
        if (left[e].b >= 0 && (left[e].b != b || !c.joint)) return 7;   // two shares at one entry
        left[e].b = b;
        left[e].n += n;
        walked += n;
        x += n;
        if (x < x1) do ++b; while (cs[b + 1] == x);
      }
    }
  }
  if (walked != chunks) return 8;
  *shares = 0;
  for (int b = 0; b < batch; ++b) {
    const OwnShares own(sh, cs[b], cs[b + 1] - cs[b]);
    int n = 0;
    for (int k = 0; k < own.n; ++k) {
      const int e = own.worker(k) + b;
      if (e < 0 || e >= entries || left[e].b != b || left[e].times++) return 9;   // not written, another's, or twice
      n += left[e].n;
    }
    if (n != cs[b + 1] - cs[b]) return 10;                  // a share is missed
    *shares += own.n;
  }
  for (const Left& l : left)
    if (l.b >= 0 && l.times != 1) return 11;                // a share that nobody reads
  return 0;
}
"""


def test_decode_and_merge_agree_on_every_share(tmp_path):
    """The functions that the kernels call, compiled for the host: for random batches (empty sequences, one long one,
    more sequences than warpgroups) every chunk is walked once, no two shares have one entry, and the merge reads
    each share of its sequence once and no other."""
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src, so = tmp_path / "split.cpp", tmp_path / "split.so"
    src.write_text(SPLIT_SOURCE)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover", "-shared", "-fPIC",
                    "-static-libgcc", "-I", cc.ROOT + "/packed_cache_attention_b200/csrc", str(src), "-o", str(so)], check=True)
    split = ctypes.CDLL(str(so)).split
    rng = np.random.default_rng(2)
    got = ctypes.c_longlong()
    batches = [([0], 1), ([1], 148), ([0, 0, 0], 18), ([5, 0, 0, 7], 1), ([1 << 24], 148), ([4] * 148, 148), ([1] * 1024, 1),
               ([0] * 500 + [3] + [0] * 523, 148), ([1 << 18] * 1024, 148)]
    for _ in range(4000):
        n = int(rng.integers(1, 1025)) if rng.random() < 0.1 else int(rng.integers(1, 20))
        c = np.floor(np.exp(rng.uniform(0, np.log(rng.choice([3, 30, 3000])), n))).astype(int) * (rng.random(n) < rng.choice([0.3, 0.9, 1.0]))
        batches.append((c.tolist(), int(rng.choice([1, 2, 3, 9, 18, 37, 74, 148]))))
    joined = 0
    for chunks, ctas in batches:
        cs = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        rc = split(len(chunks), cs.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), ctas, ctypes.byref(got))
        assert rc == 0, (rc, chunks, ctas)
        joined += got.value < min(4 * ctas, int(cs[-1]))
    assert joined > 100                                                   # (some CTAs left one share for several warpgroups)


@pytest.mark.parametrize("scale", [1.0, 1e-4])
@pytest.mark.parametrize("tokens", [5, 40, 300])
def test_the_precision_bound_tells_a_share_of_11_bits_from_a_pair(tokens, scale):
    """The kernels' shares restated: 2^(logit - M) |v| / sqrt(128) * 2^13 as an fp16 pair stays inside the bound of the GPU
    tests, its high part alone does not, nor a fixed scale of 2 for small values. (The largest share of a row is a
    power of two, so one token alone would not show.)"""
    import torch
    rng = np.random.default_rng(tokens)
    code = kvq.kvq_codebook(4)[0].astype(np.float64)[rng.integers(0, 16, (tokens, 128))]
    norm = (scale * 11.3 * np.exp(0.1 * rng.standard_normal(tokens))).astype(np.float16).astype(np.float32)
    vn = norm * np.float32(1 / math.sqrt(128.0))
    k, v, q = rng.standard_normal((tokens, 128)), code * vn[:, None].astype(np.float64), np.zeros((3, 128))
    want, bound = rows_and_bound(k, v, q)

    def rows(parts, M, s):
        w = np.float32(2.0 ** -M)
        y = (vn * np.float32(s)) * w
        hi = y.astype(np.float16)
        lo = (y - hi.astype(np.float32)).astype(np.float16)
        share = hi.astype(np.float64) + (lo.astype(np.float64) if parts == 2 else 0.0)
        out = (share @ code) / s / (w.astype(np.float64) * tokens)
        return torch.from_numpy(np.repeat(out[None], 3, 0).astype(np.float32))
    top = float(np.log2(vn).max())
    check_close(rows(2, top, 8192.0), want, bound, torch.float32)
    with pytest.raises(AssertionError):
        check_close(rows(1, top, 8192.0), want, bound, torch.float32)
    if scale < 1e-3:
        with pytest.raises(AssertionError):
            check_close(rows(2, 0.0, 2.0), want, bound, torch.float32)
