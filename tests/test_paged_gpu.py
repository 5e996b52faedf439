"""Rotary positions, the paged append and the paged decode against plain forms on the CPU."""
import numpy as np
import pytest

from oracle import blockgtq as bg
from packed_cache_attention_b200 import kvq
from tests.paged_util import Paged, angle_table, check_rows, rotate_f32
from tests.parity_util import TOL, host_f32, rel_err

pytestmark = pytest.mark.gpu
ERR_RANGE = 5


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvq._check("kvq_init", kvq.lib().kvq_init())
    return torch.device("cuda:0")


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _axis(n):
    b = np.arange(64)
    return np.minimum((b + 8) // 24, 2) if n == 3 else b % n


def _desc(dev, table, pos, axis):
    import torch
    return kvq.rope_desc(torch.from_numpy(table).to(dev), torch.from_numpy(np.ascontiguousarray(pos, np.int32)).to(dev),
                         [int(a) for a in axis])


def _round(x, dtype):
    import torch
    return torch.from_numpy(x).to(dtype)


# ------------------------------------------------------------------------------ rope

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,heads,axes", [(1, 1, 1), (3, 5, 2), (33, 16, 3), (32, 2, 4), (200, 9, 1), (1500, 7, 3)])
def test_rope_is_the_formula_bit_for_bit(dev, dtype, tokens, heads, axes):
    import torch
    rng = np.random.default_rng(tokens + heads)
    table, axis = angle_table(3000), _axis(axes)
    pos = rng.integers(0, 3000, (axes, tokens))
    x = torch.randn((tokens, heads, 128), device=dev).to(_dt(dtype))
    before = x.clone()
    r = _desc(dev, table, pos, axis)
    want = _round(rotate_f32(host_f32(x), table, pos, axis), _dt(dtype))
    got = kvq.kvq_rope(x, r)
    assert torch.equal(got.cpu(), want) and torch.equal(x, before)
    assert kvq.kvq_rope(x, r, out=x) is x and torch.equal(x.cpu(), want)           # in place


def test_rope_strides_and_batches(dev):
    """The queries of a fused projection, rotated in place, and a batch with heads before tokens."""
    import torch
    table, axis = angle_table(64), _axis(2)
    rng = np.random.default_rng(0)
    pos = rng.integers(0, 64, (2, 21))
    r = _desc(dev, table, pos, axis)
    qkv = torch.randn((21, 8, 128), device=dev).to(torch.bfloat16)
    keep = qkv.clone()
    kvq.kvq_rope(qkv[:, :5], r, out=qkv[:, :5])
    assert torch.equal(qkv[:, 5:], keep[:, 5:])
    assert torch.equal(qkv[:, :5].cpu(), _round(rotate_f32(host_f32(keep[:, :5]), table, pos, axis), torch.bfloat16))
    x = torch.randn((3, 7, 4, 128), device=dev).transpose(1, 2)                     # [B][H][T][128], tokens first
    got = kvq.kvq_rope(x, r)
    rows = host_f32(x.transpose(1, 2)).reshape(21, 4, 128)
    want = rotate_f32(rows, table, pos, axis).reshape(3, 7, 4, 128)
    np.testing.assert_array_equal(host_f32(got.transpose(1, 2)), want)


def test_rope_outside_the_table_is_nan_in_its_blocks_alone(dev):
    import torch
    table, axis = angle_table(10), _axis(3)
    pos = np.tile(np.arange(6), (3, 1))
    pos[1, 2], pos[0, 4], pos[2, 5] = 10, -1, 2 ** 31 - 1
    x = torch.randn((6, 2, 128), device=dev)
    got = host_f32(kvq.kvq_rope(x, _desc(dev, table, pos, axis)))
    want = rotate_f32(host_f32(x), table, np.clip(pos, 0, 9), axis)
    bad = np.zeros((6, 2, 128), bool)
    for t, a in ((2, 1), (4, 0), (5, 2)):
        bad[t][:, np.tile(axis == a, 2)] = True
    assert np.isnan(got[bad]).all()
    np.testing.assert_array_equal(got[~bad], want[~bad])


def test_rope_offsets_past_32_bits(dev):
    """Rows 2^31 + 256 elements apart."""
    import torch
    big = torch.empty(2 ** 31 + 512, dtype=torch.bfloat16, device=dev)
    x = torch.as_strided(big, (2, 2, 128), (2 ** 31 + 256, 128, 1))
    x.normal_()
    table, axis = angle_table(8), _axis(1)
    pos = np.array([[3, 7]])
    want = _round(rotate_f32(host_f32(x), table, pos, axis), torch.bfloat16)
    kvq.kvq_rope(x, _desc(dev, table, pos, axis), out=x)
    assert torch.equal(x.cpu(), want)


# ------------------------------------------------------------------------------ append

def _expect_records(P, K, V, n):
    """Oracle records of one sequence's rows (host fp32 [n][hkv][128])."""
    k, v = (x.transpose(1, 0, 2)[None] for x in (K, V))
    return bg.pack_cache(bg.quantize(k, v, P.ref, P.bits_v), P.ref, P.bits_v, -(-n // 32) * 32)


@pytest.mark.parametrize("dtype,bits_k,bits_v,hkv,page,axes", [
    ("bf16", 3, 3, 2, 64, 1), ("f16", 4, 2, 3, 32, 3), ("f32", 2, 5, 1, 128, 0), ("bf16", 8, 8, 1, 256, 2), ("bf16", 1, 1, 8, 64, 4),
    ("f32", 5, 7, 2, 32, 1), ("f16", 2, 6, 2, 64, 0)])
def test_append_in_pieces_stores_the_oracles_bytes(dev, dtype, bits_k, bits_v, hkv, page, axes):
    """Ragged calls of 0, 1 and many tokens, starting in, at and before tile and page ends, leave the bytes
    that one quantization of the whole sequence gives, and touch no other byte."""
    import torch
    total = [131, 64, 1, 300, 0]
    P = Paged(dev, 7, hkv, bits_k, bits_v, page, total)
    n = sum(total)
    K, V = P.rows(n, _dt(dtype))
    starts = np.concatenate([[0], np.cumsum(total)])
    table = angle_table(2000)
    axis = _axis(max(axes, 1))
    pos = np.stack([np.concatenate([np.arange(t) * (a + 1) + 5 for t in total]) for a in range(max(axes, 1))])
    Kr = host_f32(K)
    if axes:
        Kr = host_f32(_round(rotate_f32(Kr, table, pos, axis), _dt(dtype)))
    before = P.pool.clone()
    done = [0] * len(total)
    for step in ([1, 0, 0, 31, 0], [31, 30, 0, 1, 0], [0, 2, 1, 97, 0], [1, 32, 0, 0, 0], [98, 0, 0, 171, 0]):
        rows = np.concatenate([np.arange(starts[b] + done[b], starts[b] + done[b] + m) for b, m in enumerate(step)]).astype(int)
        idx = torch.from_numpy(rows).to(dev)
        pad = torch.full((3, hkv, 128), float("nan"), device=dev, dtype=_dt(dtype))        # rows behind the last sequence
        kk, vv = torch.cat([K[idx], pad]), torch.cat([V[idx], pad])
        rope = _desc(dev, table, np.concatenate([pos[:, rows], np.full((len(pos), 3), -9)], 1), axis) if axes else None
        P.append(kk, vv, done, np.concatenate([[0], np.cumsum(step)]), rope=rope)
        done = [d + m for d, m in zip(done, step)]
    assert done == total and kvq.kvq_packed_status(P.pool) == 0
    used = np.zeros((P.desc.n_pages, page // 32), bool)
    for b, m in enumerate(total):
        if m == 0:
            continue
        tiles = -(-m // 32)
        got = P.records(P.table_np[b][:-(-m // page)])[:, :, :tiles]
        sl = slice(starts[b], starts[b + 1])
        np.testing.assert_array_equal(got, _expect_records(P, Kr[sl], host_f32(V)[sl], m))
        for t in range(tiles):
            used[P.table_np[b][t // (page // 32)], t % (page // 32)] = True
    shape = (P.desc.n_pages, hkv, page // 32, P.rec)
    a, b = (x[P.hdr:].cpu().numpy().reshape(shape).transpose(0, 2, 1, 3) for x in (before, P.pool))
    np.testing.assert_array_equal(a[~used], b[~used])
    assert torch.equal(before[:P.hdr], P.pool[:P.hdr])


def test_append_reads_strided_rows_of_a_projection(dev):
    import torch
    P = Paged(dev, 3, 2, 3, 3, 64, [50, 9])
    kv = torch.cat(P.rows(59, torch.bfloat16), 1)                                   # [59][4][128]
    P.append(kv[:, :2], kv[:, 2:], [0, 0], [0, 50, 59])
    for b, sl in enumerate((slice(0, 50), slice(50, 59))):
        n = sl.stop - sl.start
        want = _expect_records(P, host_f32(kv[sl, :2]), host_f32(kv[sl, 2:]), n)
        np.testing.assert_array_equal(P.records(P.table_np[b][:1])[:, :, :want.shape[2]], want)


def test_append_loses_what_does_not_fit_and_nothing_else(dev):
    """Rows out of order, more positions than the table holds, and a page outside the pool: their tiles are
    left as they were, the other sequences are stored, the status says RANGE, init clears it."""
    import torch
    lens = [0, 60, 0, 0, 0]
    P = Paged(dev, 11, 2, 3, 3, 64, [64, 64, 64, 64, 64])
    P.append(*P.rows(60, torch.bfloat16), [0] * 5, [0, 0, 60, 60, 60, 60])
    before = P.pool.clone()
    K, V = P.rows(200, torch.bfloat16)
    table = P.table.clone()
    table[2, 0] = P.desc.n_pages                                                    # outside the pool
    P.append(K, V, lens, [0, 10, 20, 30, 25, 95], table=table)                      # 1: 70 positions of 64, 3: descending, 4: 70 of 64
    assert kvq.kvq_packed_status(P.pool) == ERR_RANGE
    want = _expect_records(P, host_f32(K[:10]), host_f32(V[:10]), 10)
    np.testing.assert_array_equal(P.records(P.table_np[0][:1])[:, :, :1], want)
    body = slice(P.hdr, None)
    keep = torch.ones(P.desc.n_pages, dtype=torch.bool)
    keep[int(P.table_np[0][0])] = False
    per = lambda t: t[body].view(P.desc.n_pages, -1).cpu()[keep]  # noqa: E731
    assert torch.equal(per(before), per(P.pool))
    # the status stays, later appends still store, decodes report it and leave out as it was
    P.append(K[:5], V[:5], [10, 60, 0, 0, 0], [0, 5, 5, 5, 5, 5])
    want = _expect_records(P, host_f32(K)[[*range(10), *range(5)]], host_f32(V)[[*range(10), *range(5)]], 15)
    np.testing.assert_array_equal(P.records(P.table_np[0][:1])[:, :, :1], want)
    assert kvq.kvq_packed_status(P.pool) == ERR_RANGE
    q = torch.randn((5, 4, 128), device=dev)
    ws = kvq.kvq_paged_decode_workspace(P.desc, 5, 4)
    out = P.decode(q, [15, 60, 0, 0, 0], ws=ws, out=torch.full((5, 4, 128), 7.0, device=dev))
    assert kvq.kvq_workspace_status(ws) == ERR_RANGE and bool((out == 7.0).all())
    kvq.kvq_paged_init(P.alloc, P.desc, P.pool)
    assert kvq.kvq_packed_status(P.pool) == 0
    kvq.kvq_workspace_init(ws)
    got = P.decode(q, [15, 60, 0, 0, 0], ws=ws)
    assert kvq.kvq_workspace_status(ws) == 0
    check_rows(got, *P.attention(q, [15, 60, 0, 0, 0]), torch.float32)


def test_append_of_a_position_outside_the_table(dev):
    """Such a token has a NaN norm, so attention over it is NaN; the others are stored."""
    import torch
    P = Paged(dev, 13, 1, 3, 3, 64, [20, 20])
    K, V = P.rows(40, torch.bfloat16)
    pos = np.concatenate([np.arange(20), np.arange(20)])[None].copy()
    pos[0, 25] = 100
    P.append(K, V, [0, 0], [0, 20, 40], rope=_desc(dev, angle_table(100), pos, _axis(1)))
    assert kvq.kvq_packed_status(P.pool) == ERR_RANGE
    norms = P.records(P.table_np[1][:1])[0, 0, 0][4 * 128 * 3:4 * 128 * 3 + 64].copy().view("<f2")
    assert list(np.flatnonzero(np.isnan(norms))) == [5]
    kvq.kvq_paged_init(P.alloc, P.desc, P.pool)
    q = torch.randn((2, 2, 128), device=dev)
    got = P.decode(q, [20, 20])
    assert bool(got[1].isnan().all())
    check_rows(got[:1], *(x[:1] for x in P.attention(q, [20, 0])), torch.float32)


def test_a_call_with_another_allocation_or_shape_writes_nothing(dev):
    import torch
    P = Paged(dev, 17, 2, 3, 3, 64, [100])
    P.fill([100], torch.bfloat16)
    K, V = P.rows(10, torch.bfloat16)
    q = torch.randn((1, 8, 128), device=dev)
    other = Paged(dev, 18, 2, 3, 3, 64, [100]).alloc
    for alloc, desc in ((other, P.desc), (P.alloc, kvq.paged_desc(P.desc.n_pages // 2, 64, 2, 3, 3)),
                        (P.alloc, kvq.paged_desc(P.desc.n_pages, 32, 2, 3, 3)), (P.alloc, kvq.paged_desc(1, 64, 2, 2, 2))):
        pool = P.pool.clone()
        table, lens = torch.zeros((1, 4), dtype=torch.int32, device=dev), P.ints([0])
        kvq.kvq_paged_append(K, V, alloc, desc, table, lens, P.ints([0, 10]), pool)
        assert kvq.kvq_packed_status(pool) == kvq.KVQ_ERR_MISMATCH
        pool[12:16] = 0
        assert torch.equal(pool, P.pool)
        for prefix in (0, 30):
            ws = kvq.kvq_paged_decode_workspace(desc, 1, 8, prefix)
            out = kvq.kvq_paged_decode_attn(q, pool, alloc, desc, table, P.ints([20]), prefix_pages=P.ints([0]), prefix_len=prefix,
                                            ws=ws, out=torch.full((1, 8, 128), 7.0, device=dev))
            assert kvq.kvq_workspace_status(ws) == kvq.KVQ_ERR_MISMATCH and bool((out == 7.0).all())


@pytest.mark.parametrize("tokens", [3, 40])
def test_an_allocation_of_another_budget_is_reported_by_the_append(dev, tokens):
    """A pool of 3 bits set up with an allocation of 2, for all heads or for one: MISMATCH, no record written."""
    import torch
    P = Paged(dev, 19, 2, 3, 3, 64, [100])
    other = Paged(dev, 19, 2, 2, 3, 64, [100]).alloc
    K, V = P.rows(tokens, torch.bfloat16)
    for heads in (slice(0, 2), slice(0, 1), slice(1, 2)):
        alloc = P.alloc.clone().view(2, -1)
        alloc[heads] = other.view(2, -1)[heads]
        alloc = alloc.flatten()
        pool = P.pool.clone()
        kvq.kvq_paged_init(alloc, P.desc, pool)
        before = pool.clone()
        kvq.kvq_paged_append(K, V, alloc, P.desc, P.table, P.ints([0]), P.ints([0, tokens]), pool)
        assert kvq.kvq_packed_status(pool) == kvq.KVQ_ERR_MISMATCH
        assert torch.equal(before[P.hdr:], pool[P.hdr:])
        ws = kvq.kvq_paged_decode_workspace(P.desc, 1, 8)
        out = torch.full((1, 8, 128), 7.0, device=dev)
        kvq.kvq_paged_decode_attn(torch.randn((1, 8, 128), device=dev), pool, alloc, P.desc, P.table, P.ints([tokens]), ws=ws, out=out)
        assert kvq.kvq_workspace_status(ws) == kvq.KVQ_ERR_MISMATCH and bool((out == 7.0).all())


# ------------------------------------------------------------------------------ decode

LENS = [0, 1, 31, 33, 128, 129, 700, 0]


@pytest.mark.parametrize("hq,hkv,bits_k,bits_v,page,qt,ot", [
    (8, 1, 3, 3, 64, "bf16", "f32"), (4, 4, 4, 4, 32, "f16", "f16"), (14, 2, 2, 6, 128, "f32", "bf16"), (3, 1, 1, 1, 256, "bf16", "f32"),
    (6, 3, 8, 8, 64, "f16", "f32"), (2, 1, 5, 7, 32, "bf16", "bf16"), (8, 2, 3, 5, 512, "f32", "f32"), (1, 1, 4, 2, 64, "f16", "f16")])
def test_decode_of_a_ragged_batch(dev, hq, hkv, bits_k, bits_v, page, qt, ot):
    import torch
    P = Paged(dev, hq + bits_k, hkv, bits_k, bits_v, page, LENS)
    P.fill(LENS, torch.bfloat16)
    q = torch.randn((len(LENS), hq, 128), device=dev).to(_dt(qt))
    ws = kvq.kvq_paged_decode_workspace(P.desc, len(LENS), hq)
    got = P.decode(q, LENS, out_dtype=_dt(ot), ws=ws)
    assert kvq.kvq_workspace_status(ws) == 0 and bool((got[[0, 7]] == 0).all())
    check_rows(got, *P.attention(q, LENS), _dt(ot))
    assert torch.equal(got, P.decode(q, LENS, out_dtype=_dt(ot), ws=ws))            # the same bits again
    qs = torch.empty((len(LENS), 2 * hq, 136), device=dev, dtype=_dt(qt))[:, ::2, :128]
    qs.copy_(q)
    assert torch.equal(got, P.decode(qs, LENS, out_dtype=_dt(ot), ws=ws))           # strided queries


@pytest.mark.parametrize("batch,hkv,longest", [(1, 1, 9000), (200, 1, 300), (40, 8, 260), (3, 2, 6000), (1, 1, 1), (1024, 1, 40)])
def test_decode_splits(dev, batch, hkv, longest):
    """Few long sequences (many splits each) and more sequences than SMs (one each or less)."""
    import torch
    rng = np.random.default_rng(batch)
    lens = [longest] + [int(x) for x in rng.integers(0, longest + 1, batch - 1)]
    P = Paged(dev, batch, hkv, 2, 2, 64, lens)
    P.fill(lens, torch.bfloat16)
    q = torch.randn((batch, 2 * hkv, 128), device=dev)
    got = P.decode(q, lens)
    rows = sorted({0, batch - 1, batch // 2, int(np.argmin(lens)), *rng.integers(0, batch, 3).tolist()})
    sub = Paged.__new__(Paged)
    sub.__dict__.update(P.__dict__)
    sub.table_np = P.table_np[rows]
    check_rows(got[rows], *sub.attention(q[rows], [lens[b] for b in rows]), torch.float32)


@pytest.mark.parametrize("batch,hq,hkv,prefix,bits_k,bits_v,page,ot", [
    (1, 1, 1, 1, 3, 3, 32, "f32"), (4, 8, 1, 31, 4, 4, 64, "f32"), (5, 14, 2, 127, 2, 5, 32, "f16"), (8, 16, 2, 128, 3, 3, 128, "f32"),
    (9, 8, 1, 129, 8, 8, 64, "bf16"), (13, 7, 1, 300, 1, 1, 64, "f32"), (16, 8, 1, 1000, 3, 2, 64, "f32"), (33, 8, 1, 777, 2, 7, 32, "f32"),
    (3, 24, 8, 2500, 4, 6, 256, "f32"), (2, 2, 2, 5000, 5, 3, 64, "f32"), (17, 8, 1, 600, 3, 3, 64, "bf16"), (24, 12, 2, 1300, 2, 4, 128, "bf16")])
def test_decode_behind_a_shared_prefix(dev, batch, hq, hkv, prefix, bits_k, bits_v, page, ot):
    import torch
    lens = ([0, 1, 40, 129, 64] * 7)[:batch]
    P = Paged(dev, prefix, hkv, bits_k, bits_v, page, lens, prefix=prefix)
    P.fill(lens, torch.bfloat16, prefix=prefix)
    q = torch.randn((batch, hq, 128), device=dev).to(torch.bfloat16)
    ws = kvq.kvq_paged_decode_workspace(P.desc, batch, hq, prefix)
    got = P.decode(q, lens, prefix, out_dtype=_dt(ot), ws=ws)
    assert kvq.kvq_workspace_status(ws) == 0
    check_rows(got, *P.attention(q, lens, prefix, _dt(ot)), _dt(ot))
    assert torch.equal(got, P.decode(q, lens, prefix, out_dtype=_dt(ot), ws=ws))


@pytest.mark.parametrize("batch,hq,hkv,bits_k,bits_v", [(1, 16, 16, 8, 8), (1, 32, 16, 1, 8), (5, 64, 8, 6, 8), (3, 64, 8, 8, 3)])
def test_a_prefix_whose_values_are_ready_late(dev, batch, hq, hkv, bits_k, bits_v):
    """Warps without query rows are done with a chunk's softmax at once, while its values (wide, one stage of
    copies) are still looked up: the products wait for them, and every call gives the same bits."""
    import torch
    prefix, lens = 9000, [3] * batch                                                # 4 to 8 chunks a CTA
    P = Paged(dev, 40 + bits_v, hkv, bits_k, bits_v, 256, lens, prefix=prefix)
    P.fill(lens, torch.bfloat16, prefix=prefix)
    q = torch.randn((batch, hq, 128), device=dev).to(torch.bfloat16)
    ws = kvq.kvq_paged_decode_workspace(P.desc, batch, hq, prefix)
    got = P.decode(q, lens, prefix, ws=ws)
    check_rows(got, *P.attention(q, lens, prefix), torch.float32)
    for _ in range(50):
        assert torch.equal(got, P.decode(q, lens, prefix, ws=ws))
    assert kvq.kvq_workspace_status(ws) == 0


@pytest.mark.parametrize("batch,hq,hkv,prefix,bits_k,bits_v", [(9, 8, 1, 129, 3, 3), (64, 16, 2, 3000, 3, 3), (5, 14, 2, 1000, 8, 8),
                                                              (4, 4, 1, 0, 4, 4)])
def test_16_bit_outputs_are_the_fp32_ones_rounded(dev, batch, hq, hkv, prefix, bits_k, bits_v):
    """The output's type changes its rounding alone, not what is computed."""
    import torch
    lens = ([0, 1, 40, 129, 64, 300] * 11)[:batch]
    P = Paged(dev, 50 + batch, hkv, bits_k, bits_v, 64, lens, prefix=prefix)
    P.fill(lens, torch.bfloat16, prefix=prefix)
    q = torch.randn((batch, hq, 128), device=dev).to(torch.bfloat16)
    want = P.decode(q, lens, prefix)
    for dt in (torch.bfloat16, torch.float16):
        assert torch.equal(P.decode(q, lens, prefix, out_dtype=dt), want.to(dt))


def test_a_logit_far_above_the_rest_and_rows_of_zeros(dev):
    """Keys that grow along the prefix move the running maximum in every chunk; one row's query is zero,
    one huge, one tiny."""
    import torch
    P = Paged(dev, 5, 1, 4, 4, 64, [200, 200, 200, 200], prefix=900)
    K, V = P.rows(900, torch.float32)
    K *= torch.linspace(0.01, 3.0, 900, device=dev)[:, None, None]
    P.append(K, V, [0], [0, 900], table=P.prefix_pages[None].contiguous())
    P.fill([200] * 4, torch.float32)
    q = torch.randn((4, 8, 128), device=dev)
    q[1] = 0.0
    q[2] *= 30.0
    q[3] *= 1e-30
    for prefix in (0, 900):
        check_rows(P.decode(q, [200] * 4, prefix), *P.attention(q, [200] * 4, prefix), torch.float32)
    tiny = torch.full((4, 8, 128), 1e-42, device=dev)
    for prefix in (0, 900):
        check_rows(P.decode(tiny, [200] * 4, prefix), *P.attention(tiny, [200] * 4, prefix), torch.float32)


def test_a_nan_query_row_stays_in_its_row(dev):
    import torch
    lens = [100, 300, 40, 0]
    P = Paged(dev, 6, 1, 3, 3, 64, lens, prefix=200)
    P.fill(lens, torch.bfloat16, prefix=200)
    q = torch.randn((4, 8, 128), device=dev)
    clean = q.clone()
    q[1, 3, 7] = float("nan")
    q[2, 0, :] = float("inf")
    for prefix in (0, 200):
        got, want = P.decode(q, lens, prefix), P.decode(clean, lens, prefix)
        bad = torch.zeros((4, 8), dtype=torch.bool, device=dev)
        bad[1, 3] = bad[2, 0] = True
        assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], want[~bad])


def test_more_kv_heads_than_sms(dev):
    """One CTA per head and more than one wave of them, own pages and prefix."""
    import torch
    lens = [40, 0, 130]
    P = Paged(dev, 12, 160, 1, 1, 32, lens, prefix=70, profile_tokens=40)
    P.fill(lens, torch.bfloat16, prefix=70)
    q = torch.randn((3, 160, 128), device=dev)
    for prefix in (0, 70):
        check_rows(P.decode(q, lens, prefix), *P.attention(q, lens, prefix), torch.float32)


def test_one_heads_allocation_swapped(dev):
    """A call whose allocation differs for one KV head reports it and leaves that head's rows; the others are right."""
    import torch
    lens = [300, 90]
    P = Paged(dev, 14, 2, 3, 3, 64, lens, prefix=200)
    P.fill(lens, torch.bfloat16, prefix=200)
    other = Paged(dev, 15, 2, 3, 3, 64, lens).alloc
    alloc = P.alloc.clone()
    alloc[2048:] = other[2048:]
    q = torch.randn((2, 8, 128), device=dev)
    for prefix in (0, 200):
        ws = kvq.kvq_paged_decode_workspace(P.desc, 2, 8, prefix)
        out = torch.full((2, 8, 128), 7.0, device=dev)
        kvq.kvq_paged_decode_attn(q, P.pool, alloc, P.desc, P.table, P.ints(lens), prefix_pages=P.prefix_pages, prefix_len=prefix,
                                  ws=ws, out=out)
        assert kvq.kvq_workspace_status(ws) == kvq.KVQ_ERR_MISMATCH and bool((out[:, 4:] == 7.0).all())
        want, bound = P.attention(q, lens, prefix)
        check_rows(out[:, :4], want[:, :4], bound[:, :4], torch.float32)


@pytest.mark.parametrize("batch,head", [(3, 0), (3, 1), (700, 0), (700, 1), (700, None)])
def test_a_refused_head_keeps_its_rows_and_no_others(dev, batch, head):
    """Whichever head's allocation differs (None: the pool's shape), its rows stay as they were, those of empty
    sequences and of the batch's end too; the other head's are right."""
    import torch
    lens = ([40, 0, 130] * 234)[:batch]
    P = Paged(dev, 24, 2, 3, 3, 64, lens, prefix=70)
    P.fill(lens, torch.bfloat16, prefix=70)
    other = Paged(dev, 15, 2, 3, 3, 64, [64]).alloc
    alloc = P.alloc.clone().view(2, -1)
    desc = P.desc
    if head is None:
        desc = kvq.paged_desc(P.desc.n_pages - 1, 64, 2, 3, 3)
    else:
        alloc[head] = other.view(2, -1)[head]
    q = torch.randn((batch, 4, 128), device=dev)
    for prefix in (0, 70):
        want = P.decode(q, lens, prefix)
        ws = kvq.kvq_paged_decode_workspace(desc, batch, 4, prefix)
        out = torch.full((batch, 4, 128), 7.0, device=dev)
        kvq.kvq_paged_decode_attn(q, P.pool, alloc.flatten(), desc, P.table, P.ints(lens), prefix_pages=P.prefix_pages,
                                  prefix_len=prefix, ws=ws, out=out)
        assert kvq.kvq_workspace_status(ws) == kvq.KVQ_ERR_MISMATCH
        for h in range(2):
            rows = slice(2 * h, 2 * h + 2)
            if head is None or h == head:
                assert bool((out[:, rows] == 7.0).all())
            else:
                assert torch.equal(out[:, rows], want[:, rows])
        kvq.kvq_workspace_init(ws)
        again = kvq.kvq_paged_decode_attn(q, P.pool, P.alloc, P.desc, P.table, P.ints(lens), prefix_pages=P.prefix_pages, prefix_len=prefix, ws=ws)
        assert torch.equal(again, want) and kvq.kvq_workspace_status(ws) == 0


def test_the_largest_batch_behind_a_prefix(dev):
    """1024 sequences of 8 heads: 64 groups of rows on the prefix, more CTAs than SMs."""
    import torch
    lens = ([0, 3, 140, 33] * 256)[:1024]
    P = Paged(dev, 26, 3, 2, 3, 32, lens, prefix=300)
    P.fill(lens, torch.bfloat16, prefix=300)
    q = torch.randn((1024, 24, 128), device=dev)
    got = P.decode(q, lens, 300)
    rows = [0, 1, 15, 16, 17, 511, 514, 1022, 1023]
    sub = Paged.__new__(Paged)
    sub.__dict__.update(P.__dict__)
    sub.table_np = P.table_np[rows]
    check_rows(got[rows], *sub.attention(q[rows], [lens[b] for b in rows], 300), torch.float32)


def test_the_largest_page(dev):
    """Pages of 65536 positions, one of them entered by four tokens."""
    import torch
    lens = [65540, 7]
    P = Paged(dev, 27, 1, 1, 2, 65536, lens, prefix=33)
    P.fill(lens, torch.float16, prefix=33)
    q = torch.randn((2, 2, 128), device=dev).half()
    for prefix in (0, 33):
        check_rows(P.decode(q, lens, prefix), *P.attention(q, lens, prefix), torch.float32)


def test_one_query_and_one_sequence_for_many_rows(dev):
    """Rows that share a query (stride 0), a sequence or its first pages as the prefix, and an output over the queries."""
    import torch
    P = Paged(dev, 28, 2, 3, 3, 64, [300, 128], prefix=0)
    P.fill([300, 128], torch.bfloat16)
    q = torch.randn((1, 8, 128), device=dev)
    table = P.table[[0, 0, 1, 0, 1]].contiguous()
    lens = [300, 120, 128, 300, 0]
    call = lambda q, **kw: kvq.kvq_paged_decode_attn(q, P.pool, P.alloc, P.desc, table, P.ints(lens), **kw)  # noqa: E731
    got = call(q.expand(5, 8, 128))
    sub = Paged.__new__(Paged)
    sub.__dict__.update(P.__dict__)
    sub.table_np = P.table_np[[0, 0, 1, 0, 1]]
    check_rows(got, *sub.attention(q.expand(5, 8, 128), lens), torch.float32)
    assert torch.equal(got[0], got[3])
    same = q.repeat(5, 1, 1)
    assert call(same, out=same) is same and torch.equal(same, got)
    lead = call(q.expand(5, 8, 128), prefix_pages=P.table[0, :2].contiguous(), prefix_len=100)
    sub.prefix_np = P.table_np[0, :2]
    check_rows(lead, *sub.attention(q.expand(5, 8, 128), lens, 100), torch.float32)
    same = q.repeat(5, 1, 1)
    call(same, prefix_pages=P.table[0, :2].contiguous(), prefix_len=100, out=same)
    assert torch.equal(same, lead)


def test_two_graphs_share_a_workspace(dev):
    """Two captured decodes of different batches on one workspace, replayed in turn on one stream, with eager calls
    between them."""
    import torch
    lens = [400, 0, 77, 129, 1, 300]
    P = Paged(dev, 29, 1, 4, 4, 64, lens, prefix=260)
    P.fill(lens, torch.bfloat16, prefix=260)
    q = torch.randn((6, 8, 128), device=dev)
    ws = kvq.kvq_paged_decode_workspace(P.desc, 6, 8, 260)
    want = [P.decode(q, lens, 260), P.decode(q, lens)]
    outs, n = [torch.empty_like(q) for _ in range(2)], P.ints(lens)
    call = lambda i: kvq.kvq_paged_decode_attn(  # noqa: E731
        q if i == 0 else q[:4], P.pool, P.alloc, P.desc, P.table if i == 0 else P.table[:4], n if i == 0 else n[:4],
        prefix_pages=P.prefix_pages if i == 0 else None, prefix_len=260 if i == 0 else 0, ws=ws, out=outs[i] if i == 0 else outs[i][:4])
    side = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g, stream=side):
            call(i)
    with torch.cuda.stream(side):
        for r in range(30):
            for o in outs:
                o.fill_(float(r))
            graphs[r % 2].replay()
            if r % 3 == 0:
                call((r + 1) % 2)
            else:
                graphs[(r + 1) % 2].replay()
            side.synchronize()
            assert torch.equal(outs[0], want[0]) and torch.equal(outs[1][:4], want[1][:4]) and bool((outs[1][4:] == r).all())
    assert kvq.kvq_workspace_status(ws) == 0


def test_calls_on_a_given_stream_without_buffers(dev):
    """Outputs and workspaces that a call makes belong to the stream it was given."""
    import torch
    lens = [200, 33]
    P = Paged(dev, 16, 2, 3, 3, 64, lens, prefix=150)
    P.fill(lens, torch.bfloat16, prefix=150)
    q = torch.randn((2, 8, 128), device=dev)
    r = _desc(dev, angle_table(16), np.arange(2)[None], _axis(1))
    want = [P.decode(q, lens, p) for p in (0, 150)] + [kvq.kvq_rope(q, r)]
    ln = P.ints(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        torch.empty(1 << 24, dtype=torch.uint8, device=dev).fill_(255)          # memory that the next call may be given
        got = [kvq.kvq_paged_decode_attn(q, P.pool, P.alloc, P.desc, P.table, ln, prefix_pages=P.prefix_pages, prefix_len=p, stream=side)
               for p in (0, 150)] + [kvq.kvq_rope(q, r, stream=side)]
    side.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_calls_that_overlap_on_two_streams(dev):
    """Two batches over one pool, decoded and extended at once with a workspace each."""
    import torch
    lens = [260, 31, 500, 64]
    P = Paged(dev, 17, 1, 4, 4, 64, [n + 40 for n in lens])
    P.fill(lens, torch.bfloat16)
    q = torch.randn((4, 8, 128), device=dev)
    K, V = P.rows(40, torch.bfloat16)
    halves = [slice(0, 2), slice(2, 4)]
    streams = [torch.cuda.Stream() for _ in halves]
    tabs, ws = [P.table[h].contiguous() for h in halves], [kvq.kvq_paged_decode_workspace(P.desc, 2, 8) for _ in halves]
    l0, l1, cu = [P.ints(lens[h]) for h in halves], [P.ints([n + 10 for n in lens[h]]) for h in halves], P.ints([0, 10, 20])
    qs, outs = [q[h].contiguous() for h in halves], [torch.empty((2, 8, 128), device=dev) for _ in halves]
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        kvq.kvq_paged_append(K[20 * i:20 * i + 20], V[20 * i:20 * i + 20], P.alloc, P.desc, tabs[i], l0[i], cu, P.pool, stream=s)
    for _ in range(10):
        for i, s in enumerate(streams):
            kvq.kvq_paged_decode_attn(qs[i], P.pool, P.alloc, P.desc, tabs[i], l1[i], out=outs[i], ws=ws[i], stream=s)
    torch.cuda.synchronize()
    assert kvq.kvq_packed_status(P.pool) == 0 and all(kvq.kvq_workspace_status(w) == 0 for w in ws)
    n = [x + 10 for x in lens]
    check_rows(torch.cat(outs), *P.attention(q, n), torch.float32)


@pytest.mark.parametrize("dtype,bits_k,bits_v", [("bf16", 4, 4), ("f16", 3, 7), ("f32", 2, 5), ("bf16", 8, 1), ("f16", 1, 8)])
def test_tokens_one_by_one_equal_tiles_at_once(dev, dtype, bits_k, bits_v):
    """One to four tokens a call (rows) and five or more (tiles) leave the same bytes, whatever the order of both."""
    import torch
    P = Paged(dev, 18, 2, bits_k, bits_v, 64, [130, 130, 130])
    K, V = P.rows(130, _dt(dtype))
    K[17] = 0.0                                                                  # a zero row: norm 0, codes at y = 0
    V[18] = 0.0
    K[19] *= 1e-6
    pos = np.arange(130)[None] * 3
    table = angle_table(400)
    for b, steps in enumerate(([130], [1] * 130, [4, 1, 5, 2, 30, 3, 1, 33, 4, 31, 16])):
        done = 0
        for n in steps:
            sl = slice(done, done + n)
            P.append(K[sl], V[sl], [done], [0, n], table=P.table[b:b + 1].contiguous(), rope=_desc(dev, table, pos[:, sl], _axis(1)))
            done += n
        assert done == 130
    got = [P.records(P.table_np[b])[:, :, :5] for b in range(3)]
    np.testing.assert_array_equal(got[0], got[1])
    np.testing.assert_array_equal(got[0], got[2])


def test_decode_errors_leave_their_rows(dev):
    """A page outside the pool, a negative length and one past the table: RANGE, those rows as they were."""
    import torch
    lens = [100, 300, 40, 70]
    P = Paged(dev, 8, 2, 3, 3, 64, lens, prefix=130)
    P.fill(lens, torch.bfloat16, prefix=130)
    q = torch.randn((4, 8, 128), device=dev)
    for prefix in (0, 130):
        want = P.decode(q, lens, prefix)
        for kind in ("page", "negative", "long", "prefix"):
            if kind == "prefix" and not prefix:
                continue
            table, ln, pages = P.table.clone(), list(lens), P.prefix_pages.clone()
            if kind == "page":
                table[1, 3] = -1
            elif kind == "negative":
                ln[1] = -5
            elif kind == "long":
                ln[1] = P.table_np.shape[1] * 64 + 1
            else:
                pages[1] = P.desc.n_pages
            ws = kvq.kvq_paged_decode_workspace(P.desc, 4, 8, prefix)
            out = torch.full((4, 8, 128), 7.0, device=dev)
            kvq.kvq_paged_decode_attn(q, P.pool, P.alloc, P.desc, table, P.ints(ln), prefix_pages=pages, prefix_len=prefix, ws=ws, out=out)
            assert kvq.kvq_workspace_status(ws) == ERR_RANGE, kind
            if kind == "prefix":
                assert bool((out == 7.0).all())
            else:
                assert bool((out[1] == 7.0).all())
                rest = [0, 2, 3]
                check_rows(out[rest], host_f32(want[rest]).astype(np.float64), P.attention(q, lens, prefix)[1][rest], torch.float32)
            kvq.kvq_workspace_init(ws)
            check_rows(P.decode(q, lens, prefix, ws=ws), *P.attention(q, lens, prefix), torch.float32)
            assert kvq.kvq_workspace_status(ws) == 0


def test_a_wait_that_runs_out_is_reported(dev):
    import torch
    lens = [100, 500]
    P = Paged(dev, 9, 1, 3, 3, 64, lens, prefix=600)
    P.fill(lens, torch.bfloat16, prefix=600)
    q = torch.randn((2, 8, 128), device=dev)
    for prefix in (0, 600):
        want = P.decode(q, lens, prefix)
        ws = kvq.kvq_paged_decode_workspace(P.desc, 2, 8, prefix)
        try:
            kvq.kvq_debug_decode(20, True)
            out = P.decode(q, lens, prefix, ws=ws, out=torch.full((2, 8, 128), 7.0, device=dev))
            assert kvq.kvq_workspace_status(ws) == kvq.KVQ_ERR_TIMEOUT
        finally:
            kvq.kvq_debug_decode()
        assert bool((out == 7.0).all())
        kvq.kvq_workspace_init(ws)
        assert torch.equal(P.decode(q, lens, prefix, ws=ws), want) and kvq.kvq_workspace_status(ws) == 0


def test_a_pool_past_4_gib(dev):
    """Pages whose byte offsets do not fit 32 bits."""
    import torch
    P = Paged(dev, 10, 8, 8, 8, 256, [300, 40], prefix=100, spare=8100)
    assert P.pool.numel() > 2 ** 32
    high = np.sort(np.concatenate([P.unused, P.table_np[P.table_np >= 0], P.prefix_np]))[::-1]
    P.table_np[0, :2], P.table_np[1, 0], P.prefix_np[0] = high[:2], high[2], high[3]
    P.table, P.prefix_pages = P.ints(P.table_np), P.ints(P.prefix_np)
    lens = [300, 40]
    P.fill(lens, torch.bfloat16, prefix=100)
    small = Paged.__new__(Paged)
    small.__dict__.update(P.__dict__)
    per = P.hkv * 8 * P.rec
    take = lambda p: P.pool[P.hdr + int(p) * per:P.hdr + (int(p) + 1) * per].cpu().numpy().reshape(P.hkv, 8, P.rec)  # noqa: E731
    small.records = lambda pages: np.concatenate([take(p) for p in pages], 1)[None]
    q = torch.randn((2, 16, 128), device=dev)
    for prefix in (0, 100):
        check_rows(P.decode(q, lens, prefix), *small.attention(q, lens, prefix), torch.float32)


# ------------------------------------------------------------------------------ together

def test_serving_steps_captured_in_a_graph(dev):
    """A prompt shared by the batch, then steps of rotate, append, attend: eager on one stream, and captured once
    and replayed with new inputs and lengths in place, on another; both agree with the plain forms."""
    import torch
    hq, hkv, B, prefix, steps = 8, 2, 3, 70, 40
    start = [5, 0, 63]
    ends = [s + steps for s in start]
    table = angle_table(400)
    axis = _axis(3)
    results = []
    for mode in ("eager", "graph"):
        P = Paged(dev, 21, hkv, 3, 3, 64, ends, prefix=prefix)
        dt = torch.bfloat16
        K, V = P.rows(prefix, dt)
        P.append(K, V, [0], [0, prefix], table=P.prefix_pages[None].contiguous(),
                 rope=_desc(dev, table, np.tile(np.arange(prefix), (3, 1)), axis))
        P.append(*P.rows(sum(start), dt), [0] * B, np.concatenate([[0], np.cumsum(start)]))
        lens, cu = P.ints(start), P.ints(range(B + 1))
        pos = torch.zeros((3, B), dtype=torch.int32, device=dev)
        q, k, v = (torch.zeros((B, h, 128), dtype=dt, device=dev) for h in (hq, hkv, hkv))
        qr, out = torch.empty_like(q), torch.empty((B, hq, 128), device=dev)
        ws = kvq.kvq_paged_decode_workspace(P.desc, B, hq, prefix)
        rope = kvq.rope_desc(torch.from_numpy(table).to(dev), pos, [int(a) for a in axis])
        now = P.ints([0] * B)

        def step():
            kvq.kvq_rope(q, rope, out=qr)
            kvq.kvq_paged_append(k, v, P.alloc, P.desc, P.table, lens, cu, P.pool, rope=rope)
            torch.add(lens, 1, out=now)
            kvq.kvq_paged_decode_attn(qr, P.pool, P.alloc, P.desc, P.table, now, prefix_pages=P.prefix_pages, prefix_len=prefix,
                                      out=out, ws=ws)
            lens.add_(1)

        gen = torch.Generator(device=dev).manual_seed(4)
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        if mode == "graph":
            saved = P.pool.clone()
            with torch.cuda.stream(side):
                step()                                     # (sets up the kernels before the capture)
            torch.cuda.synchronize()
            P.pool.copy_(saved)
            lens.copy_(P.ints(start))
            with torch.cuda.graph(graph, stream=side):
                step()
        outs = []
        for i in range(steps):
            for t in (q, k, v):
                t.copy_(torch.randn(t.shape, generator=gen, device=dev))
            pos.copy_(prefix + lens.long()[None] // torch.tensor([1, 2, 3], device=dev)[:, None])
            torch.cuda.synchronize()
            if mode == "graph":
                graph.replay()
            else:
                with torch.cuda.stream(side):
                    step()
            torch.cuda.synchronize()
            outs.append(out.clone())
            if i in (0, 1, steps - 1):
                n = [s + i + 1 for s in start]
                assert lens.tolist() == n
                want_q = _round(rotate_f32(host_f32(q), table, pos.cpu().numpy(), axis), dt)
                assert torch.equal(qr.cpu(), want_q)
                check_rows(out, *P.attention(qr, n, prefix), torch.float32)
        assert kvq.kvq_workspace_status(ws) == 0 and kvq.kvq_packed_status(P.pool) == 0
        results.append(torch.stack(outs))
    assert torch.equal(results[0], results[1])


def test_a_paged_cache_answers_as_a_contiguous_one(dev):
    """The same tokens quantized into a contiguous cache and appended to pages: the same records, and the two
    decodes agree within both kernels' bounds."""
    import torch
    n = 700
    P = Paged(dev, 23, 2, 3, 3, 64, [n, n])
    K, V = P.rows(2 * n, torch.bfloat16)
    P.append(K, V, [0, 0], [0, n, 2 * n])
    kc, vc = (x.view(2, n, 2, 128).transpose(1, 2).contiguous() for x in (K, V))
    cache = kvq.cache_desc(2, 2, n, 3, 3)
    packed = kvq.kvq_quantize(kc, vc, P.alloc, cache)
    tiles = -(-n // 32)
    want = packed[P.hdr:].cpu().numpy().reshape(2, 2, tiles, P.rec)
    for b in range(2):
        np.testing.assert_array_equal(P.records(P.table_np[b])[0][:, :tiles], want[b])
    q = torch.randn((2, 16, 128), device=dev).to(torch.bfloat16)
    ref, bound = P.attention(q, [n, n])
    check_rows(P.decode(q, [n, n]), ref, bound, torch.float32)
    check_rows(kvq.kvq_decode_attn(q, packed, P.alloc, cache, n), ref, bound, torch.float32)


@pytest.mark.parametrize("seed", range(6))
def test_long_contexts_agree_with_the_contiguous_decode(dev, seed):
    """More chunks per warpgroup than copies in flight; each kernel is within its tolerance of the exact rows."""
    import torch
    n = 60000 + 117 * seed
    P = Paged(dev, 30 + seed, 2, 3, 3, 256, [n], prefix=256 * 100)
    K, V = P.rows(n, torch.bfloat16)
    P.append(K, V, [0], [0, n])
    cache = kvq.cache_desc(1, 2, n, 3, 3)
    packed = kvq.kvq_quantize(*(x.transpose(0, 1)[None].contiguous() for x in (K, V)), P.alloc, cache)
    q = torch.randn((1, 16, 128), device=dev).to(torch.bfloat16)
    want = host_f32(kvq.kvq_decode_attn(q, packed, P.alloc, cache, n))
    assert rel_err(host_f32(P.decode(q, [n])), want) <= 2 * TOL
    # the first 100 pages as a shared prefix, the others as the sequence's own
    lead = P.table[0, :100].contiguous()
    got = kvq.kvq_paged_decode_attn(q, P.pool, P.alloc, P.desc, P.table[:, 100:].contiguous(), P.ints([n - 25600]), prefix_pages=lead,
                                    prefix_len=25600)
    assert rel_err(host_f32(got), want) <= 2 * TOL


def test_binding_refuses_mixed_arguments(dev):
    import torch
    P = Paged(dev, 25, 2, 3, 3, 64, [64, 64])
    q = torch.zeros((2, 8, 128), device=dev)
    with pytest.raises(ValueError):
        P.decode(q.cpu(), [1, 1])
    with pytest.raises(ValueError):
        P.decode(q, [1, 1, 1])                                            # another batch
    with pytest.raises(kvq.KvqError):
        P.decode(q[:1], [1, 1])
    with pytest.raises(ValueError):
        P.decode(q, [1, 1], out=torch.zeros((2, 8, 128), device=dev, dtype=torch.float16), out_dtype=torch.float32)
    with pytest.raises(ValueError):
        P.decode(q.double(), [1, 1])
    with pytest.raises(ValueError):
        kvq.kvq_paged_decode_attn(q, P.pool[:-1], P.alloc, P.desc, P.table, P.ints([1, 1]))
    with pytest.raises(ValueError):
        kvq.kvq_paged_decode_attn(q, P.pool, P.alloc, P.desc, P.table, P.ints([1, 1]), prefix_len=3)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_paged_decode_attn(q, P.pool, P.alloc, P.desc, P.table, P.ints([1, 1]), prefix_pages=P.ints([0]), prefix_len=65)
    K, V = P.rows(4, torch.bfloat16)
    with pytest.raises(ValueError):
        P.append(K, V, [0, 0], [0, 4])                                    # cu_tokens of another batch
    with pytest.raises(ValueError):
        P.append(K, V, [0, 0], [0, 2, 4], rope=_desc(dev, angle_table(4), np.zeros((1, 3)), _axis(1)))
    with pytest.raises(kvq.KvqError):
        P.append(K, V[:3], [0, 0], [0, 2, 4])
