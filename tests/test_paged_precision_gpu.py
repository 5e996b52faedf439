"""Paged attention against rows in 64 bits where a fixed scale would lose digits: small and mixed value
norms, values of zero, queries with one coordinate far above the rest."""
import math

import numpy as np
import pytest

from packed_cache_attention_b200 import kvq
from tests.paged_util import Paged, check_close as check, rows_and_bound
from tests.parity_util import host_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvq._check("kvq_init", kvq.lib().kvq_init())
    return torch.device("cuda:0")


def exact_rows(P, q, lens, prefix):
    """Rows in 64 bits of q [B][Hq][128] and the bound of an fp32 kernel's error (paged_util.rows_and_bound)."""
    q = host_f32(q).astype(np.float64)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    pk, pv = P.kv(P.prefix_np, prefix)
    for b, n in enumerate(lens):
        k, v = P.kv(P.table_np[b], n)
        k, v = np.concatenate([pk, k], 1)[0], np.concatenate([pv, v], 1)[0]
        if len(k):
            out[b], bound[b] = rows_and_bound(k, v, q[b])
    return out, bound


def _pool(dev, seed, bits_k, bits_v, lens, prefix, scale_of):
    """A pool whose token i of a sequence (or of the prefix) has values of scale scale_of(rng, tokens)[i]."""
    import torch
    P = Paged(dev, seed, 1, bits_k, bits_v, 64, lens, prefix=prefix)
    keys = []
    for n, table in [(prefix, P.prefix_pages[None].contiguous())] + [(n, P.table[b:b + 1].contiguous()) for b, n in enumerate(lens)]:
        if n == 0:
            keys.append(None)
            continue
        K, V = P.rows(n, torch.float32)
        V = V * torch.from_numpy(scale_of(P.rng, n)).float().to(dev)[:, None, None]
        P.append(K, V, [0], [0, n], table=table)
        keys.append((K, V))
    assert kvq.kvq_packed_status(P.pool) == 0
    return P, keys


@pytest.mark.parametrize("bits_k,bits_v,heads", [(3, 3, 8), (4, 8, 3), (8, 2, 4)])
@pytest.mark.parametrize("scale", [1e3, 1.0, 1e-3, 1e-5, 2e-7])
def test_outputs_do_not_depend_on_the_scale_of_the_values(dev, bits_k, bits_v, heads, scale):
    """Equal logits (a zero query) and small ones, values of one scale: own pages, a prefix, both."""
    import torch
    lens, prefix = [2000, 1, 130], 4001
    P, _ = _pool(dev, 60 + bits_v, bits_k, bits_v, lens, prefix, lambda rng, n: np.full(n, scale))
    q = torch.randn((3, heads, 128), device=dev) * 0.02
    q[0] = 0.0
    for pre in (0, prefix):
        want, bound = exact_rows(P, q, lens, pre)
        for dt in (torch.float32, torch.bfloat16, torch.float16):
            if dt == torch.float16 and scale == 1e3 and np.abs(want).max() > 6e4:
                continue
            check(P.decode(q, lens, pre, out_dtype=dt), want, bound, dt)


@pytest.mark.parametrize("scale", [1.0, 1e-4])
@pytest.mark.parametrize("tokens", [1, 2, 5, 40])
def test_few_tokens_of_equal_weight(dev, tokens, scale):
    """A mean of few values, of own pages or of a prefix: shares of 11 bits would show."""
    import torch
    lens = [tokens] * 4
    P, _ = _pool(dev, 100 + tokens, 3, 4, lens, tokens, lambda rng, n: np.full(n, scale))
    q = torch.zeros((4, 8, 128), device=dev)
    for own, pre in ((tokens, 0), (0, tokens), (tokens, tokens)):
        want, bound = exact_rows(P, q, [own] * 4, pre)
        check(P.decode(q, [own] * 4, pre), want, bound, torch.float32)


@pytest.mark.parametrize("bits_k,bits_v,heads", [(3, 3, 8), (4, 8, 3), (8, 2, 4)])
def test_value_norms_over_seven_decades(dev, bits_k, bits_v, heads):
    """Every row's query is the direction of one key, whose value is the smallest of all, or zero: the output is
    that small value, or what the other tokens add up to."""
    import torch
    lens, prefix = [1500, 40, 700], 3000
    P, keys = _pool(dev, 70 + bits_v, bits_k, bits_v, lens, prefix, lambda rng, n: 10.0 ** rng.uniform(-6, 1, n))
    spread = torch.randn((3, heads, 128), device=dev)
    for pre in (0, prefix):
        for sharp in (0.0, 12.0, 25.0):
            q = spread * 0.3
            for b in range(3):
                K, V = keys[0] if pre and b < 2 else keys[b + 1]
                at = torch.argsort(V[:, 0].norm(dim=1))[:heads]              # tokens of the smallest values
                k = K[at, 0]
                # the direction in which this key stands out: q . k = sharp sqrt(128), keys weighted by their spread
                d = k / P.scale[0] ** 2
                q[b] = q[b] + sharp * math.sqrt(128.0) * d / (d * k).sum(1, keepdim=True)
            want, bound = exact_rows(P, q, lens, pre)
            for dt in (torch.float32, torch.bfloat16):
                check(P.decode(q, lens, pre, out_dtype=dt), want, bound, dt)


def test_the_top_logit_has_a_value_of_zero(dev):
    """A token that takes almost all weight and adds nothing: the output is what the others add, 2^-17 to 2^-58 of
    their values."""
    import torch
    lens, prefix = [300, 60], 900
    P = Paged(dev, 80, 1, 4, 4, 64, lens, prefix=prefix)
    sink = []
    for n, table in [(prefix, P.prefix_pages[None].contiguous())] + [(n, P.table[b:b + 1].contiguous()) for b, n in enumerate(lens)]:
        K, V = P.rows(n, torch.float32)
        V[n // 2] = 0.0
        P.append(K, V, [0], [0, n], table=table)
        sink.append(K[n // 2, 0])
    for pre in (0, prefix):
        for sharp in (12.0, 25.0, 40.0):
            q = torch.randn((2, 8, 128), device=dev) * 0.05
            for b in range(2):
                k = sink[0] if pre else sink[b + 1]
                d = k / P.scale[0] ** 2
                q[b] += sharp * math.sqrt(128.0) * d / (d * k).sum()
            want, bound = exact_rows(P, q, lens, pre)
            check(P.decode(q, lens, pre), want, bound, torch.float32)


def _no_bits(P):
    """Blocks of the head without key bits."""
    w = np.asarray(P.ref["w"])[0]
    assert (w == 0).any()
    return np.flatnonzero(w == 0)


@pytest.mark.parametrize("bits_k,heads", [(1, 8), (2, 3)])
@pytest.mark.parametrize("power", [10, 16, 40, 100])
def test_a_coordinate_without_key_bits_does_not_cost_the_others_digits(dev, bits_k, heads, power):
    """Queries 2^power times larger in a block whose keys are stored as zero: the logits do not see it."""
    import torch
    lens, prefix = [500, 1, 60], 700
    P, _ = _pool(dev, 90 + bits_k, bits_k, 3, lens, prefix, lambda rng, n: np.ones(n))
    b = int(_no_bits(P)[0])
    for dt in (torch.float32, torch.bfloat16):
        q = (torch.randn((3, heads, 128), device=dev) / P.scale[0]).to(dt)
        big = q.clone()
        big[..., [b, b + 64]] = 2.0 ** power
        for pre in (0, prefix):
            want, bound = exact_rows(P, q, lens, pre)
            check(P.decode(big, lens, pre), want, bound, torch.float32)


def test_a_query_that_is_not_finite_in_a_block_without_key_bits(dev):
    """0 * inf and 0 * NaN: the row is NaN, the other rows are as they were."""
    import torch
    lens, prefix = [200, 40, 0], 300
    P, _ = _pool(dev, 95, 1, 3, lens, prefix, lambda rng, n: np.ones(n))
    b = int(_no_bits(P)[-1])
    q = torch.randn((3, 8, 128), device=dev)
    bad = torch.zeros((3, 8), dtype=torch.bool, device=dev)
    odd = q.clone()
    odd[0, 1, b], odd[1, 7, b + 64], odd[1, 2, b] = float("inf"), float("nan"), -float("inf")
    bad[0, 1] = bad[1, 7] = bad[1, 2] = True
    for pre in (0, prefix):
        got, want = P.decode(odd, lens, pre), P.decode(q, lens, pre)
        assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], want[~bad])


def test_queries_at_the_ends_of_the_fp32_range(dev):
    """Largest and smallest queries, whose logits are one token's, or nothing."""
    import torch
    lens, prefix = [150, 90], 200
    P, _ = _pool(dev, 96, 3, 3, lens, prefix, lambda rng, n: np.ones(n))
    for size in (3e38, 1e30, 1e-30, 1e-38, 1e-45):
        q = torch.full((2, 8, 128), size, device=dev)
        for pre in (0, prefix):
            want, bound = exact_rows(P, q, lens, pre)
            got = P.decode(q, lens, pre)
            if size < 1:
                check(got, want, bound, torch.float32)
                continue
            # one token has all the weight: its value, or NaN where the logits pass fp32
            g = host_f32(got)
            right = np.isclose(g, want, rtol=2.0 ** -20, atol=0).all(2)
            assert right.all() if size == 1e30 else (right | np.isnan(g).all(2)).all()
