"""Chunks over the paged cache where something is not finite, or a total is very large.

A chunk of n tokens is n decode steps: what a query does not see cannot reach its output, whatever it holds.  What it
sees does: an infinite value gives an infinite output, NaN and infinities of both signs NaN; a NaN in a query or key
gives NaN to the query's output, to the totals of the keys that it sees, and through them to later outputs.  Finite
outputs and totals are held to the tolerances of tests/test_gpu_paged_chunk.py.
"""
import numpy as np
import pytest
import torch

from long_context_attention_gb300 import binding as b
from tests._parity import host64
from tests._paged import DEV, LONG
from tests.test_gpu_paged_chunk import make, oracle, run

pytestmark = pytest.mark.gpu

# the kernels for short calls and for few rows; several heads a tile; one head a tile, its last one partial
SIZES = [([300, 90], [4, 2]), ([300, 90], [20, 5]), ([700, 90], [130, 5]), ([130, 260], [130, 140])]


def tolerance(cu, info, d, bf16, ro):
    n = int(cu[-1])
    news = np.diff(cu.cpu().numpy())
    g = (2 * d + 8) * 2.0 ** -24 * info["spread"][:n]
    base = (2 * (4 * g + np.repeat(news, news)[:, None] * 2.0 ** -24 + 2.0 ** -19) * info["vmax"][:n])[..., None]
    return base + ((2.0 ** -8 * np.abs(ro) + 2.0 ** -8 * (1 + 2.0 ** -7) * info["dev"][:n]) if bf16 else 2.0 ** -24 * np.abs(ro))


def run_odd(cache, q, cu, max_new, max_len, spoil):
    """The call after `spoil`, by both kinds of kernels, against the oracle: the same outputs and totals are not finite,
    the others right (by the tolerances of the call before `spoil`, whose finite values it shares)."""
    with np.errstate(all="ignore"):
        clean = oracle(cache, q, cu)
        spoil(cache, q)
        ro, rD, info = oracle(cache, q, cu)
    start, d, bf16 = cache.demand_pages.clone(), q.shape[-1], q.dtype == torch.bfloat16
    assert not np.isfinite(ro).all() and np.isfinite(ro).any()
    for most in sorted({max_len, max(max_len, LONG)}):
        cache.demand_pages.copy_(start)
        ws = b.dilution_attn_paged_chunk_workspace(cache, q.shape[0], max_new, most)
        ws[256:] = 0xC7
        got = host64(b.dilution_attn_paged_chunk(q, cache, cu, max_new, most, workspace=ws))
        assert b.dilution_attn_get_error(ws) == b.DA_OK
        fine = np.isfinite(ro)
        assert np.array_equal(got[~fine], ro[~fine], equal_nan=True)
        assert np.isfinite(got[fine]).all()
        assert (np.abs(got[fine] - ro[fine]) <= tolerance(cu, clean[2], d, bf16, ro)[fine]).all()
        D, fine = host64(cache.demand_pages), np.isfinite(rD)
        assert np.array_equal(D[~fine], rD[~fine], equal_nan=True)
        assert np.abs(D[fine] - rD[fine]).max() <= 1e-4 * max(1.0, np.abs(rD[fine]).max())


def put(pages, cache, s, place, head, cols, value):
    page = cache.page_size
    pages[cache.page_table[s, place // page].long(), head, place % page, cols] = value


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 4, 2, 16), (128, 3, 3, 128), (64, 2, 2, 64)])
@pytest.mark.parametrize("lens,news", SIZES)
def test_values_that_a_query_does_not_see(lens, news, d, Hq, Hkv, page, dtype):
    """Infinite and NaN values of later new tokens: earlier rows do not know of them."""
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, dtype, seed=sum(news) + d)

    def spoil(cache, q):
        P, n = lens[0] - news[0], news[0]
        j = n // 2
        for cols, value in ((slice(0, 8), np.inf), (slice(8, 11), -np.inf), (slice(20, 23), np.nan), (slice(d - 1, d), np.inf)):
            put(cache.v_pages, cache, 0, P + j, 0, cols, value)
        put(cache.v_pages, cache, 0, P + j + 1, 0, slice(0, 3), -np.inf)       # and inf - inf
        put(cache.v_pages, cache, 0, P + n - 1, Hkv - 1, slice(30, 64), np.nan)   # the last row alone sees it
        put(cache.v_pages, cache, 1, lens[1] - 1, 0, slice(5, 6), np.inf)
    run_odd(cache, q, cu, max(news), max(lens), spoil)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", SIZES + [([300, 2700, 90], [6, 4, 5])])
def test_the_next_call_knows_nothing_of_it(lens, news, dtype):
    """One captured call on one workspace: values that are not finite, then finite ones again."""
    cache, q, cu = make(lens, news, 3, 3, 64, 32, dtype, seed=31)
    start, values = cache.demand_pages.clone(), cache.v_pages.clone()
    for max_len in (max(lens), LONG + 200):
        ref = b.dilution_attn_paged_chunk(q, cache, cu, max(news), max_len)
        total = cache.demand_pages.clone()
        ws = b.dilution_attn_paged_chunk_workspace(cache, q.shape[0], max(news), max_len)
        out, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.dilution_attn_paged_chunk(q, cache, cu, max(news), max_len, out, workspace=ws)
        for spoilt in (True, False, True):
            cache.demand_pages.copy_(start)
            if spoilt:
                put(cache.v_pages, cache, 1, lens[1] - 1, 0, slice(0, 64), np.nan)
            g.replay()
            row = int(cu[2]) - 1
            same = (out == ref).all(-1)
            same[row, 0] ^= spoilt       # that row's head 0 alone is NaN, and only then
            assert same.all() and torch.equal(cache.demand_pages, total)
            assert torch.isnan(out[row, 0]).all() == spoilt
            cache.v_pages.copy_(values)
        cache.demand_pages.copy_(start)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["key", "query"])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 4, 2, 16), (128, 3, 3, 128)])
@pytest.mark.parametrize("lens,news", SIZES)
def test_keys_and_queries_that_come_later(lens, news, d, Hq, Hkv, page, odd, which, dtype):
    """A NaN in a new key or in a query: rows before it, and totals of keys that only later rows see, stay finite."""
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, dtype, seed=sum(news) + d + odd)
    j = news[0] // 4 * 2 + odd

    def spoil(cache, q):
        if which == "key":
            put(cache.k_pages, cache, 0, lens[0] - news[0] + j, 0, slice(3, 4), np.nan)
        else:
            q[j, 0, 5] = float("nan")
    run_odd(cache, q, cu, max(news), max(lens), spoil)


@pytest.mark.parametrize("P,n", [(256, 129), (240, 17)])
def test_a_key_of_its_own_block(P, n):
    """A NaN in the last key, the only one of its 32 that the last row sees."""
    cache, q, cu = make([P + n], [n], 2, 2, 64, 64, "bf16", seed=n)
    run_odd(cache, q, cu, n, P + n, lambda c, q: put(c.k_pages, c, 0, P + n - 1, 0, slice(0, 1), np.nan))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("lens,news", SIZES)
def test_very_large_totals(lens, news, flags, dtype):
    """Finite totals of up to 1e30 divide as any other: all of a head's, some of another's."""
    cache, q, cu = make(lens, news, 4, 2, 64, 32, dtype, seed=7, fresh=False)
    g = torch.Generator().manual_seed(8)
    size = torch.randint(18, 31, cache.demand_pages.shape, generator=g).float()
    big = (10.0 ** size * (1 + torch.rand(size.shape, generator=g))).to(DEV)
    some = (torch.rand(size.shape, generator=g) < 0.3).to(DEV)
    some[:, 0] = some[:, 3] = True
    big[:, 3] = (1e27 * (1 + 1e3 * torch.rand(big[:, 3].shape, generator=g))).to(DEV)     # of that head's none is below 1e27
    cache.demand_pages.copy_(torch.where(some, big, cache.demand_pages))
    run(cache, q, cu, max(news), max(lens), flags=flags)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", SIZES)
def test_all_totals_infinite(lens, news, dtype):
    """No key has a share: NaN, as a decode step's 0 / 0, of that head alone."""
    cache, q, cu = make(lens, news, 4, 2, 64, 32, dtype, seed=9)

    def spoil(cache, q):
        t = torch.arange(lens[0], device=DEV)
        cache.demand_pages[cache.demand_table[0, t // 32].long(), 2, t % 32] = float("inf")
    run_odd(cache, q, cu, max(news), max(lens), spoil)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("lens,news", SIZES)
def test_a_very_large_eps(lens, news, flags, dtype):
    """eps of 1e25: the shares are the bids', and the totals grow by them all the same."""
    cache, q, cu = make(lens, news, 4, 2, 64, 32, dtype, seed=10)
    run(cache, q, cu, max(news), max(lens), flags=flags, eps=1e25)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,places", [(3000, [0, 7, 8, 255, 256, 2049, 2999]), (8500, [100, 8191, 8192, 8300]), (2900, list(range(2900)))])
def test_long_parts(T, places, dtype):
    """Infinite values here and there, across the slices of a long part, or of every token: each row has those of the tokens
    up to its own, and the bits of the clean call elsewhere."""
    d = 64
    cache, q, cu = make([T, 70], [T, 3], 2, 1, d, 64, dtype, seed=T, fresh=False)
    start = cache.demand_pages.clone()
    ref = b.dilution_attn_paged_chunk(q, cache, cu, T, T)
    total = cache.demand_pages.clone()
    cache.demand_pages.copy_(start)
    for i, t in enumerate(places):
        put(cache.v_pages, cache, 0, t, 0, slice(i % d, i % d + 1), np.inf if i % 2 else -np.inf)
    out = b.dilution_attn_paged_chunk(q, cache, cu, T, T)
    want = ref.clone()
    for i, t in enumerate(places[:d]):
        want[t:T, :, i % d] = np.inf if i % 2 else -np.inf
    assert torch.equal(out, want) and torch.equal(cache.demand_pages, total)
