"""Evictions of long sequences: every loop of the kernels more than once, bit for bit."""
import numpy as np
import pytest
import torch

from long_context_attention_gb300 import binding as b
from oracle import paged as op
from tests._paged import DEV, make_cache
from tests._paged_long import evict64
from tests.test_gpu_paged_evict import dst_tables, pools

pytestmark = pytest.mark.gpu


def evict_long(cache, lens, keeps, max_keep, max_len, sinks=0, recent=0, to=None, kept=True):
    rK, rV, rD, rl, rk = evict64(cache, lens, keeps, max_keep, sinks, recent, to)
    ws = b.dilution_attn_paged_evict_workspace(cache, max_keep, max_len)
    ws[256:] = 0xC7
    kt = torch.full((cache.S, cache.Hkv, max_keep), 99, dtype=torch.int32, device=DEV) if kept else None
    got = b.dilution_attn_paged_evict(cache, torch.tensor(keeps, dtype=torch.int32, device=DEV), max_keep, max_len,
                                      sinks=sinks, recent=recent, kept=kt, workspace=ws,
                                      dst_page_table=None if to is None else to[0],
                                      dst_demand_table=None if to is None else to[1])
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    assert got.tolist() == rl.tolist()
    if kept:
        assert np.array_equal(kt.cpu().numpy(), rk)
    for x, y in zip(pools(cache), (rK, rV, rD)):
        assert np.array_equal(x, y, equal_nan=True)


def test_the_two_oracles_agree():
    cache, _, _ = make_cache(2, [300, 41], 4, 2, 64, 16, "bf16", seed=1, spare=30, extra_width=1)
    cache.demand_pages.copy_((cache.demand_pages * 3).round())
    to = dst_tables(cache, [300, 41], [120, 50], 2)
    for x, y in zip(evict64(cache, [300, 41], [120, 50], 130, 2, 9, to),
                    op.paged_evict(*pools(cache), *(x.cpu().numpy() for x in (cache.page_table, cache.demand_table)), [300, 41],
                                   [120, 50], 130, 2, 9, *(x.cpu().numpy() for x in to))):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("dtype,d,page,Hq,Hkv,lens,keeps", [
    ("bf16", 64, 64, 2, 2, [40000], [17000]),               # 5000 keys a CTA
    ("f32", 128, 256, 3, 1, [30001, 7000], [9001, 6999]),
    ("bf16", 128, 32, 20, 20, [30000], [12345]),            # a CTA a key head
    ("bf16", 64, 16, 2, 1, [65536, 1, 4097], [4096, 1, 4096]),
])
def test_long_slices(dtype, d, page, Hq, Hkv, lens, keeps, place):
    """More keys a CTA than one step of its threads takes; thousands of rows and of totals to move."""
    spare = sum(-(-min(n, k) // page) for n, k in zip(lens, keeps)) + 2
    cache, _, _ = make_cache(len(lens), lens, Hq, Hkv, d, page, dtype, seed=sum(lens), spare=spare, extra_width=1)
    most = max(min(n, k) for n, k in zip(lens, keeps))
    evict_long(cache, lens, keeps, most + 1, max(lens), 3, 77, None if place else dst_tables(cache, lens, keeps, 4))


@pytest.mark.parametrize("place,kept", [(True, True), (False, True), (True, False)])
def test_more_scores_than_shared_memory_holds(place, kept):
    """340,000 tokens of one key head: 42,500 scores a CTA, in the workspace; ties across the CTAs' borders."""
    n, keep = 340000, 100000
    cache, _, _ = make_cache(1, [n], 2, 1, 64, 256, "bf16", seed=5, spare=400, extra_width=1)
    cache.demand_pages.copy_((cache.demand_pages * 4096).round() / 4096)
    evict_long(cache, [n], [keep], keep, n, 4, 1000, None if place else dst_tables(cache, [n], [keep], 6), kept)


def test_few_different_scores_over_long_slices():
    """Scores of two values: tens of thousands of equal ones, the first of which stay."""
    cache, _, _ = make_cache(1, [50000], 1, 1, 64, 64, "bf16", seed=6, extra_width=1)
    cache.demand_pages.copy_((cache.demand_pages > 0.7).float())
    evict_long(cache, [50000], [30000], 30000, 50000, 0, 0)
    cache, _, _ = make_cache(1, [50000], 1, 1, 64, 64, "bf16", seed=6, extra_width=1)
    cache.demand_pages.fill_(2.0)
    evict_long(cache, [50000], [49999], 49999, 50000, 0, 1)
