"""Eviction from the paged cache: bit for bit the oracle's rows, places and lengths."""
import numpy as np
import pytest
import torch

from long_context_attention_gb300 import binding as b
from oracle import paged as op
from tests._parity import host64
from tests._paged import DEV, make_cache

pytestmark = pytest.mark.gpu


def pools(cache):
    return [host64(x) if x.dtype != torch.float32 else x.cpu().numpy() for x in (cache.k_pages, cache.v_pages, cache.demand_pages)]


def dst_tables(cache, lens, keeps, seed):
    """Pages that no sequence holds for every row that stays, and the tables that name them."""
    g = torch.Generator().manual_seed(seed)
    page = cache.page_size
    need = [-(-min(n, k) // page) for n, k in zip(lens, keeps)]
    out = []
    for table, n in ((cache.page_table, cache.k_pages.shape[0]), (cache.demand_table, cache.demand_pages.shape[0])):
        free = sorted(set(range(n)) - set(table.flatten().tolist()))
        free = [free[i] for i in torch.randperm(len(free), generator=g).tolist()]
        t, at = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32), 0
        for s, m in enumerate(need):
            t[s, :m] = torch.tensor(free[at:at + m], dtype=torch.int32)
            at += m
        out.append(t.to(DEV))
    return out


def evict(cache, lens, keeps, max_keep, max_len, sinks=0, recent=0, to=None, kept=True, **kw):
    """The call against the oracle, everything compared; then with the lengths written where they are read, which the
    kernel for short sequences does not take."""
    before = pools(cache)
    start = [x.clone() for x in (cache.k_pages, cache.v_pages, cache.demand_pages)]
    tables = [x.cpu().numpy() for x in (cache.page_table, cache.demand_table)]
    dst = [None, None] if to is None else [x.cpu().numpy() for x in to]
    rK, rV, rD, rl, rk = op.paged_evict(*before, *tables, lens, keeps, max_keep, sinks, recent, *dst)
    lengths = cache.seq_lens.clone()
    for new_lens in (None, cache.seq_lens):
        for x, y in zip((cache.k_pages, cache.v_pages, cache.demand_pages), start):
            x.copy_(y)
        ws = b.dilution_attn_paged_evict_workspace(cache, max_keep, max_len)
        ws[256:] = 0xC7
        kt = torch.full((cache.S, cache.Hkv, max_keep), 99, dtype=torch.int32, device=DEV) if kept else None
        got = b.dilution_attn_paged_evict(cache, torch.tensor(keeps, dtype=torch.int32, device=DEV), max_keep, max_len, new_lens,
                                          sinks=sinks, recent=recent, kept=kt, workspace=ws,
                                          dst_page_table=None if to is None else to[0],
                                          dst_demand_table=None if to is None else to[1], **kw)
        assert b.dilution_attn_get_error(ws) == b.DA_OK
        assert got.tolist() == rl.tolist()
        if kept:
            assert np.array_equal(kt.cpu().numpy(), rk)
        for x, y in zip(pools(cache), (rK, rV, rD)):
            assert np.array_equal(x, y, equal_nan=True)
    cache.seq_lens.copy_(lengths)


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("dtype,d,page,Hq,Hkv", [("bf16", 64, 16, 2, 2), ("f32", 128, 32, 6, 2), ("bf16", 128, 256, 8, 1),
                                                 ("f32", 64, 64, 3, 3)])
@pytest.mark.parametrize("lens,keeps,sinks,recent", [
    ([1], [1], 0, 0), ([1], [0], 0, 0), ([2], [1], 0, 0), ([40], [39], 0, 0), ([40], [39], 4, 8), ([300], [100], 4, 33),
    ([500, 0, 257, 1, 90], [250, 5, 1, 1, 200], 2, 10), ([600], [64], 0, 0), ([700, 33], [699, 0], 1, 1),
    ([128], [20], 16, 16), ([1500, 1100], [700, 1099], 0, 64), ([507, 512, 31], [300, 511, 20], 1, 7), ([513], [512], 0, 0),
])
def test_evict(lens, keeps, sinks, recent, dtype, d, page, Hq, Hkv, place):
    most = max(min(n, k) for n, k in zip(lens, keeps))
    spare = sum(-(-min(n, k) // page) for n, k in zip(lens, keeps)) + 3
    cache, _, _ = make_cache(len(lens), lens, Hq, Hkv, d, page, dtype, seed=sum(lens), spare=spare, extra_width=1,
                             junk=float("nan"))
    to = None if place else dst_tables(cache, lens, keeps, 1)
    evict(cache, lens, keeps, most + 3, max(lens) + 5 if max(lens) + 5 <= cache.max_pages * page else max(lens), sinks, recent,
          to)


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("values", ["equal", "few", "special", "close"])
def test_ties_and_special_values(values, place):
    """Equal scores go by the lower place; zeros of both signs are equal; infinities; NaN stays; neighbours in the last bit."""
    lens, keeps = [777, 300], [300, 17]
    cache, _, _ = make_cache(2, lens, 4, 2, 64, 32, "bf16", seed=9, spare=20, extra_width=1)
    g = torch.Generator().manual_seed(3)
    shape = cache.demand_pages.shape
    if values == "equal":
        dem = torch.ones(shape)
    elif values == "few":
        dem = torch.randint(0, 3, shape, generator=g).float()
    elif values == "special":
        pick = torch.tensor([0.0, -0.0, float("inf"), float("nan"), -1.0, 1e-42, 3e38, -float("nan"), -float("inf"), 2.0])
        dem = pick[torch.randint(0, len(pick), shape, generator=g)]
    else:
        dem = torch.tensor(1.0).view(torch.int32).add(torch.randint(0, 300, shape, generator=g).int()).view(torch.float32)
    cache.demand_pages.copy_(dem)
    with np.errstate(invalid="ignore", over="ignore"):
        evict(cache, lens, keeps, 300, 777, 0, 5, None if place else dst_tables(cache, lens, keeps, 2))


def test_long_and_many_key_heads():
    """Clusters of several CTAs, whole slices that stay or go, a max_len far above the lengths."""
    cache, _, _ = make_cache(1, [9000], 1, 1, 64, 256, "bf16", seed=4, extra_width=40)
    evict(cache, [9000], [4000], 4000, 9000 + 256 * 30)
    cache, _, _ = make_cache(1, [6000], 2, 1, 64, 256, "f32", seed=5, extra_width=1)
    t = torch.arange(6000, device=DEV)
    cache.demand_pages[cache.demand_table[0, t // 256].long(), :, t % 256] = (t[:, None] < 3100).float() * 2 + 1
    evict(cache, [6000], [3200], 3200, 6000)
    cache, _, _ = make_cache(3, [70, 64, 65], 80, 80, 64, 16, "bf16", seed=6, extra_width=1)
    evict(cache, [70, 64, 65], [64, 64, 64], 64, 70, 1, 5)


def test_scores_in_the_workspace():
    """A max_len whose scores do not fit in shared memory: the lengths that come are short all the same."""
    S, page = 1, 256
    cache, _, _ = make_cache(S, [3000], 2, 2, 64, page, "bf16", seed=7, extra_width=1700)
    evict(cache, [3000], [1000], 1000, 8 * 48 * 1024 + 4096, 3, 50)
    cache, _, _ = make_cache(S, [3000], 2, 2, 64, page, "bf16", seed=8, extra_width=1700)
    evict(cache, [3000], [1000], 1000, 3000, 3, 50, kept=False)


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("S", [33, 1024, 1100])
def test_many_sequences(S, place):
    """More sequences than the counted chunks of the moving kernel, empty and untouched ones among them."""
    lens = [s * 11 % 41 for s in range(S)]
    keeps = [s * 5 % 29 for s in range(S)]
    most = max(min(n, k) for n, k in zip(lens, keeps))
    spare = sum(-(-min(n, k) // 16) for n, k in zip(lens, keeps)) + 2
    cache, _, _ = make_cache(S, lens, 4, 2, 64, 16, "bf16", seed=S, spare=spare, extra_width=1)
    evict(cache, lens, keeps, most, max(lens), 1, 3, None if place else dst_tables(cache, lens, keeps, 4))


def test_nothing_to_do():
    """Bounds of zero, sequences without tokens."""
    cache, _, _ = make_cache(2, [0, 0], 2, 1, 64, 16, "bf16", seed=14, extra_width=2)
    evict(cache, [0, 0], [5, 0], 0, 0)
    evict(cache, [0, 0], [5, 0], 5, 20)
    cache, _, _ = make_cache(2, [30, 0], 2, 1, 64, 16, "bf16", seed=15, extra_width=2)
    evict(cache, [30, 0], [0, 7], 0, 30)
    evict(cache, [30, 0], [30, 7], 30, 30, 2 ** 31 - 1, 2 ** 31 - 1)


def test_groups_of_heads():
    """Groups that are no multiple of four heads, sums in the heads' order."""
    for Hq, Hkv in ((7, 1), (10, 2), (9, 9), (15, 3)):
        cache, _, _ = make_cache(2, [333, 65], Hq, Hkv, 128, 32, "bf16", seed=Hq, spare=30, extra_width=1)
        cache.demand_pages.mul_(torch.logspace(-6, 6, Hq, device=DEV)[None, :, None])
        evict(cache, [333, 65], [111, 64], 111, 333, 0, 3)


def test_shared_prefix_keeps_its_pages():
    """Two sequences share the pages of 64 tokens; both keep them all (sinks), to tables that name the same pages."""
    cache, _, prefix = make_cache(2, [300, 200], 2, 1, 64, 32, "bf16", seed=10, prefix=64, spare=20, extra_width=1)
    lens, keeps = [300, 200], [128, 100]
    to = dst_tables(cache, lens, keeps, 5)
    to[0][:, :2] = prefix
    before = cache.k_pages[prefix.long()].clone()
    evict(cache, lens, keeps, 128, 300, 64, 10, to)
    assert torch.equal(cache.k_pages[prefix.long()], before)
    cache, _, _ = make_cache(2, [300, 200], 2, 1, 64, 32, "bf16", seed=10, prefix=64, spare=20, extra_width=1)
    evict(cache, lens, keeps, 128, 300, 64, 10)      # in place too


def test_lengths_in_place_streams_and_graphs():
    lens, keeps = [400, 90, 300], [200, 200, 100]
    make = lambda: make_cache(3, lens, 4, 2, 128, 32, "bf16", seed=12, extra_width=1)[0]
    want = make()
    keep = torch.tensor(keeps, dtype=torch.int32, device=DEV)
    kept = torch.empty(3, 2, 200, dtype=torch.int32, device=DEV)
    want_lens = b.dilution_attn_paged_evict(want, keep, 200, 400, sinks=2, recent=9, kept=kept)

    def same(cache):
        assert cache.seq_lens.tolist() == want_lens.tolist() == [200, 90, 100]
        assert all(np.array_equal(x, y, equal_nan=True) for x, y in zip(pools(cache), pools(want)))
        assert b.dilution_attn_get_error(cache.status) == b.DA_OK
    cache = make()
    assert b.dilution_attn_paged_evict(cache, keep, 200, 400, cache.seq_lens, sinks=2, recent=9) is cache.seq_lens
    same(cache)
    cache = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.dilution_attn_paged_evict(cache, keep, 200, 400, cache.seq_lens, sinks=2, recent=9, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same(cache)
    cache = make()
    fresh = [x.clone() for x in (cache.k_pages, cache.v_pages, cache.demand_pages, cache.seq_lens)]
    ws = b.dilution_attn_paged_evict_workspace(cache, 200, 400)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.dilution_attn_paged_evict(cache, keep, 200, 400, cache.seq_lens, sinks=2, recent=9, workspace=ws)
    for _ in range(2):
        for x, y in zip((cache.k_pages, cache.v_pages, cache.demand_pages, cache.seq_lens), fresh):
            x.copy_(y)
        g.replay()
        same(cache)


@pytest.mark.parametrize("inside", [False, True])
def test_bad_lengths_budgets_and_pages(inside):
    """``inside``: the lengths written where they are read."""
    lens, keeps = [100, 200, 150], [50, 60, 70]
    for place in (True, False):
        def call(change, max_keep=70, max_len=200, keeps=keeps, good=(0, 2), whole=True):
            cache, _, _ = make_cache(3, lens, 4, 2, 64, 16, "bf16", seed=13, spare=20, extra_width=1)
            to = None if place else dst_tables(cache, lens, keeps, 3)
            change(cache, to)
            before = pools(cache)
            l2, k2 = cache.seq_lens.tolist(), list(keeps)
            for s in range(3):
                if s not in good:
                    k2[s] = 0           # the oracle moves nothing of it
            l3 = [n if s in good else 0 for s, n in enumerate(l2)]
            tables = [x.cpu().numpy() for x in (cache.page_table, cache.demand_table)]
            dst = [None, None] if to is None else [x.cpu().numpy() for x in to]
            ref = op.paged_evict(*before, *tables, l3, k2, max_keep, 1, 5, *dst)
            ws = b.dilution_attn_paged_evict_workspace(cache, max_keep, max_len)
            kept = torch.full((3, 2, max_keep), 99, dtype=torch.int32, device=DEV)
            got = b.dilution_attn_paged_evict(cache, torch.tensor(keeps, dtype=torch.int32, device=DEV), max_keep, max_len,
                                              cache.seq_lens if inside else None, sinks=1, recent=5, kept=kept, workspace=ws,
                                              dst_page_table=None if place else to[0], dst_demand_table=None if place else to[1])
            assert b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID
            assert b.dilution_attn_get_error(ws) == b.DA_OK
            for s in good:
                assert got[s] == ref[3][s] and np.array_equal(kept[s].cpu().numpy(), ref[4][s])
            if whole:       # a sequence that is not valid stays as it is
                bad = ({0, 1, 2} - set(good)).pop()
                assert got[bad] == l2[bad] and (kept[bad] == -1).all()
                assert all(np.array_equal(x, y, equal_nan=True) for x, y in zip(pools(cache), ref))

        def length(bad):
            return lambda cache, to: cache.seq_lens.__setitem__(1, bad)
        for bad in (-1, 201, 10 ** 9):
            call(length(bad))
        call(lambda c, t: None, keeps=[50, -1, 70])
        call(lambda c, t: None, keeps=[50, 71, 70])
        for bad in (-1, 10 ** 9, -2 ** 31):
            call(lambda cache, to: cache.page_table[1].fill_(bad), whole=False)
            call(lambda cache, to: cache.demand_table[1].fill_(bad), whole=False)
            if not place:
                call(lambda cache, to: to[0][1].fill_(bad), whole=False)
                call(lambda cache, to: to[1][1].fill_(bad), whole=False)
