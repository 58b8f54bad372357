"""CPU checks of the chunk and eviction entry points: refusals before any CUDA call, the oracle's own pins."""
import ctypes

import numpy as np
import pytest

from long_context_attention_gb300 import binding as b
from oracle import paged as op

FAKE = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return b.load()


def cache(k=FAKE, dem=FAKE, S=2, Hq=4, Hkv=2, d=64, page=16, pages=10, dpages=10, width=8, dtype=1, lens=FAKE, table=FAKE):
    return b._CPagedCache(k, FAKE, dem, table, FAKE, lens, S, Hq, Hkv, d, page, pages, dpages, width, dtype)


def test_chunk_refusals(lib):
    def call(q=FAKE, c=None, cu=FAKE, N=5, max_new=5, max_len=100, out=FAKE, tau=1.0, tau_bh=None, eps=1e-6, flags=0,
             ws=FAKE, n=BIG, status=None):
        return lib.dilution_attn_paged_chunk(q, ctypes.byref(cache() if c is None else c), cu, N, max_new, max_len, out, tau,
                                             tau_bh, eps, flags, ws, n, status, None)
    for kw in (dict(q=None), dict(q=FAKE + 8), dict(out=None), dict(out=FAKE + 2), dict(cu=None), dict(cu=FAKE + 1), dict(N=-1),
               dict(max_new=-1), dict(max_len=-1), dict(max_len=129), dict(tau=-1.0), dict(tau=float("nan")),
               dict(tau=float("inf")), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(flags=2), dict(flags=4),
               dict(tau_bh=FAKE + 2), dict(ws=FAKE + 16), dict(status=FAKE + 16), dict(c=cache(Hq=5)), dict(c=cache(k=None)),
               dict(c=cache(dem=FAKE + 4)), dict(c=cache(lens=None)), dict(c=cache(table=FAKE + 2)), dict(c=cache(dtype=2)),
               dict(c=cache(pages=-1)), dict(c=cache(page=0))):
        assert call(**kw) == b.DA_ERR_INVALID, kw
    for kw in (dict(eps=1e-19), dict(N=(1 << 30) + 1), dict(c=cache(d=96)), dict(c=cache(page=8)), dict(c=cache(page=24)),
               dict(c=cache(pages=1 << 30, Hkv=2)), dict(c=cache(S=1 << 23)), dict(c=cache(width=1 << 27), max_len=(1 << 30) + 1)):
        assert call(**kw) == b.DA_ERR_UNSUPPORTED, kw
    assert lib.dilution_attn_paged_chunk(FAKE, None, FAKE, 5, 5, 5, FAKE, 1.0, None, 1e-6, 0, FAKE, BIG, None, None) == \
        b.DA_ERR_INVALID
    need = b.dilution_attn_paged_chunk_workspace_size(2, 4, 2, 64, 5, 5, 100, 1)
    assert need >= 256
    assert call(n=need - 1) == b.DA_ERR_WORKSPACE and call(ws=None) == b.DA_ERR_WORKSPACE
    # nothing to do, whatever the pointers
    assert call(q=None, out=None, cu=None, N=0, ws=None) == b.DA_OK
    assert call(c=cache(S=0, k=None), q=None) == b.DA_OK


def test_chunk_workspace_size(lib):
    size = b.dilution_attn_paged_chunk_workspace_size
    for bad in ((-1, 4, 2, 64, 5, 5, 9, 1), (2, 0, 2, 64, 5, 5, 9, 1), (2, 4, 3, 64, 5, 5, 9, 1), (2, 4, 2, 96, 5, 5, 9, 1),
                (2, 4, 2, 64, -1, 5, 9, 1), (2, 4, 2, 64, 5, -1, 9, 1), (2, 4, 2, 64, 5, 5, -1, 1), (2, 4, 2, 64, 5, 5, 9, 3),
                (2, 4, 2, 64, 5, 5, (1 << 30) + 1, 1)):
        assert size(*bad) == 0
    for dt in (0, 1):
        assert size(2, 4, 2, 64, 5, 50, 100, dt) == size(2, 4, 2, 64, 5, 5, 100, dt)      # never more than N of a sequence
        assert size(2, 4, 2, 64, 500, 50, 7, dt) == size(2, 4, 2, 64, 500, 7, 7, dt)      # nor more than its length
        assert size(4, 4, 2, 64, 500, 50, 100, dt) >= size(2, 4, 2, 64, 500, 50, 100, dt)
        assert size(64, 64, 2, 128, 1 << 20, 1 << 20, 1 << 20, dt) > 1 << 33              # past 32 bits
        # a workspace serves every call within its bounds
        for hq, hkv, d in ((12, 12, 64), (16, 4, 128), (32, 1, 64), (8, 8, 128)):
            for S in (1, 7, 300):
                steps = ((1, 1, 1), (3, 1, 100), (5, 3, 5000), (8, 8, 5000), (9, 8, 131072), (300, 8, 131072), (300, 16, 131072),
                         (4000, 16, 131072), (4000, 2048, 131072), (4000, 2048, 1 << 22), (40000, 40000, 1 << 24))
                sizes = [size(S, hq, hkv, d, *x, dt) for x in steps]
                assert sizes == sorted(sizes), (S, hq, hkv, d)


def test_evict_refusals(lib):
    def call(c=None, dst=None, ddst=None, width=8, keep=FAKE, max_keep=50, max_len=100, sinks=0, recent=0, lens=FAKE, kept=None,
             ws=FAKE, n=BIG, status=None):
        return lib.dilution_attn_paged_evict(ctypes.byref(cache() if c is None else c), dst, ddst, width, keep, max_keep, max_len,
                                             sinks, recent, lens, kept, ws, n, status, None)
    for kw in (dict(dst=FAKE), dict(ddst=FAKE), dict(dst=FAKE + 2, ddst=FAKE), dict(dst=FAKE, ddst=FAKE + 1),
               dict(dst=FAKE, ddst=FAKE, width=3), dict(dst=FAKE, ddst=FAKE, width=-1), dict(keep=None), dict(keep=FAKE + 2),
               dict(max_keep=-1), dict(max_len=-1), dict(max_len=129), dict(sinks=-1), dict(recent=-1), dict(lens=None),
               dict(lens=FAKE + 1), dict(kept=FAKE + 1), dict(ws=FAKE + 16), dict(status=FAKE + 16), dict(c=cache(Hq=5)),
               dict(c=cache(k=None)), dict(c=cache(dtype=2))):
        assert call(**kw) == b.DA_ERR_INVALID, kw
    for kw in (dict(c=cache(d=96)), dict(c=cache(page=8)), dict(c=cache(S=1 << 23)),
               dict(c=cache(width=1 << 27), max_len=(1 << 30) + 1)):
        assert call(**kw) == b.DA_ERR_UNSUPPORTED, kw
    need = b.dilution_attn_paged_evict_workspace_size(2, 2, 50, 100)
    assert call(n=need - 1) == b.DA_ERR_WORKSPACE and call(ws=None) == b.DA_ERR_WORKSPACE
    assert call(c=cache(S=0, k=None), keep=None, lens=None) == b.DA_OK


def test_evict_workspace_size(lib):
    size = b.dilution_attn_paged_evict_workspace_size
    assert size(-1, 1, 5, 5) == size(1, 0, 5, 5) == size(1, 1, -1, 5) == size(1, 1, 5, -1) == size(1, 1, 5, (1 << 30) + 1) == 0
    assert size(2, 3, 500, 100) == size(2, 3, 100, 100)
    assert size(64, 64, 1 << 20, 1 << 20) > 1 << 33
    for S, hkv in ((1, 1), (3, 12), (200, 4)):       # a workspace serves every call within its bounds
        sizes = [size(S, hkv, *x) for x in ((0, 1), (1, 1), (5, 500), (500, 500), (500, 513), (500, 40000), (500, 1 << 19), (500, 1 << 20),
                                            (1 << 19, 1 << 20), (1 << 19, 1 << 24))]
        assert sizes == sorted(sizes), (S, hkv)


def rand_cache(g, lens, Hq, Hkv, d, page):
    width = max(-(-n // page) for n in lens)
    t = g.permutation(len(lens) * width).reshape(len(lens), width)
    n = len(lens) * width
    return (g.standard_normal((n, Hkv, page, d)), g.standard_normal((n, Hkv, page, d)),
            g.exponential(size=(n, Hq, page)).astype(np.float32), t, t[::-1])


def test_oracle_chunk_is_decode_steps():
    """A chunk of n tokens is n decode steps, each a token longer."""
    g = np.random.default_rng(0)
    lens, news = [23, 9], [6, 9]
    K, V, D, t, dt = rand_cache(g, lens, 4, 2, 8, 4)
    q = g.standard_normal((15, 4, 8))
    cu = [0, 6, 15]
    for earlier in (False, True):
        out, D1, info = op.paged_chunk(q, K, V, D, t, dt, lens, cu, 1.3, 1e-3, earlier)
        D2 = np.array(D, np.float64)
        for s in range(2):
            for i in range(news[s]):
                one = [0, 0]
                one[s] = lens[s] - news[s] + i + 1
                qs = np.zeros((2, 4, 8))
                qs[s] = q[cu[s] + i]
                o, D2, _ = op.paged_decode(qs, K, V, D2, t, dt, one, 1.3, 1e-3, earlier)
                assert np.allclose(o[s], out[cu[s] + i], atol=1e-12)
        assert np.allclose(D1, D2, atol=1e-12)
        assert np.allclose(sum(p.sum() for p in info["bids"].values()), 15 * 4)


def test_oracle_evict_keeps_the_highest():
    g = np.random.default_rng(1)
    lens, keeps = [30, 12, 0], [11, 20, 3]
    K, V, D, t, dt = rand_cache(g, lens[:2], 4, 2, 8, 4)
    t, dt = np.vstack([t, t[:1]]), np.vstack([dt, dt[:1]])
    K2, V2, D2, nl, kept = op.paged_evict(K, V, D, t, dt, lens, keeps, 20, 2, 3)
    assert nl.tolist() == [11, 12, 0] and (kept[2] == -1).all() and (kept[1, :, :12] == np.arange(12)).all()
    for h in range(2):
        stay = kept[0, h, :11]
        assert (np.diff(stay) > 0).all() and {0, 1, 27, 28, 29} <= set(stay.tolist())
        score = (D[dt[0][np.arange(30) // 4], 2 * h, np.arange(30) % 4] + D[dt[0][np.arange(30) // 4], 2 * h + 1, np.arange(30) % 4])
        rest = [i for i in range(30) if i not in stay]
        free = [i for i in stay if 2 <= i < 27]
        assert min(score[free]) >= max(score[rest])
        for r, i in enumerate(stay):
            assert np.array_equal(K2[t[0][r // 4], h, r % 4], K[t[0][i // 4], h, i % 4])
            assert np.array_equal(D2[dt[0][r // 4], 2 * h:2 * h + 2, r % 4], D[dt[0][i // 4], 2 * h:2 * h + 2, i % 4])
