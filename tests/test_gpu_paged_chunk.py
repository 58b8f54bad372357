"""Chunks of new tokens over the paged cache against the float64 oracle.

Tolerances (written before any run).  A logit is off by at most
g = (2 d + 8) 2^-24 sum |q_i k_i| tau / sqrt(d), a bid by a factor 1 +- 2 g (see
tests/_paged.py).  A total is a running fp32 sum: after n queries it is off by
2 g and 2^-20 (the exponentials) of its bids and by n 2^-24 of itself; a share by
4 g + n 2^-24 + 2^-19, and a row of A by twice that, which times the largest value
bounds the row of out.  bf16: each share is rounded, by at most 2^-8 of itself, and
numerator and sum hold the same rounded shares, so that out moves by at most
2^-8 sum A |v - out| (1 + 2^-7); out itself is rounded by 2^-8.  Those roundings
are independent with a standard deviation of at most 2^-8 / sqrt(3) each: the root
mean square of the errors, each relative to its own standard deviation, is at most
1; 1.5 allows for few rows (the smallest test has 128 elements: 4 standard errors).
"""
import numpy as np
import pytest
import torch

from long_context_attention_gb300 import binding as b
from long_context_attention_gb300 import rope_inv_freq
from oracle import paged as op
from tests._parity import host64
from tests._paged import DEV, LONG, TYPES, make_cache, oracle_step

pytestmark = pytest.mark.gpu


def make(lens, news, Hq, Hkv, d, page, dtype, seed=0, junk=None, pad=0, spare=2, fresh=True):
    """A cache whose sequences' last news[s] tokens are new (no demand yet), their queries and cu_tokens."""
    cache, _, _ = make_cache(len(lens), lens, Hq, Hkv, d, page, dtype, seed=seed, junk=junk, spare=spare)
    g = torch.Generator().manual_seed(seed + 1)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    N = int(cu[-1]) + pad
    q = (torch.randn(N, Hq, d, generator=g) * 1.5).to(TYPES[dtype])
    if pad:
        q[int(cu[-1]):] = float("nan")
    if fresh:
        for s, n in enumerate(news):
            if n:
                t = torch.arange(lens[s] - n, lens[s], device=DEV)
                cache.demand_pages[cache.demand_table[s, t // page].long(), :, t % page] = 0.0
    return cache, q.to(DEV), torch.tensor(cu, device=DEV)


def oracle(cache, q, cu, tau=1.0, eps=1e-6, earlier=False):
    with np.errstate(invalid="ignore"):
        return op.paged_chunk(host64(q), host64(cache.k_pages), host64(cache.v_pages), host64(cache.demand_pages),
                              cache.page_table.cpu().numpy(), cache.demand_table.cpu().numpy(),
                              cache.seq_lens.cpu().numpy(), cu.cpu().numpy(), tau, eps, earlier)


def check(cache, q, cu, before, out, ref):
    ro, rD, info = ref
    n_rows, d, bf16 = int(cu[-1]), q.shape[-1], out.dtype == torch.bfloat16
    got, ro = host64(out)[:n_rows], ro[:n_rows]
    news = np.diff(cu.cpu().numpy())
    per_row = np.repeat(news, news)[:, None]
    g = (2 * d + 8) * 2.0 ** -24 * info["spread"][:n_rows]
    base = (2 * (4 * g + per_row * 2.0 ** -24 + 2.0 ** -19) * info["vmax"][:n_rows])[..., None]
    step = (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(ro)
    share = 2.0 ** -8 * (1 + 2.0 ** -7) * info["dev"][:n_rows] if bf16 else 0.0
    err = np.abs(got - ro)
    assert np.isfinite(got).all()
    assert (err <= base + step + share).all(), float((err - base - step - share).max())
    if bf16 and n_rows:
        sd = np.sqrt(((2.0 ** -8 * info["dev2"][:n_rows]) ** 2 + step ** 2) / 3) + base
        assert np.sqrt(np.mean((err / sd) ** 2)) <= 1.5
    D, page, dt = host64(cache.demand_pages), cache.page_size, cache.demand_table.cpu().numpy()
    seen = np.zeros(D.shape, dtype=bool)
    cuh = cu.cpu().numpy()
    for (s, h), p in info["bids"].items():
        t = np.arange(len(p))
        at = (dt[s][t // page], h, t % page)
        seen[at] = True
        gs = g[cuh[s]:cuh[s + 1], h].max()
        bound = p * (2 * gs + 2.0 ** -20) + (news[s] + 1) * 2.0 ** -24 * rD[at] + 1e-30
        assert (np.abs(D[at] - rD[at]) <= bound).all(), (s, h, float((np.abs(D[at] - rD[at]) - bound).max()))
    assert np.array_equal(D[~seen], host64(before)[~seen], equal_nan=True)


def run(cache, q, cu, max_new, max_len, **kw):
    """The call with max_len and with one past what the kernel for short calls takes, which the result does not depend
    on; the cache is left as after one call."""
    tau = kw.get("tau", 1.0) if kw.get("tau_bh") is None else host64(kw["tau_bh"]).reshape(cache.S, cache.Hq)
    before = cache.demand_pages.clone()
    ref = oracle(cache, q, cu, tau, kw.get("eps", 1e-6), bool(kw.get("flags", 0) & b.DA_FLAG_EARLIER_DEMAND_ONLY))
    for most in sorted({max_len, max(max_len, min(LONG, cache.max_pages * cache.page_size))}):
        cache.demand_pages.copy_(before)
        ws = b.dilution_attn_paged_chunk_workspace(cache, q.shape[0], max_new, most)
        ws[256:] = 0xC7          # whatever an earlier call left
        out = torch.full_like(q, 7.0)
        got = b.dilution_attn_paged_chunk(q, cache, cu, max_new, most, out, workspace=ws, **kw)
        assert got is out and b.dilution_attn_get_error(ws) == b.DA_OK
        check(cache, q, cu, before, out, ref)
        assert (out[int(cu[-1]):] == 7.0).all()          # rows behind the last sequence
    return out


# lengths and new tokens around every border: rows of 8, half and whole column tiles, key tiles, pages
SHAPES = [
    ([1], [1]), ([5], [5]), ([130], [1]), ([300], [7]), ([64], [64]), ([129], [33]), ([257], [65]), ([128], [128]),
    ([200], [129]), ([385], [300]), ([1, 2, 3], [1, 2, 3]), ([70, 0, 150, 9, 260], [3, 0, 65, 0, 130]),
    ([40, 41, 33, 500], [8, 9, 31, 64]), ([127, 255, 256], [63, 127, 256]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,page,Hq,Hkv", [(64, 16, 2, 2), (128, 32, 3, 1), (64, 256, 4, 2)])
@pytest.mark.parametrize("lens,news", SHAPES)
def test_shapes(lens, news, d, page, Hq, Hkv, dtype):
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, dtype, seed=len(lens) + sum(lens), junk=float("nan"), pad=3)
    run(cache, q, cu, max(news), max(lens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (20, 1), (34, 2), (5, 5)])
@pytest.mark.parametrize("n", [1, 9, 17, 40, 70])
def test_groups(Hq, Hkv, n, dtype):
    """Many query heads on a key head: narrow tiles of several heads, several column tiles of them."""
    cache, q, cu = make([n + 150, 61], [n, min(n, 61)], Hq, Hkv, 64, 64, dtype, seed=Hq + n)
    run(cache, q, cu, n + 5, n + 150)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_long(d, dtype):
    """Many pieces a segment, several column tiles."""
    cache, q, cu = make([2900, 1111, 1500], [200, 1, 30], 2, 1, d, 128, dtype, seed=3)
    run(cache, q, cu, 200, 2900)


@pytest.mark.parametrize("d,Hq,Hkv,page,lens,news", [
    (64, 12, 12, 64, [40000], [4]), (64, 6, 6, 16, [30000, 5000], [5, 130]), (64, 8, 2, 32, [20000], [150]),
    (128, 12, 4, 256, [40000], [3]), (128, 6, 6, 64, [25000, 300], [140, 300]), (64, 12, 12, 64, [40000], [10]),
    (128, 12, 4, 16, [40000], [9]),
])
def test_long_pieces(d, Hq, Hkv, page, lens, news):
    """A dozen key tiles and several column tiles a piece: every order of the rings, of all remainders."""
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, "bf16", seed=d + lens[0])
    run(cache, q, cu, max(news), max(lens))


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("d,Hq,Hkv,page,news", [
    (64, 8, 8, 16, [8, 1, 3]), (64, 8, 1, 32, [1, 0, 1]), (64, 6, 2, 64, [2, 1, 2]), (128, 16, 1, 16, [1, 1, 0]),
    (128, 8, 2, 256, [4, 2, 3]), (128, 3, 3, 32, [16, 9, 1]), (128, 12, 4, 128, [5, 0, 4]), (128, 6, 6, 64, [7, 8, 1]),
])
def test_few_rows(d, Hq, Hkv, page, news, flags):
    """Up to d / 8 rows a key head over lengths past the one-launch kernel's, with odd ends and pages inside a tile."""
    lens = [5003, 2700, 31]
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, "bf16", seed=d + Hq, junk=float("nan"), pad=2)
    tau = torch.rand(3 * Hq, generator=torch.Generator().manual_seed(3)).mul_(2).to(DEV)
    start = cache.demand_pages.clone()
    out = run(cache, q, cu, max(news), 5003, flags=flags, tau_bh=tau)
    total = cache.demand_pages.clone()
    cache.demand_pages.copy_(start)
    again = b.dilution_attn_paged_chunk(q, cache, cu, max(news), 5003, flags=flags, tau_bh=tau)
    n = int(cu[-1])
    assert torch.equal(out[:n], again[:n]) and torch.equal(cache.demand_pages.view(torch.int32), total.view(torch.int32))


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("d,Hq,Hkv,page,news", [
    (64, 5, 5, 16, [8, 1, 3]), (64, 2, 2, 256, [1, 0, 1]), (128, 3, 3, 32, [4, 8, 2]), (128, 1, 1, 128, [0, 7, 0]),
    (64, 3, 3, 64, [16, 9, 11]), (64, 6, 3, 32, [8, 1, 5]), (128, 4, 2, 16, [3, 8, 0]), (128, 2, 2, 64, [12, 0, 16]),
])
def test_few_rows_in_fp32(d, Hq, Hkv, page, news, flags):
    lens = [5003, 2700, 31]
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, "f32", seed=d + Hq, junk=float("nan"), pad=1)
    run(cache, q, cu, max(news), 5003, flags=flags)


def test_one_workspace_for_all_calls():
    """A workspace sized for long parts serves drafts, single tokens and a padded batch."""
    news = [[130, 70, 200], [4, 3, 1], [1, 1, 1], [5, 4, 5], [2, 0, 4]]
    caches = [make([5000, 2700, 400], n, 6, 3, 64, 32, "bf16", seed=45 + i, pad=i) for i, n in enumerate(news)]
    ws = b.dilution_attn_paged_chunk_workspace(caches[0][0], 412, 200, 5000)
    for (cache, q, cu), n in zip(caches, news):
        start = cache.demand_pages.clone()
        ref = b.dilution_attn_paged_chunk(q, cache, cu, max(n), 5000)
        total = cache.demand_pages.clone()
        cache.demand_pages.copy_(start)
        ws[256:] = 0xC7
        out = b.dilution_attn_paged_chunk(q, cache, cu, max(n), 5000, workspace=ws)
        used = int(cu[-1])
        assert torch.equal(out[:used], ref[:used]) and torch.equal(cache.demand_pages, total)
        assert b.dilution_attn_get_error(ws) == b.DA_OK


def test_few_rows_with_bad_pages():
    lens, news = [2700, 2800, 2650], [2, 3, 1]
    for name in ("page_table", "demand_table"):
        for bad in (-1, 10 ** 9, -2 ** 31):
            cache, q, cu = make(lens, news, 4, 2, 64, 32, "bf16", seed=44)
            ro, rD, info = oracle(cache, q, cu)
            getattr(cache, name)[1, 50:53] = bad
            ws = b.dilution_attn_paged_chunk_workspace(cache, 6, 3, 2800)
            out = b.dilution_attn_paged_chunk(q, cache, cu, 3, 2800, workspace=ws)
            assert b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID
            got = host64(out)
            assert np.abs(got[:2] - ro[:2]).max() < 0.05 and np.abs(got[5:] - ro[5:]).max() < 0.05


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [dict(tau=0.0), dict(tau=2.5), dict(eps=1.0), dict(eps=1e-3, flags=1), dict(flags=1),
                                dict(tau=1.7, eps=1e-15)])
def test_options(kw, dtype):
    cache, q, cu = make([150, 90, 40], [70, 20, 3], 4, 2, 64, 16, dtype, seed=11, fresh=False)
    run(cache, q, cu, 70, 150, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tau_per_head(dtype):
    cache, q, cu = make([150, 90], [70, 20], 4, 2, 64, 16, dtype, seed=12)
    tau = torch.rand(8, generator=torch.Generator().manual_seed(1)).mul_(3).to(DEV)
    run(cache, q, cu, 70, 150, tau_bh=tau)
    tau[3] = float("nan")
    ws = b.dilution_attn_paged_chunk_workspace(cache, q.shape[0], 70, 150)
    b.dilution_attn_paged_chunk(q, cache, cu, 70, 150, tau_bh=tau, workspace=ws)
    assert b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_are_a_decode_step(d, dtype):
    """One new token each: the decode step's definition."""
    lens = [700, 1, 33, 0, 256]
    cache, q, cu = make(lens, [min(1, n) for n in lens], 6, 2, d, 32, dtype, seed=5)
    before = cache.demand_pages.clone()
    qs = torch.zeros(5, 6, d, dtype=q.dtype, device=DEV)
    live = [i for i, n in enumerate(lens) if n]
    qs[live] = q
    ro, rD, _ = oracle_step(cache, qs)
    out = run(cache, q, cu, 1, 700)
    assert np.abs(host64(out) - ro[live]).max() < 0.05 and np.abs(host64(cache.demand_pages) - rD).max() < 1e-5
    cache.demand_pages.copy_(before)
    step = b.dilution_attn_paged_decode(qs, cache, 700)
    assert (out.float() - step[live].float()).abs().max() < 0.05
    torch.testing.assert_close(cache.demand_pages.cpu().double(), torch.tensor(rD), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype,d,T", [("f32", 64, 200), ("bf16", 64, 330), ("bf16", 128, 129)])
def test_whole_prompt_is_the_forward(dtype, d, T):
    """n = length with no demand: dilution_attn_fwd of the prompt, its demand and its heads shared."""
    cache, q, cu = make([T], [T], 4, 2, d, 32, dtype, seed=T)
    at = torch.arange(T, device=DEV)
    pages = cache.page_table[0, at // 32].long()
    k, v = (x[pages, :, at % 32].transpose(0, 1)[None].repeat_interleave(2, 1).contiguous()
            for x in (cache.k_pages, cache.v_pages))
    demand = torch.empty(1, 4, T, device=DEV)
    ref = b.dilution_attn_fwd(q.transpose(0, 1)[None].contiguous(), k, v, demand_out=demand)
    out = run(cache, q, cu, T, T)
    tol = 3e-2 if dtype == "bf16" else 2e-5
    assert (out.transpose(0, 1)[None].float() - ref.float()).abs().max() < tol
    got = cache.demand_pages[cache.demand_table[0, at // 32].long(), :, at % 32].t()[None]
    torch.testing.assert_close(got, demand, rtol=2e-3 if dtype == "bf16" else 1e-5, atol=1e-4 if dtype == "bf16" else 1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_chunks_are_one(dtype):
    """A prompt in two chunks leaves the totals of one chunk; outputs agree with the oracle in both."""
    cache, q, cu = make([300], [300], 2, 2, 64, 64, dtype, seed=21)
    start = cache.demand_pages.clone()
    run(cache, q, cu, 300, 300)
    whole = cache.demand_pages.clone()
    cache.demand_pages.copy_(start)
    for a, e in ((0, 110), (110, 300)):
        cache.seq_lens.fill_(e)
        run(cache, q[a:e].contiguous(), torch.tensor([0, e - a], dtype=torch.int32, device=DEV), 190, 300)
    torch.testing.assert_close(cache.demand_pages, whole, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news,most", [([130, 64, 5], 130), ([20, 30, 5], 32)])
def test_equal_bits_in_place_and_streams(news, most, dtype):
    """Equal calls give equal bits: into q's own place, on another stream, without a workspace, from a graph."""
    cache, q, cu = make([900, 120, 77], news, 4, 2, 64, 32, dtype, seed=31, pad=2)
    start = cache.demand_pages.clone()
    ref = torch.zeros_like(q)
    b.dilution_attn_paged_chunk(q, cache, cu, most, 900, ref)
    total = cache.demand_pages.clone()

    def same(out):
        n = int(cu[-1])
        assert torch.equal(out[:n], ref[:n]) and torch.equal(cache.demand_pages, total)
        cache.demand_pages.copy_(start)
    cache.demand_pages.copy_(start)
    own = q.clone()
    b.dilution_attn_paged_chunk(own, cache, cu, most, 900, own)
    same(own)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = b.dilution_attn_paged_chunk(q, cache, cu, most, 900, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same(out)
    ws = b.dilution_attn_paged_chunk_workspace(cache, q.shape[0], most, 900)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(q)
    with torch.cuda.graph(g):
        b.dilution_attn_paged_chunk(q, cache, cu, most, 900, out, workspace=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        same(out)
    # the captured call follows lengths that change
    cache.seq_lens.copy_(torch.tensor([800, 119, 70], dtype=torch.int32))
    cu.copy_(torch.tensor([0, 3, 30, 30], dtype=torch.int32))
    r = oracle(cache, q, cu)
    g.replay()
    check(cache, q, cu, start, out, r)
    assert b.dilution_attn_get_error(ws) == b.DA_OK and b.dilution_attn_get_error(cache.status) == b.DA_OK


@pytest.mark.parametrize("dtype,mid", [("f32", 70), ("bf16", 70), ("bf16", 30)])
def test_bad_lengths_and_pages(dtype, mid):
    """What the host cannot see: recorded, nothing else read or written, other sequences unharmed.  (Up to 32 new tokens
    take the kernel for short calls.)"""
    lens, news = [100, 200, 150], [20, mid, 5]
    first = np.concatenate([[0], np.cumsum(news)])

    def call(change, max_new=mid, max_len=200, good=(0, 2)):
        cache, q, cu = make(lens, news, 4, 2, 64, 16, dtype, seed=41)
        ro, rD, info = oracle(cache, q, cu)
        start = cache.demand_pages.clone()
        change(cache, cu)
        ws = b.dilution_attn_paged_chunk_workspace(cache, q.shape[0], max_new, max_len)
        out = torch.full_like(q, 7.0)
        b.dilution_attn_paged_chunk(q, cache, cu, max_new, max_len, out, workspace=ws)
        assert b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID
        assert b.dilution_attn_get_error(ws) == b.DA_OK
        for s in good:
            r = slice(first[s], first[s + 1])
            assert np.abs(host64(out)[r] - ro[r]).max() < 0.05
        return cache, out, start

    def set_cu(*values):
        return lambda cache, cu: cu.copy_(torch.tensor(values, dtype=torch.int32))

    def set_at(name, at, value):
        return lambda cache, cu: getattr(cache, name).__setitem__(at, value)
    a, e, N = (int(x) for x in first[1:])
    for bad in (-1, 201, 300, mid - 1):      # the last: shorter than its new tokens
        cache, out, start = call(set_at("seq_lens", 1, bad))
        assert (out[a:e] == 7.0).all()
        t = torch.arange(lens[1], device=DEV)
        at = cache.demand_table[1, t // 16].long(), slice(None), t % 16
        assert torch.equal(cache.demand_pages[at], start[at])
    call(lambda cache, cu: None, max_new=mid - 1)
    for bad in (-1, 10 ** 9, -2 ** 31):
        call(set_at("page_table", (1, 3), bad))
        call(set_at("demand_table", (1, 3), bad))
    call(set_cu(0, a, a - 10, N), good=(0,))
    call(set_cu(0, a, e, N + 4), good=(0, 1))
    call(set_cu(-5, a, e, N), good=(1, 2))
    # tokens counted twice: more rows than there is room for
    cache, q, cu = make([mid] * 4, [mid, 0, 0, 0], 2, 2, 64, 16, dtype, seed=42)
    cu.copy_(torch.tensor([0, mid, 0, mid, 0], dtype=torch.int32))
    ws = b.dilution_attn_paged_chunk_workspace(cache, mid, mid, mid)
    b.dilution_attn_paged_chunk(q, cache, cu, mid, mid, workspace=ws)
    assert b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sharp_and_extreme_logits(dtype):
    """Logits hundreds apart, all far below zero, and the type's largest values in rows past the end."""
    cache, q, cu = make([300, 140], [100, 9], 2, 1, 64, 32, dtype, seed=51, junk=torch.finfo(TYPES[dtype]).max)
    q[:40] *= 30.0
    q[40:60] = -cache.k_pages[cache.page_table[0, 2], 0, 3] * 20.0
    run(cache, q, cu, 100, 300)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,wide", [(33, 0), (33, 70), (128, 70), (129, 70), (1100, 0), (1100, 90), (2500, 40)])
def test_many_sequences(S, wide, dtype):
    """More sequences than a warp's lanes, and than a block's threads, most of them short, some without new tokens."""
    lens = [s * 7 % 23 for s in range(S)]
    news = [min(n, s % 5) for s, n in enumerate(lens)]
    if wide:
        lens[S // 2] = news[S // 2] = wide
    cache, _, _ = make_cache(S, lens, 2, 1, 64, 16, dtype, seed=S + wide, extra_width=8)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = (torch.randn(int(cu[-1]), 2, 64, generator=torch.Generator().manual_seed(2)) * 1.5).to(TYPES[dtype]).to(DEV)
    run(cache, q, torch.tensor(cu, device=DEV), max(news), max(lens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_to_do(dtype):
    """No tokens, no sequence with any, bounds of zero: nothing is written."""
    cache, q, cu = make([50, 0], [0, 0], 2, 2, 64, 16, dtype, seed=61, pad=4)
    before = cache.demand_pages.clone()
    for rows, most, length in ((4, 0, 50), (4, 30, 50), (0, 0, 0), (0, 5, 50), (4, 100, 2600)):
        out = torch.full_like(q[:rows], 7.0)
        ws = b.dilution_attn_paged_chunk_workspace(cache, rows, most, length)
        b.dilution_attn_paged_chunk(q[:rows], cache, cu, most, length, out, workspace=ws)
        assert (out == 7.0).all() and torch.equal(cache.demand_pages, before)
        assert b.dilution_attn_get_error(ws) == b.DA_OK
    # a bound of zero that a sequence passes
    cache, q, cu = make([50, 20], [3, 0], 2, 2, 64, 16, dtype, seed=62)
    out = torch.full_like(q, 7.0)
    ws = b.dilution_attn_paged_chunk_workspace(cache, 3, 0, 50)
    b.dilution_attn_paged_chunk(q, cache, cu, 0, 50, out, workspace=ws)
    assert (out == 7.0).all() and b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_scale_of_a_short_call(dtype):
    cache, q, cu = make([50, 20], [3, 2], 4, 2, 64, 16, dtype, seed=63)
    tau = torch.ones(8, device=DEV)
    tau[6] = float("nan")
    ws = b.dilution_attn_paged_chunk_workspace(cache, 5, 3, 50)
    b.dilution_attn_paged_chunk(q, cache, cu, 3, 50, tau_bh=tau, workspace=ws)
    assert b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_at_once(dtype):
    """Four caches on four streams, long and short calls and evictions in each, against the same calls one by one."""
    shapes = [([3000, 400], [150, 30]), ([500, 60], [5, 1]), ([2500], [4]), ([700, 0, 333], [64, 0, 333])]
    keep = torch.full((3,), 200, dtype=torch.int32, device=DEV)

    def calls(i, stream=None):
        lens, news = shapes[i]
        cache, q, cu = make(lens, news, 4, 2, 64, 32, dtype, seed=70 + i)
        outs = []
        torch.cuda.synchronize()

        def go():
            for _ in range(6):
                outs.append(b.dilution_attn_paged_chunk(q, cache, cu, max(news), max(lens), stream=stream))
            b.dilution_attn_paged_evict(cache, keep[:len(lens)], 200, max(lens), cache.seq_lens, sinks=2, recent=100, stream=stream)
        return go, outs, cache
    ref = [calls(i) for i in range(4)]
    for go, _, _ in ref:
        go()
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [calls(i, streams[i]) for i in range(4)]
    for go, _, _ in got:
        go()
    torch.cuda.synchronize()
    for (_, a, x), (_, c, y) in zip(ref, got):
        assert all(torch.equal(m, n) for m, n in zip(a, c))
        for pool in ("k_pages", "v_pages", "demand_pages", "seq_lens"):
            assert torch.equal(getattr(x, pool), getattr(y, pool))
        assert b.dilution_attn_get_error(y.status) == b.DA_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graphs_that_share_a_workspace(dtype):
    """A long call, a short one and an eviction, each captured with the same workspace, replayed by turns."""
    caches = [make(lens, news, 4, 2, 64, 32, dtype, seed=100 + i)
              for i, (lens, news) in enumerate((([900, 77], [130, 5]), ([300, 40], [4, 1])))]
    keep = torch.tensor([150, 30], dtype=torch.int32, device=DEV)
    third = make([700, 90], [1, 1], 4, 2, 64, 32, dtype, seed=102)[0]

    def calls(outs, ws):
        return [lambda i=i, most=most: b.dilution_attn_paged_chunk(*caches[i][1::-1], caches[i][2], *most, outs[i], workspace=ws)
                for i, most in enumerate(((130, 900), (4, 300)))] + \
               [lambda: b.dilution_attn_paged_evict(third, keep, 150, 700, outs[2], sinks=1, recent=20, workspace=ws)]
    pools = [caches[0][0].demand_pages, caches[1][0].demand_pages, third.demand_pages, third.k_pages, third.v_pages]
    start = [x.clone() for x in pools]

    def reset():
        for x, y in zip(pools, start):
            x.copy_(y)
    outs = lambda: [torch.zeros_like(c[1]) for c in caches] + [torch.zeros(2, dtype=torch.int32, device=DEV)]
    ref = outs()
    for f in calls(ref, None):
        f()
    ref += [x.clone() for x in pools]
    reset()
    ws = max((b.dilution_attn_paged_chunk_workspace(caches[0][0], 135, 130, 900),
              b.dilution_attn_paged_evict_workspace(third, 150, 700)), key=len)
    got, graphs = outs(), []
    for f in calls(got, ws):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for order in ((0, 1, 2), (2, 1, 0), (1, 2, 0)):
        reset()
        for i in order:
            graphs[i].replay()
        assert all(torch.equal(x, y) for x, y in zip(ref, got + pools))
        assert b.dilution_attn_get_error(ws) == b.DA_OK


@pytest.mark.parametrize("d,lens,news", [(64, [9000], [4]), (64, [6000, 100], [140, 3]), (128, [7000], [130])])
def test_long_pieces_repeat_their_bits(d, lens, news):
    cache, q, cu = make(lens, news, 6, 3, d, 64, "bf16", seed=81)
    start, ref = cache.demand_pages.clone(), None
    for _ in range(12):
        cache.demand_pages.copy_(start)
        out = b.dilution_attn_paged_chunk(q, cache, cu, max(news), max(lens))
        now = (out, cache.demand_pages.clone())
        ref = ref or now
        assert torch.equal(now[0], ref[0]) and torch.equal(now[1], ref[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", [([300, 90], [20, 5]), ([700, 90], [130, 5])])
def test_pools_past_32_bits(lens, news, dtype):
    """Pages whose first elements lie past 2^31: the bits of the same cache in a small pool, and of its eviction."""
    cache, q, cu = make(lens, news, 8, 8, 128, 64, dtype, seed=91)
    kv, dem = 2 ** 31 // (8 * 64 * 128), 2 ** 31 // (8 * 64)
    n_kv, n_dem = cache.k_pages.shape[0], cache.demand_pages.shape[0]
    pools = []
    for small, first in ((cache.k_pages, kv), (cache.v_pages, kv), (cache.demand_pages, dem)):
        big = torch.empty((first + small.shape[0] + 1, *small.shape[1:]), dtype=small.dtype, device=DEV)
        big[first:first + small.shape[0]] = small
        pools.append(big)
    shift = lambda t, by: torch.where(t >= 0, t + by, t)
    far = b.PagedCache(*pools, shift(cache.page_table, kv), shift(cache.demand_table, dem), cache.seq_lens.clone())
    keep = torch.tensor([100, 90], dtype=torch.int32, device=DEV)
    for max_len in (max(lens), LONG):
        outs = [b.dilution_attn_paged_chunk(q, c, cu, max(news), max_len) for c in (cache, far)]
        assert torch.equal(*outs)
        assert torch.equal(far.demand_pages[dem:dem + n_dem], cache.demand_pages)
    for c in (cache, far):
        b.dilution_attn_paged_evict(c, keep, 100, max(lens), c.seq_lens, sinks=1, recent=9)
        assert c.seq_lens.tolist() == [100, 90] and b.dilution_attn_get_error(c.status) == b.DA_OK
    for name, first, n in (("k_pages", kv, n_kv), ("v_pages", kv, n_kv), ("demand_pages", dem, n_dem)):
        x, y = getattr(far, name)[first:first + n], getattr(cache, name)
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", [([300, 90], [4, 2]), ([300, 90], [20, 3]), ([700, 90], [130, 5])])
def test_infinite_totals(lens, news, dtype):
    """Keys with an infinite total take part in the softmax and have no share; their totals stay."""
    cache, q, cu = make(lens, news, 4, 2, 64, 32, dtype, seed=95)
    t = torch.arange(5, 60, 3, device=DEV)
    at = cache.demand_table[0, t // 32].long(), slice(None), t % 32
    cache.demand_pages[at] = float("inf")
    cache.demand_pages[cache.demand_table[1, 0].long(), 1, 7] = 3e38
    start = cache.demand_pages.clone()
    with np.errstate(invalid="ignore", over="ignore"):
        ro = oracle(cache, q, cu)[0]
    for max_len in (max(lens), LONG):
        cache.demand_pages.copy_(start)
        out = b.dilution_attn_paged_chunk(q, cache, cu, max(news), max_len)
        assert np.abs(host64(out) - ro).max() < (0.05 if dtype == "bf16" else 1e-4)
        assert (cache.demand_pages[at] == float("inf")).all() and not torch.isnan(cache.demand_pages).any()


def test_serving_run_together():
    """Rotation, append and chunk of ragged prompts, a second chunk behind them, eviction, single tokens and a decode step:
    the calls of a serving loop, each against the oracle on the cache as it then is."""
    torch.manual_seed(0)
    S, Hq, Hkv, d, page, room = 3, 6, 2, 64, 32, 12
    t = torch.bfloat16
    tables = torch.randperm(S * room).to(torch.int32).view(S, room).to(DEV)
    cache = b.PagedCache(torch.zeros(S * room, Hkv, page, d, dtype=t, device=DEV),
                         torch.zeros(S * room, Hkv, page, d, dtype=t, device=DEV),
                         torch.zeros(S * room, Hq, page, device=DEV), tables, tables.flip(0).contiguous(),
                         torch.zeros(S, dtype=torch.int32, device=DEV))
    spec = b.rope_spec(rope_inv_freq(d).to(DEV))
    seen = np.zeros(S, dtype=np.int64)       # tokens so far, evicted ones among them
    lens = np.zeros(S, dtype=np.int64)

    def chunk(news):
        nonlocal lens, seen
        news = np.array(news)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV)
        N = int(cu[-1])
        rows = torch.randn(N, Hq + 2 * Hkv, d, dtype=t, device=DEV)
        pos = np.concatenate([np.arange(seen[s], seen[s] + n) for s, n in enumerate(news)])
        lens, seen = lens + news, seen + news
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q = b.dilution_attn_paged_append(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], cache, cu, rope=spec,
                                         positions=torch.tensor(pos[None], dtype=torch.int32, device=DEV))
        run(cache, q, cu, int(news.max()), int(lens.max()))

    chunk([100, 37, 250])
    chunk([20, 1, 0])
    keep = torch.tensor([64, 64, 64], dtype=torch.int32, device=DEV)
    ref = op.paged_evict(host64(cache.k_pages), host64(cache.v_pages), cache.demand_pages.cpu().numpy(),
                         tables.cpu().numpy(), tables.flip(0).cpu().numpy(), lens, [64] * 3, 64, 4, 16)
    b.dilution_attn_paged_evict(cache, keep, 64, int(lens.max()), cache.seq_lens, sinks=4, recent=16)
    for got, want in zip((cache.k_pages, cache.v_pages, cache.demand_pages), ref):
        assert np.array_equal(host64(got), want.astype(np.float64))
    lens = np.minimum(lens, 64)
    assert cache.seq_lens.tolist() == lens.tolist()
    chunk([1, 1, 1])
    chunk([5, 0, 70])
    q = torch.randn(S, Hq, d, dtype=t, device=DEV)
    before = oracle_step(cache, q)
    out = b.dilution_attn_paged_decode(q, cache, int(lens.max()))
    assert np.abs(host64(out) - before[0]).max() < 0.03
    assert b.dilution_attn_get_error(cache.status) == b.DA_OK
