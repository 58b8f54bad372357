"""Chunks over long sequences, long parts and shared pages against 64 bits, and one workspace for all calls of a type.
Tolerances: those of tests/test_gpu_paged_chunk.py."""
import numpy as np
import pytest
import torch

from long_context_attention_gb300 import binding as b
from oracle import paged as op
from tests._parity import host64
from tests._paged import DEV, make_cache
from tests._paged_long import chunk64
from tests.test_gpu_paged_chunk import check, make, oracle, run

pytestmark = pytest.mark.gpu


def run_long(cache, q, cu, max_new, max_len, **kw):
    before = cache.demand_pages.clone()
    ref = chunk64(cache, q, cu, earlier=bool(kw.get("flags", 0)))
    ws = b.dilution_attn_paged_chunk_workspace(cache, q.shape[0], max_new, max_len)
    ws[256:] = 0xC7
    out = b.dilution_attn_paged_chunk(q, cache, cu, max_new, max_len, workspace=ws, **kw)
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    check(cache, q, cu, before, out, ref)
    return out


def test_the_two_oracles_agree():
    cache, q, cu = make([150, 40], [70, 3], 4, 2, 64, 16, "f32", seed=1, fresh=False)
    for earlier in (False, True):
        (o1, d1, i1), (o2, d2, i2) = oracle(cache, q, cu, earlier=earlier), chunk64(cache, q, cu, earlier=earlier, block=32)
        assert np.abs(o1 - o2).max() < 1e-12 and np.abs(d1 - d2).max() < 1e-12
        assert np.abs(i1["spread"] - i2["spread"]).max() < 1e-12 and np.abs(i1["dev2"] - i2["dev2"]).max() < 1e-6
        assert (i1["dev"] <= i2["dev"] + 1e-9).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,Hq,Hkv,lens,news", [
    (64, 2, 2, [131072], [4]), (64, 2, 1, [131072, 100], [150, 20]), (128, 4, 2, [131071], [3]), (128, 2, 2, [100001, 131072], [129, 1]),
    (64, 3, 3, [120000], [300]),
])
def test_long_contexts(d, Hq, Hkv, lens, news, dtype):
    cache, q, cu = make(lens, news, Hq, Hkv, d, 64, dtype, seed=d + sum(news))
    run_long(cache, q, cu, max(news), max(lens), flags=news[0] % 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,lens,news", [
    (64, [8400, 61], [8400, 40]), (128, [9000], [8193]), (64, [8250, 17000, 8192], [8192, 16500, 8192]),
])
def test_long_parts(d, lens, news, dtype):
    """More new tokens of a sequence than are walked at once, beside ones with fewer."""
    cache, q, cu = make(lens, news, 2, 1, d, 64, dtype, seed=d + sum(news), pad=5)
    out = run_long(cache, q, cu, max(news) + 3, max(lens))
    start = torch.zeros_like(out)
    # into q's own place, by equal bits (the demand is the call's own by now: twice from the same totals)
    held = cache.demand_pages.clone()
    b.dilution_attn_paged_chunk(q, cache, cu, max(news) + 3, max(lens), start)
    cache.demand_pages.copy_(held)
    own = q.clone()
    b.dilution_attn_paged_chunk(own, cache, cu, max(news) + 3, max(lens), own)
    n = int(cu[-1])
    assert torch.equal(own[:n], start[:n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,news", [([300, 140], [4, 2]), ([500, 300, 129], [70, 100, 1]), ([333, 257], [20, 33])])
def test_shared_pages(lens, news, dtype):
    """Keys and values of a prefix in pages that the sequences share, each with totals of its own."""
    cache, _, _ = make_cache(len(lens), lens, 4, 2, 64, 64, dtype, seed=17, prefix=128)
    assert (cache.page_table[:, 0] == cache.page_table[0, 0]).all()
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = (torch.randn(int(cu[-1]), 4, 64, generator=torch.Generator().manual_seed(3)) * 1.5).to(cache.dtype).to(DEV)
    run(cache, q, torch.tensor(cu, device=DEV), max(news), max(lens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (4, 2), (6, 2)])
def test_a_workspace_for_every_smaller_call(Hq, Hkv, d, dtype):
    """Of exactly the size for one set of bounds, filled with what an earlier call may leave: every smaller call fits."""
    bounds = [(412, 200, 5000), (60, 24, 5000), (48, 17, 5000), (48, 16, 5000)]
    calls = [[130, 70, 200], [24, 3, 20], [17, 9, 1], [16, 16, 16], [15, 2, 0], [8, 8, 8], [4, 3, 1], [1, 1, 1], [0, 5, 2]]
    for N, most, length in bounds:
        fit = [n for n in calls if sum(n) <= N and max(n) <= most]
        assert fit
        for i, news in enumerate(fit):
            cache, q, cu = make([5000, 2700, 400], news, Hq, Hkv, d, 32, dtype, seed=45 + i, pad=i % 3)
            if q.shape[0] > N:
                q = q[:N].contiguous()
            start = cache.demand_pages.clone()
            ref = b.dilution_attn_paged_chunk(q, cache, cu, max(news), length)
            total = cache.demand_pages.clone()
            size = b.dilution_attn_paged_chunk_workspace_size(3, Hq, Hkv, d, N, most, length, cache._code)
            ws = torch.full((size + 512,), 0xC7, dtype=torch.uint8, device=DEV)
            ws[:256] = 0
            cache.demand_pages.copy_(start)
            out = b.dilution_attn_paged_chunk(q, cache, cu, max(news), length, workspace=ws[:size])
            used = int(cu[-1])
            assert torch.equal(out[:used], ref[:used]) and torch.equal(cache.demand_pages, total)
            assert (ws[size:] == 0xC7).all() and b.dilution_attn_get_error(ws[:size]) == b.DA_OK


def test_oracle_pin():
    """A chunk is decode steps, in the writing that the long tests use."""
    cache, q, cu = make([70], [3], 2, 1, 64, 32, "f32", seed=2)
    out, D, _ = chunk64(cache, q, cu)
    total = host64(cache.demand_pages)
    for i in range(3):
        o, total, _ = op.paged_decode(host64(q[i:i + 1]), host64(cache.k_pages), host64(cache.v_pages), total,
                                      cache.page_table.cpu().numpy(), cache.demand_table.cpu().numpy(), [68 + i], 1.0, 1e-6)
        assert np.abs(o[0] - out[i]).max() < 1e-12
    assert np.abs(total - D).max() < 1e-12
