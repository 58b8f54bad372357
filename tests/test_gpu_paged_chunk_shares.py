"""Drafted and single tokens in bf16: shares of a chunk to 2^-16, as the decode step holds them.

Tolerance (written before any run).  A share goes into the value product as two bf16 terms: what the first leaves is at
most 2^-8 of the share, what the second leaves at most 2^-8 of that, so that a share is off by 2^-16 of itself, a row of
A by at most 2^-15 sum A |v - out| <= 2^-14 max |v|, besides what tests/test_gpu_paged_chunk.py derives for the logits,
the running sums and the exponentials; out itself is rounded, by at most 2^-8 of itself.  Queries are scaled by 2^-6, so
that the logits' share of the tolerance is small beside that of the shares.  (Shares of one bf16 term would be off by
2^-8: on short sequences, where few keys average it, several times this tolerance.)
"""
import numpy as np
import pytest

from long_context_attention_gb300 import binding as b
from tests._parity import host64
from tests._paged import LONG
from tests.test_gpu_paged_chunk import make as make_batch
from tests.test_gpu_paged_chunk import oracle

pytestmark = pytest.mark.gpu


def make(*args, **kw):
    cache, q, cu = make_batch(*args, **kw)
    return cache, q * 2.0 ** -6, cu


def check_two_terms(out, cu, ref, rows=None):
    ro, _, info = ref
    n, d = int(cu[-1]), out.shape[-1]
    news = np.diff(cu.cpu().numpy())
    per_row = np.repeat(news, news)[:, None]
    g = (2 * d + 8) * 2.0 ** -24 * info["spread"][:n]
    e = ((2 * (4 * g + per_row * 2.0 ** -24 + 2.0 ** -19) + 2.0 ** -14) * info["vmax"][:n])[..., None]
    err = np.abs(host64(out)[:n] - ro[:n]) - (e + 2.0 ** -8 * (np.abs(ro[:n]) + e))
    pick = slice(None) if rows is None else rows
    assert (err[pick] <= 0).all(), float(err[pick].max())


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("d,Hq,Hkv,page,lens,news", [
    (64, 4, 4, 16, [9, 30, 41], [4, 1, 8]), (64, 6, 2, 32, [12, 27, 500], [1, 2, 1]), (128, 16, 1, 16, [20, 33], [1, 1]),
    (128, 8, 2, 64, [17, 40, 70], [4, 2, 3]), (128, 2, 2, 256, [25, 64], [16, 9]), (128, 12, 4, 32, [9, 300], [5, 5]),
])
def test_drafts(d, Hq, Hkv, page, lens, news, flags):
    """Calls of few rows, by the kernel for short calls and by the one that keeps its logits."""
    for max_len in (max(lens), LONG):
        cache, q, cu = make(lens, news, Hq, Hkv, d, page, "bf16", seed=d + Hq)
        ref = oracle(cache, q, cu, earlier=bool(flags))
        out = b.dilution_attn_paged_chunk(q, cache, cu, max(news), max_len, flags=flags)
        check_two_terms(out, cu, ref)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (64, 8, 1), (128, 4, 2), (128, 8, 1)])
def test_short_calls_of_many_rows(d, Hq, Hkv):
    """The kernel for short calls, up to its 64 rows."""
    n = 64 // (Hq // Hkv)
    cache, q, cu = make([n + 5, 7, n], [n, 7, n - 3], Hq, Hkv, d, 32, "bf16", seed=d + Hq)
    ref = oracle(cache, q, cu)
    check_two_terms(b.dilution_attn_paged_chunk(q, cache, cu, n, n + 5), cu, ref)


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 3, 3, 16), (64, 8, 1, 64), (128, 3, 1, 32), (128, 8, 2, 128)])
def test_mixed_batch(d, Hq, Hkv, page, flags):
    """Beside a part of a prompt: sequences of up to 64 rows a key head, n rounded up to 8 for each query head."""
    G = Hq // Hkv
    few = 64 // G // 8 * 8
    lens, news = [200, 9, 150, 20, few + 3, 30, 2600], [130, 1, 3, 5, few, 8, 2]
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, "bf16", seed=d + Hq)
    ref = oracle(cache, q, cu, earlier=bool(flags))
    out = b.dilution_attn_paged_chunk(q, cache, cu, 130, 2600, flags=flags)
    check_two_terms(out, cu, ref, slice(130, int(cu[-1])))
    assert np.abs(host64(out) - ref[0]).max() < 0.05     # the part's too


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(64, 12, 1, 16), (64, 16, 1, 64), (128, 20, 1, 32), (128, 34, 2, 128), (64, 3, 3, 32)])
@pytest.mark.parametrize("part", [0, 130])
def test_many_heads_on_a_key_head(d, Hq, Hkv, page, part, flags):
    """Up to four new tokens, however many query heads share their keys: alone, and beside a part of a prompt."""
    lens, news = [9, 150, 20, 2600, 33, 200], [1, 3, 4, 2, 1, part]
    cache, q, cu = make(lens, news, Hq, Hkv, d, page, "bf16", seed=d + Hq)
    ref = oracle(cache, q, cu, earlier=bool(flags))
    out = b.dilution_attn_paged_chunk(q, cache, cu, max(news), 2600, flags=flags)
    check_two_terms(out, cu, ref, slice(0, 11))
    assert np.abs(host64(out) - ref[0]).max() < 0.05


def test_a_single_token_is_as_exact_as_a_decode_step():
    """The same token by a chunk, alone and beside a prompt, and by a decode step: errors of one size."""
    lens, news = [33, 12, 60], [1, 1, 1]
    cache, q, cu = make(lens, news, 4, 2, 64, 16, "bf16", seed=6)
    start = cache.demand_pages.clone()
    ref = oracle(cache, q, cu)
    step = b.dilution_attn_paged_decode(q, cache, 60)
    check_two_terms(step, cu, ref)
    for max_len in (60, LONG):
        cache.demand_pages.copy_(start)
        check_two_terms(b.dilution_attn_paged_chunk(q, cache, cu, 1, max_len), cu, ref)
