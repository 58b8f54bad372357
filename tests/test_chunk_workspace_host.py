"""Workspace sizes of chunks over the paged cache: bounded for long parts, and enough for every smaller call."""
import pytest

from long_context_attention_gb300 import binding as b


@pytest.fixture(scope="module")
def size():
    b.load()
    return b.dilution_attn_paged_chunk_workspace_size


@pytest.mark.parametrize("dtype,most", [(1, 1.0e9), (0, 1.6e9)])
@pytest.mark.parametrize("d", [64, 128])
def test_long_prompts(size, d, dtype, most):
    """One prompt, however long: about what its forward takes, not places for all of it in every CTA.  (bf16: beside the
    logits that calls of few rows keep, up to 2 GB.)"""
    for hkv in (4, 12):
        for S in (1, 2, 16):
            for n in (1 << 14, 1 << 17, 1 << 20, 1 << 30):
                logits = min(1 << 31, S * (d // 8 // (12 // hkv)) * 12 * n * 4) if dtype == 1 else 0
                own = S * (8192 + 8) * 12 * 4 * (d + 8)      # the rows' own places
                assert 0 < size(S, 12, hkv, d, S * n if S * n <= 1 << 30 else 1 << 30, n, n, dtype) < most + logits + own


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("hq,hkv", [(12, 12), (12, 4), (16, 1), (6, 3), (5, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_every_smaller_call_fits(size, d, hq, hkv, dtype):
    """The number of CTAs, and so of places, depends on max_new: the size for a bound covers every bound below it."""
    for S in (1, 3, 40):
        for length in (500, 5000, 131072):
            sizes = [size(S, hq, hkv, d, 4000, n, length, dtype) for n in list(range(0, 71)) + [127, 128, 129, 1000, 4000]]
            assert sizes == sorted(sizes), (S, length)
            for n in (3, 8, 17, 64, 70):
                by_tokens = [size(S, hq, hkv, d, N, n, length, dtype) for N in (1, 2, 7, 8, 9, 63, 64, 65, 500, 4000)]
                assert by_tokens == sorted(by_tokens), (S, length, n)
        by_length = [size(S, hq, hkv, d, 4000, 16, L, dtype) for L in (1, 127, 128, 129, 500, 2048, 2049, 5000, 131072, 1 << 20)]
        assert by_length == sorted(by_length)
