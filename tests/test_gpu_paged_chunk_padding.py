"""Batches padded to a captured graph's size: the kernels, and so the bits, are those of the batch without padding."""
import pytest
import torch

from long_context_attention_gb300 import binding as b
from tests.test_gpu_paged_chunk import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hkv,news", [(64, 4, 4, [4, 1, 3]), (64, 8, 1, [1, 0, 1]), (128, 6, 2, [5, 2, 0]), (128, 3, 3, [16, 9, 1])])
@pytest.mark.parametrize("pad", [40, 700])
def test_padded_few_rows(d, Hq, Hkv, news, pad):
    lens = [5003, 2700, 31]
    cache, q, cu = make(lens, news, Hq, Hkv, d, 64, "bf16", seed=d + pad, junk=float("nan"), pad=pad)
    start, n = cache.demand_pages.clone(), int(cu[-1])
    out = run(cache, q, cu, max(news), 5003)
    total = cache.demand_pages.clone()
    cache.demand_pages.copy_(start)
    ref = b.dilution_attn_paged_chunk(q[:n].contiguous(), cache, cu, max(news), 5003)
    assert torch.equal(out[:n], ref) and torch.equal(cache.demand_pages.view(torch.int32), total.view(torch.int32))


def test_padded_and_captured():
    """One graph of a fixed size follows the batch; its workspace is that of the padded bounds."""
    cache, q, cu = make([5003, 2700, 31], [4, 2, 3], 6, 3, 64, 32, "bf16", seed=3, pad=119)
    start = cache.demand_pages.clone()
    ws = b.dilution_attn_paged_chunk_workspace(cache, 128, 4, 5003)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.dilution_attn_paged_chunk(q, cache, cu, 4, 5003, out, workspace=ws)
    for news, lens in (([4, 2, 3], [5003, 2700, 31]), ([1, 0, 4], [4000, 0, 30]), ([0, 4, 0], [5003, 2690, 31])):
        cu.copy_(torch.tensor([0, news[0], news[0] + news[1], sum(news)], dtype=torch.int32))
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cache.demand_pages.copy_(start)
        ref = b.dilution_attn_paged_chunk(q[:sum(news)].contiguous(), cache, cu, 4, 5003)
        total = cache.demand_pages.clone()
        cache.demand_pages.copy_(start)
        out.fill_(7.0)
        g.replay()
        assert torch.equal(out[:sum(news)], ref) and (out[sum(news):] == 7.0).all()
        assert torch.equal(cache.demand_pages.view(torch.int32), total.view(torch.int32))
        assert b.dilution_attn_get_error(ws) == b.DA_OK
