"""Chunks and evictions of long sequences in 64 bits on the GPU, vectorised over rows, and checks against them.

`chunk64` is oracle.paged.paged_chunk in another writing; instead of sums of A |v - out| it gives the bound
sqrt(sum A (v - out)^2) (Jensen's inequality), so that tests.test_gpu_paged_chunk.check holds with it.
"""
import numpy as np
import torch

from tests._parity import host64
from tests._paged import DEV


def chunk64(cache, q, cu, tau=1.0, eps=1e-6, earlier=False, block=512):
    N, Hq, d = q.shape
    G, page = Hq // cache.Hkv, cache.page_size
    out = torch.zeros(N, Hq, d, dtype=torch.float64, device=DEV)
    D = cache.demand_pages.double()
    info = {"dev": torch.zeros_like(out), "dev2": torch.zeros_like(out), "bids": {}}
    for name in ("spread", "vmax"):
        info[name] = torch.zeros(N, Hq, dtype=torch.float64, device=DEV)
    cu = cu.tolist()
    for s, n in enumerate(cache.seq_lens.tolist()):
        a, e = cu[s], cu[s + 1]
        if a == e:
            continue
        t = torch.arange(n, device=DEV)
        pg, dpg, row = cache.page_table[s][t // page].long(), cache.demand_table[s][t // page].long(), t % page
        for h in range(Hq):
            k, v = cache.k_pages[pg, h // G, row].double(), cache.v_pages[pg, h // G, row].double()
            total = D[dpg, h, row]
            first = total.clone()
            for i in range(a, e, block):
                j = min(i + block, e)
                qs = q[i:j, h].double()
                place = torch.arange(n - e + i, n - e + j, device=DEV)[:, None]
                seen = t[None] <= place
                p = torch.softmax((qs @ k.T * (tau / d ** 0.5)).masked_fill(~seen, -np.inf), 1)
                after = total + p.cumsum(0)
                share = p / ((after - p if earlier else after) + eps)
                total = after[-1]
                A = share / share.sum(1, keepdim=True)
                o = A @ v
                out[i:j, h] = o
                info["dev"][i:j, h] = (A @ (v * v) - o * o).clamp_min(0).sqrt()
                A2 = A * A
                info["dev2"][i:j, h] = (A2 @ (v * v) - 2 * o * (A2 @ v) + o * o * A2.sum(1, keepdim=True)).clamp_min(0).sqrt()
                info["spread"][i:j, h] = (qs.abs() @ k.abs().T).masked_fill(~seen, 0).amax(1) * tau / d ** 0.5
                info["vmax"][i:j, h] = v.abs().max()
            D[dpg, h, row] = total
            info["bids"][s, h] = (total - first).cpu().numpy()
    cast = lambda x: x.cpu().numpy() if torch.is_tensor(x) else x
    return cast(out), cast(D), {n: cast(x) for n, x in info.items()}


def evict64(cache, lens, keeps, max_keep, sinks=0, recent=0, to=None):
    """oracle.paged.paged_evict with a stable sort of all scores at once, on the host."""
    K, V = host64(cache.k_pages), host64(cache.v_pages)
    D = cache.demand_pages.cpu().numpy()
    K2, V2, D2 = K.copy(), V.copy(), D.copy()
    table, dtable = (x.cpu().numpy() for x in (cache.page_table, cache.demand_table))
    to, dto = (table, dtable) if to is None else (x.cpu().numpy() for x in to)
    G, page = cache.Hq // cache.Hkv, cache.page_size
    new_lens, kept = np.minimum(lens, keeps), np.full((len(lens), cache.Hkv, max_keep), -1, np.int32)
    for s, n in enumerate(lens):
        m, t = int(new_lens[s]), np.arange(n)
        pg, dpg, row = table[s][t // page], dtable[s][t // page], t % page
        r = np.arange(m)
        tpg, tdpg, trow = to[s][r // page], dto[s][r // page], r % page
        for h in range(cache.Hkv):
            score = D[dpg, h * G, row]
            for g in range(1, G):
                score = (score + D[dpg, h * G + g, row]).astype(np.float32)
            score = np.where(np.isnan(score) | (t < sinks) | (t >= n - recent), np.float32(np.inf), score)
            stay = np.sort(np.argsort(-score, kind="stable")[:m])
            kept[s, h, :m] = stay
            K2[tpg, h, trow], V2[tpg, h, trow] = K[pg[stay], h, row[stay]], V[pg[stay], h, row[stay]]
            for g in range(h * G, (h + 1) * G):
                D2[tdpg, g, trow] = D[dpg[stay], g, row[stay]]
    return K2, V2, D2, new_lens, kept
