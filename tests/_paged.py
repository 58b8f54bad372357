"""Shared helpers of the paged-cache tests: random caches and the derived tolerances.

Tolerances of a decode step (written before any run):
  A logit is a dot product of d terms summed in fp32; its error is at most
  g = (2 d + 8) 2^-24 sum |q_i k_i| tau / sqrt(d) (twice the usual bound, since
  tensor cores may truncate partial sums; 8 for the scale and the exponential's
  argument).  A bid then is off by a factor 1 +- 2 g (numerator and
  normaliser), a share by as much (its denominator D + p + eps moves less), a
  row of A by 4 g, so |d out| <= 4 g max|v|, plus
    fp32: 2^-20 max|v| (exponential, division and the sums),
    bf16: 2^-14 max|v| (shares enter the products as two bf16 terms, 2^-16
          relative) and half a step of the output, 2^-8 |out|.
  The new demand D + p is off by p (2 g + 2^-20) and half a step, 2^-24 (D + p).
"""
import numpy as np
import torch

from long_context_attention_gb300 import binding as b
from oracle import paged as op
from tests._parity import host64

DEV = "cuda"
LONG = 2600     # a max_len past what the one-launch kernel for short bf16 calls takes
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make_cache(S, lens, Hq, Hkv, d, page, dtype, seed=0, prefix=0, spare=2, extra_width=None, junk=None):
    """A random paged cache; pages in shuffled order, unused table entries -1.
    The tables are wide enough for LONG tokens unless extra_width is given.
    ``prefix`` tokens (whole pages) are shared by every sequence.  ``junk``
    fills the rows past each sequence's end (keys, values and demand)."""
    g = torch.Generator().manual_seed(seed)
    lens = list(lens)
    pp = prefix // page
    need = [-(-n // page) for n in lens]
    width = max(need + [pp]) + (-(-LONG // page) if extra_width is None else extra_width)
    n_kv = pp + sum(max(0, n - pp) for n in need) + spare
    n_dem = sum(need) + spare
    order = torch.randperm(n_kv, generator=g).to(torch.int32)
    dorder = torch.randperm(n_dem, generator=g).to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32)
    dtable = torch.full((S, width), -1, dtype=torch.int32)
    at, dat = pp, 0
    for s, n in enumerate(need):
        if n == 0:
            continue
        table[s, :pp] = order[:pp]
        table[s, pp:n] = order[at:at + n - pp]
        dtable[s, :n] = dorder[dat:dat + n]
        at, dat = at + n - pp, dat + n
    t = TYPES[dtype]
    k = torch.randn(n_kv, Hkv, page, d, generator=g).to(t)
    v = torch.randn(n_kv, Hkv, page, d, generator=g).to(t)
    dem = -torch.log(torch.rand(n_dem, Hq, page, generator=g).clamp_min(1e-6))
    if junk is not None:
        for s, n in enumerate(lens):
            if n % page:
                pg, dpg = int(table[s, n // page]), int(dtable[s, n // page])
                k[pg, :, n % page:], v[pg, :, n % page:], dem[dpg, :, n % page:] = junk, junk, junk
    q = (torch.randn(S, Hq, d, generator=g) * 1.5).to(t)
    host = dict(k_pages=k, v_pages=v, demand_pages=dem, page_table=table, demand_table=dtable,
                seq_lens=torch.tensor(lens, dtype=torch.int32))
    dev = {n: x.to(DEV) for n, x in host.items()}
    prefix_table = order[:pp].clone().to(DEV) if pp else None
    return b.PagedCache(**dev), q.to(DEV), prefix_table


def oracle_step(cache, q, tau=1.0, eps=1e-6, earlier=False, prefix_table=None):
    """The float64 step on the cache as it is now."""
    with np.errstate(invalid="ignore"):
        return op.paged_decode(host64(q), host64(cache.k_pages), host64(cache.v_pages), host64(cache.demand_pages),
                               cache.page_table.cpu().numpy(), cache.demand_table.cpu().numpy(),
                               cache.seq_lens.cpu().numpy(), tau, eps, earlier,
                               None if prefix_table is None else prefix_table.cpu().numpy())


def check_step(cache, q, before, out, ref):
    """out and the cache's demand against the oracle; demand outside the sequences is untouched."""
    ro, rD, info = ref
    got, d = host64(out), q.shape[-1]
    bf16 = out.dtype == torch.bfloat16
    g = (2 * d + 8) * 2.0 ** -24 * info["spread"]
    tol = (4 * g + (2.0 ** -14 if bf16 else 2.0 ** -20)) * info["vmax"]
    tol = tol[..., None] + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(ro)
    assert np.isfinite(got).all()
    assert (np.abs(got - ro) <= tol).all(), float((np.abs(got - ro) - tol).max())
    D, page = host64(cache.demand_pages), cache.page_size
    dt = cache.demand_table.cpu().numpy()
    seen = np.zeros(D.shape, dtype=bool)
    for (s, h), p in info["bids"].items():
        t = np.arange(len(p))
        at = (dt[s][t // page], h, t % page)
        seen[at] = True
        bound = p * (2 * g[s, h] + 2.0 ** -20) + 2.0 ** -24 * rD[at] + 1e-30
        assert (np.abs(D[at] - rD[at]) <= bound).all(), (s, h, float((np.abs(D[at] - rD[at]) - bound).max()))
    old = host64(before)
    assert np.array_equal(D[~seen], old[~seen], equal_nan=True)


def both_sizes(cache, q, max_len, **kw):
    """The step with max_len and with a max_len that takes the kernels for long caches."""
    old = cache.demand_pages.clone()
    step_and_check(cache, q, max_len, **kw)
    cache.demand_pages.copy_(old)
    return step_and_check(cache, q, max(max_len, LONG), **kw)


def step_and_check(cache, q, max_len, **kw):
    prefix_table = kw.get("prefix_table")
    tau_bh = kw.get("tau_bh")
    tau = kw.get("tau", 1.0) if tau_bh is None else host64(tau_bh).reshape(cache.S, cache.Hq)
    before = cache.demand_pages.clone()
    ref = oracle_step(cache, q, tau, kw.get("eps", 1e-6), bool(kw.get("flags", 0) & b.DA_FLAG_EARLIER_DEMAND_ONLY),
                      prefix_table)
    ws = kw.pop("workspace", None)
    if ws is None:
        ws = b.dilution_attn_paged_decode_workspace(cache, max_len)
        ws[256:] = 0xC7          # whatever an earlier call left
    out = b.dilution_attn_paged_decode(q, cache, max_len, workspace=ws, **kw)
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    check_step(cache, q, before, out, ref)
    return out
