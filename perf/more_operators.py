"""Cases of prompts and chunks over the paged cache and of its eviction: what each call computes in plain torch, and its cost.

Operators
  chunk   dilution attention of the new tokens of a ragged batch over the paged cache: each sequence's last n tokens are
          the queries, from one (a decode step) over a few (drafts to be verified) and parts of a long prompt to whole
          prompts (n is the length); every key's demand grows by the bids it receives
  evict   the keys with the most demand stay, per sequence and key head, with the first and the latest tokens; the rows
          that stay move together, in place or to other pages
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ----------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # five drafted tokens of one short chat, to be verified: latency
        dict(name="chunk_drafts_1x500", op="chunk", S=1, Hq=12, Hkv=12, d=64, page=16, dtype="bf16", lo=500, hi=500,
             new_lo=5, new_hi=5, idle=False),
        # four drafted tokens of each of eight long contexts: the cache is read for little work
        dict(name="chunk_drafts_8x131072", op="chunk", S=8, Hq=12, Hkv=12, d=64, page=64, dtype="bf16", lo=131072,
             hi=131072, new_lo=4, new_hi=4, idle=False),
        # a scheduler's mixed batch: single tokens beside parts of prompts, keys shared by three heads, idle slots
        dict(name="chunk_mixed_48", op="chunk", S=48, Hq=12, Hkv=4, d=128, page=32, dtype="bf16", lo=70, hi=16384,
             new_lo=1, new_hi=512, idle=True),
        # 16 whole prompts of different lengths, packed one behind the other
        dict(name="chunk_prompts_16", op="chunk", S=16, Hq=12, Hkv=4, d=128, page=32, dtype="bf16", lo=37, hi=8191,
             new_lo=8191, new_hi=8191, idle=False),
        # the next 2048 tokens of a prompt at the long-context length
        dict(name="chunk_part_2048_at_131072", op="chunk", S=1, Hq=12, Hkv=12, d=64, page=64, dtype="bf16", lo=131072,
             hi=131072, new_lo=2048, new_hi=2048, idle=False),
        # eight parts of 128 tokens, four query heads on a key head
        dict(name="chunk_parts_8x128", op="chunk", S=8, Hq=16, Hkv=4, d=128, page=64, dtype="bf16", lo=1001, hi=32768,
             new_lo=128, new_hi=128, idle=False),
        # the fp32 type: odd parts of medium contexts
        dict(name="chunk_f32_4", op="chunk", S=4, Hq=12, Hkv=12, d=64, page=32, dtype="f32", lo=1001, hi=8001, new_lo=3,
             new_hi=301, idle=False),
        # one short chat that has reached its budget: latency
        dict(name="evict_one_500", op="evict", S=1, Hq=12, Hkv=12, d=64, page=16, dtype="bf16", lo=500, hi=500,
             budget=0.5, sinks=4, recent=64, idle=False, place=True),
        # a full batch in the steady state: one key out for every new token
        dict(name="evict_steady_64", op="evict", S=64, Hq=12, Hkv=4, d=128, page=32, dtype="bf16", lo=4097, hi=4097,
             budget=4096 / 4097, sinks=4, recent=256, idle=False, place=True),
        # a ragged batch cut down to a third, idle slots, to pages of its own (the old ones are shared)
        dict(name="evict_ragged_48", op="evict", S=48, Hq=12, Hkv=4, d=128, page=32, dtype="bf16", lo=1, hi=16384,
             budget=0.33, sinks=0, recent=33, idle=True, place=False),
        # long contexts down to a quarter
        dict(name="evict_long_4x131072", op="evict", S=4, Hq=12, Hkv=4, d=128, page=64, dtype="bf16", lo=131072,
             hi=131072, budget=0.25, sinks=16, recent=1024, idle=False, place=True),
        # the fp32 type, medium lengths
        dict(name="evict_f32_4", op="evict", S=4, Hq=12, Hkv=12, d=64, page=32, dtype="f32", lo=4001, hi=16001,
             budget=0.6, sinks=1, recent=100, idle=False, place=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw_once(rng):
    hkv, group = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 1, 2, 3, 4, 8])
    hi = _log_int(rng, 1, 131072)
    case = dict(op=rng.choice(["chunk", "chunk", "evict"]), S=_log_int(rng, 1, 64), Hq=hkv * group, Hkv=hkv,
                d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                lo=_log_int(rng, 1, hi), hi=hi, idle=rng.random() < 0.3)
    if case["op"] == "chunk":
        new_hi = hi if rng.random() < 0.25 else _log_int(rng, 1, min(hi, 4096))   # whole prompts, or their ends
        return dict(case, new_hi=new_hi, new_lo=new_hi if rng.random() < 0.5 else _log_int(rng, 1, new_hi))
    return dict(case, budget=rng.uniform(0.05, 1.0), sinks=rng.choice([0, 0, 1, 4, 37]), recent=_log_int(rng, 1, 1024) - 1,
                place=rng.random() < 0.5)


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_, flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        case = _draw_once(rng)
        cost = work(case)
        if cost["bytes"] <= bytes_ and cost["flops"] <= flops:
            return case


def _spread(S, lo, hi):
    """S whole numbers from lo to hi, spread evenly over their logarithm."""
    n = [int(round(lo * (hi / lo) ** (i / max(1, S - 1)))) if lo < hi else hi for i in range(S)]
    return n[:-1] + [hi]


def _lens(case):
    """The sequences' lengths, before they are shuffled."""
    lens = _spread(case["S"], case["lo"], case["hi"])
    return [0 if case["idle"] and i % 8 == 3 else n for i, n in enumerate(lens)]


def _news(case):
    """How many tokens of each are new: short and long parts at every length."""
    S, lens = case["S"], _lens(case)
    news = _spread(S, case["new_lo"], case["new_hi"])
    return [min(n, news[(7 * i + 3) % S]) for i, n in enumerate(lens)]


def _keeps(case):
    """How many keys each sequence may keep."""
    return [int(round(case["budget"] * n)) if n != 1 else 1 for n in _lens(case)]


def work(case):
    """chunk: every key, value and total once, two products a visible pair.  evict: every total read once, the rows that
    stay (but for the first tokens, which lie where they were) read and written."""
    d, e, hq, hkv = case["d"], 2 if case["dtype"] == "bf16" else 4, case["Hq"], case["Hkv"]
    lens = _lens(case)
    if case["op"] == "evict":
        kept = sum(min(n, k) - (min(case["sinks"], n, k) if case["place"] else 0) for n, k in zip(lens, _keeps(case)))
        return {"bytes": 4 * hq * sum(lens) + 2 * kept * (2 * hkv * d * e + 4 * hq) + 4 * hkv * kept,
                "flops": hq * sum(lens)}
    news = _news(case)
    held = sum(n for n, m in zip(lens, news) if m > 0)
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, news))
    return {"bytes": 2 * held * hkv * d * e + 8 * held * hq + 2 * sum(news) * hq * d * e, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------------------------------------- the inputs
def _randn(g, *shape, std=1.0, dtype=torch.float32):
    """Normal values, rounded once to `dtype`."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 28) // max(1, flat.shape[1]))      # rows at a time: a pool is as large as memory lets it
    for i in range(0, shape[0], step):
        flat[i:i + step] = torch.randn(flat[i:i + step].shape, generator=g, device=DEV) * std
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, S, page, d, hq, hkv = TYPES[case["dtype"]], *(case[x] for x in ("S", "page", "d", "Hq", "Hkv"))
    order = torch.randperm(S, generator=g, device=DEV).tolist()
    mix = lambda xs: [xs[i] for i in order]
    lens = mix(_lens(case))
    moves = case["op"] == "evict" and not case["place"]
    keeps = mix(_keeps(case)) if case["op"] == "evict" else None
    need = [-(-n // page) for n in lens]
    more = [-(-min(n, k) // page) for n, k in zip(lens, keeps)] if moves else [0] * S
    width, width2 = max(need) + 1, max(more) + 1
    pages = sum(need) + sum(more) + 2
    # pages in random order, entries past a sequence's end -1
    ids, dids = (torch.randperm(pages, generator=g, device=DEV).cpu().to(torch.int32) for _ in range(2))
    tables = [torch.full((S, w), -1, dtype=torch.int32) for w in (width, width, width2, width2)]
    at = 0
    for s in range(S):
        for n, (a, b) in ((need[s], tables[:2]), (more[s], tables[2:])):
            a[s, :n], b[s, :n] = ids[at:at + n], dids[at:at + n]
            at += n
    page_table, demand_table, dst_page_table, dst_demand_table = (x.to(DEV) for x in tables)
    # about one unit of demand a key, with the heavy tail that earlier queries leave
    demand = torch.rand((pages, hq, page), generator=g, device=DEV).clamp_min_(1e-6).log_().neg_()
    st = dict(case=dict(case), lens=lens, max_len=max(lens), page_table=page_table, demand_table=demand_table,
              k_pages=_randn(g, pages, hkv, page, d, dtype=t), v_pages=_randn(g, pages, hkv, page, d, dtype=t),
              demand_pages=demand, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if case["op"] == "chunk":
        news = mix(_news(case))
        cu = [0]
        for s, m in enumerate(news):
            cu.append(cu[-1] + m)
            if m > 0:                                       # the new tokens were appended: no demand yet
                pos = torch.arange(lens[s] - m, lens[s], device=DEV)
                demand[demand_table[s, pos // page].long(), :, pos % page] = 0.0
        st.update(news=news, cu=cu, max_new=max(news), cu_tokens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                  q=_randn(g, max(1, cu[-1]), hq, d, std=1.5, dtype=t)[:cu[-1]])
    else:
        st.update(keeps=keeps, max_keep=max(min(n, k) for n, k in zip(lens, keeps)),
                  keep=torch.tensor(keeps, dtype=torch.int32, device=DEV),
                  dst_page_table=dst_page_table if moves else None, dst_demand_table=dst_demand_table if moves else None)
    if own:
        from long_context_attention_gb300 import binding
        st["cache"] = binding.PagedCache(st["k_pages"], st["v_pages"], demand, page_table, demand_table, st["seq_lens"])
        if case["op"] == "chunk":
            st["workspace"] = binding.dilution_attn_paged_chunk_workspace(st["cache"], st["q"].shape[0], st["max_new"],
                                                                          st["max_len"])
        else:
            st["workspace"] = binding.dilution_attn_paged_evict_workspace(st["cache"], st["max_keep"], st["max_len"])
    return st


# ------------------------------------------------------------------------------------------------------ the plain forms
def _run_chunk(st):
    case, page = st["case"], st["case"]["page"]
    if own:
        from long_context_attention_gb300 import binding
        out = binding.dilution_attn_paged_chunk(st["q"], st["cache"], st["cu_tokens"], st["max_new"], st["max_len"],
                                                eps=EPS, workspace=st["workspace"])
        return {"out": out, "demand_pages": st["demand_pages"]}
    hkv, group, d = case["Hkv"], case["Hq"] // case["Hkv"], case["d"]
    out = torch.empty_like(st["q"])
    for s, (n, m) in enumerate(zip(st["lens"], st["news"])):
        if m == 0:
            continue
        pages = -(-n // page)
        ids, dids = st["page_table"][s, :pages].long(), st["demand_table"][s, :pages].long()
        a, b = st["cu"][s], st["cu"][s + 1]
        hidden = torch.ones(m, n, dtype=torch.bool, device=DEV).triu_(n - m + 1)
        most = max(1, int(5e8) // (m * n * group))          # key heads at a time
        for h in range(0, hkv, most):
            hs = slice(h, min(h + most, hkv))
            qs = slice(hs.start * group, hs.stop * group)
            k = st["k_pages"][ids, hs].float().transpose(0, 1).flatten(1, 2)[:, None, :n]
            v = st["v_pages"][ids, hs].float().transpose(0, 1).flatten(1, 2)[:, None, :n]
            q = st["q"][a:b, qs].float().transpose(0, 1).unflatten(0, (-1, group)) / math.sqrt(d)
            x = (q @ k.transpose(-1, -2)).masked_fill_(hidden, -math.inf)
            p = x.sub_(x.amax(-1, keepdim=True)).exp_()
            p = p.div_(p.sum(-1, keepdim=True))
            rows = st["demand_pages"][dids, qs]                              # [pages, heads, page]
            held = rows.transpose(0, 1).flatten(1)[:, :n].unflatten(0, (-1, group))
            demand = p.cumsum(-2).add_(held[:, :, None])                     # after each query
            share = p.div_(demand + EPS)
            o = (share @ v) / share.sum(-1, keepdim=True)
            out[a:b, qs] = o.flatten(0, 1).transpose(0, 1).to(out.dtype)
            full = rows.transpose(0, 1).reshape(qs.stop - qs.start, -1)
            full[:, :n] = demand[:, :, -1].flatten(0, 1)
            st["demand_pages"][dids, qs] = full.view(-1, pages, page).transpose(0, 1)
    return {"out": out, "demand_pages": st["demand_pages"]}


def _run_evict(st):
    case, page = st["case"], st["case"]["page"]
    if own:
        from long_context_attention_gb300 import binding
        kept = torch.empty(case["S"], case["Hkv"], st["max_keep"], dtype=torch.int32, device=DEV)
        new_lens = binding.dilution_attn_paged_evict(
            st["cache"], st["keep"], st["max_keep"], st["max_len"], sinks=case["sinks"], recent=case["recent"], kept=kept,
            dst_page_table=st["dst_page_table"], dst_demand_table=st["dst_demand_table"], workspace=st["workspace"])
    else:
        S, hkv, group = case["S"], case["Hkv"], case["Hq"] // case["Hkv"]
        kept = torch.full((S, hkv, st["max_keep"]), -1, dtype=torch.int32, device=DEV)
        new_lens = torch.minimum(st["seq_lens"], st["keep"])
        heads = torch.arange(hkv, device=DEV)[:, None]
        for s, (n, most) in enumerate(zip(st["lens"], st["keeps"])):
            m = min(n, most)
            if m == 0:
                continue
            table, dtable = st["page_table"][s].long(), st["demand_table"][s].long()
            rows = st["demand_pages"][dtable[:-(-n // page)]].transpose(0, 1).flatten(1)[:, :n]
            rows = rows.reshape(hkv, group, n)
            score = rows[:, 0]
            for r in range(1, group):                                        # 32-bit sums, in the heads' order
                score = score + rows[:, r]
            score = score.clone()
            score[:, :case["sinks"]] = math.inf
            score[:, max(0, n - case["recent"]):] = math.inf
            stay = score.sort(dim=-1, descending=True, stable=True)[1][:, :m].sort(dim=-1)[0]     # [hkv, m]
            to = torch.arange(m, device=DEV)
            table2, dtable2 = (table, dtable) if case["place"] else (st["dst_page_table"][s].long(),
                                                                     st["dst_demand_table"][s].long())
            for pool in (st["k_pages"], st["v_pages"]):
                pool[table2[to // page], heads, to % page] = pool[table[stay // page], heads, stay % page]
            qh = (heads * group + torch.arange(group, device=DEV)).flatten()[:, None]
            wide = stay.repeat_interleave(group, 0)
            st["demand_pages"][dtable2[to // page], qh, to % page] = st["demand_pages"][dtable[wide // page], qh, wide % page]
            kept[s, :, :m] = stay
    return {"new_lens": new_lens, "kept": kept, "k_pages": st["k_pages"], "v_pages": st["v_pages"],
            "demand_pages": st["demand_pages"]}


def run(state):
    return _run_chunk(state) if state["case"]["op"] == "chunk" else _run_evict(state)


# ------------------------------------------------------------------------------------- the definition, in 64 bits, apart
def _exact_chunk(case, st):
    """One query head and one run of queries at a time, the keys' totals carried from run to run."""
    page, d, group = case["page"], case["d"], case["Hq"] // case["Hkv"]
    if work(case)["flops"] > 2.0e12:
        return None
    D = st["demand_pages"].double()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for s, (n, m) in enumerate(zip(st["lens"], st["news"])):
        if m == 0:
            continue
        place = torch.arange(n, device=DEV)
        pg, dpg, row = st["page_table"][s, place // page].long(), st["demand_table"][s, place // page].long(), place % page
        step = max(1, min(512, int(1e8) // n))
        for h in range(case["Hq"]):
            k, v = (st[x][pg, h // group, row].double() for x in ("k_pages", "v_pages"))
            total = D[dpg, h, row]
            for i in range(0, m, step):
                j = min(i + step, m)
                q = st["q"][st["cu"][s] + i:st["cu"][s] + j, h].double()
                logit = torch.einsum("id,td->it", q, k) / math.sqrt(d)
                seen = place[None] <= (n - m + torch.arange(i, j, device=DEV))[:, None]
                logit = torch.where(seen, logit, -math.inf)
                bid = torch.exp(logit - torch.logsumexp(logit, 1, keepdim=True))
                upto = total + torch.cumsum(bid, 0)
                part = bid / (upto + EPS)
                out[st["cu"][s] + i:st["cu"][s] + j, h] = torch.einsum("it,td->id", part, v) / part.sum(1)[:, None]
                total = upto[-1]
            D[dpg, h, row] = total
    return {"out": out, "demand_pages": D}


def _exact_evict(case, st):
    """The score that the last key to stay has, by counting; then every key above it and the first ones that equal it."""
    page, group = case["page"], case["Hq"] // case["Hkv"]
    K, V, D = (st[x].double() for x in ("k_pages", "v_pages", "demand_pages"))
    kept = torch.full((case["S"], case["Hkv"], st["max_keep"]), -1, dtype=torch.int64)
    new_lens = [min(n, k) for n, k in zip(st["lens"], st["keeps"])]
    for s, n in enumerate(st["lens"]):
        m = new_lens[s]
        place = torch.arange(n, device=DEV)
        pg, dpg = st["page_table"][s, place // page].long(), st["demand_table"][s, place // page].long()
        to_pg, to_dpg = (pg, dpg) if case["place"] else (st[x][s, place[:m] // page].long()
                                                         for x in ("dst_page_table", "dst_demand_table"))
        for h in range(case["Hkv"] if m else 0):
            score = torch.zeros(n, dtype=torch.float64, device=DEV)
            for r in range(h * group, (h + 1) * group):
                score = (score + st["demand_pages"][dpg, r, place % page].double()).float().double()   # each sum rounded
            sure = (place < case["sinks"]) | (place >= n - case["recent"])
            score = torch.where(sure, math.inf, score)
            least = score.sort()[0][n - m]
            above, equal = score > least, score == least
            left = m - int(above.sum())
            stay = torch.nonzero(above | (equal & (torch.cumsum(equal.int(), 0) <= left)))[:, 0]
            a, b = to_pg[:m], to_dpg[:m]
            rows = place[:m] % page
            for pool, src in ((K, st["k_pages"]), (V, st["v_pages"])):
                pool[a, h, rows] = src[pg[stay], h, stay % page].double()
            for r in range(h * group, (h + 1) * group):
                D[b, r, rows] = st["demand_pages"][dpg[stay], r, stay % page].double()
            kept[s, h, :m] = stay.cpu()
    return {"new_lens": torch.tensor(new_lens, dtype=torch.int32, device=DEV), "kept": kept.to(DEV, torch.int32),
            "k_pages": K, "v_pages": V, "demand_pages": D}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_chunk(case, st) if case["op"] == "chunk" else _exact_evict(case, st)
