"""Cases of the paged serving path and the rotary positions: what each call computes in plain torch, and what it costs.

Operators
  rope / rope_bwd   rotary positions with one to three axes on the queries and keys of a fused projection
  append            new keys and values into a paged cache, rotated on the way, with each key's demand
  decode            one dilution-attention query per sequence over the paged cache (ragged lengths, shared heads)
  prefix            the same for a batch whose sequences share a long prefix
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
MOST_BYTES = 4.2e9      # of one pass: the largest listed case is a little below


# ----------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the queries and keys of one short prompt on their way into attention: a launch and little else
        dict(name="rope_prompt_512", op="rope", B=1, Hq=12, Hk=12, T=512, d=64, dtype="bf16", axes=1, adjacent=False,
             rot=64, interleaved=False, bwd=False),
        # gradients of a training step at the training context, video tokens (time, height, width)
        dict(name="rope_bwd_train_16384", op="rope", B=4, Hq=12, Hk=12, T=16384, d=64, dtype="bf16", axes=3,
             adjacent=False, rot=64, interleaved=False, bwd=True),
        # the long-context prefill in the fp32 type, pairs side by side, head dimension 128
        dict(name="rope_long_131072_f32", op="rope", B=1, Hq=12, Hk=12, T=131072, d=128, dtype="f32", axes=1,
             adjacent=True, rot=128, interleaved=False, bwd=False),
        # one new token of each of 8 sequences: what a serving loop calls before every decode step
        dict(name="append_step_8", op="append", S=8, Hq=12, Hkv=12, d=64, page=64, dtype="bf16", lo=100, hi=4000,
             tokens="one", with_q=True, demand=False, axes=1, adjacent=False),
        # 16 prompts of different lengths, text and images, after their prefill (its demand goes into the cache)
        dict(name="append_prompts_16", op="append", S=16, Hq=12, Hkv=4, d=128, page=32, dtype="bf16", lo=37, hi=8191,
             tokens="all", with_q=False, demand=True, axes=3, adjacent=False),
        # a single user's short chat: latency
        dict(name="decode_one_500", op="decode", S=1, Hq=12, Hkv=12, d=64, page=16, dtype="bf16", lo=500, hi=500,
             idle=False),
        # a batch of mixed lengths from one token up, keys shared by three heads, some slots without a sequence
        dict(name="decode_ragged_48", op="decode", S=48, Hq=12, Hkv=4, d=128, page=32, dtype="bf16", lo=1, hi=16384,
             idle=True),
        # eight caches of 131072 tokens: the long-context decode workload
        dict(name="decode_long_8x131072", op="decode", S=8, Hq=12, Hkv=12, d=64, page=64, dtype="bf16", lo=131072,
             hi=131072, idle=False),
        # the fp32 type, medium lengths
        dict(name="decode_f32_4", op="decode", S=4, Hq=12, Hkv=12, d=64, page=32, dtype="f32", lo=4001, hi=16001,
             idle=False),
        # a chat service: 16 conversations behind one system prompt
        dict(name="prefix_chat_16", op="prefix", S=16, Hq=12, Hkv=12, d=64, page=16, dtype="bf16", prefix=2048, lo=1,
             hi=300),
        # questions about one document, shared heads
        dict(name="prefix_document_32", op="prefix", S=32, Hq=16, Hkv=4, d=128, page=64, dtype="bf16", prefix=32768,
             lo=5, hi=700),
        # 64 samples drawn behind one long context
        dict(name="prefix_long_64", op="prefix", S=64, Hq=12, Hkv=12, d=64, page=128, dtype="bf16", prefix=131072,
             lo=1, hi=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw_once(rng):
    op = rng.choice(["rope", "append", "decode", "prefix"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8, 12])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    axes = rng.choice([1, 2, 3])
    adjacent = rng.random() < 0.4
    if op == "rope":
        return dict(op=op, B=rng.choice([1, 2, 3, 4]), Hq=hkv * group, Hk=hkv, T=_log_int(rng, 1, 131072), d=d, dtype=dtype,
                    axes=axes, adjacent=adjacent, rot=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                    interleaved=rng.random() < 0.5, bwd=rng.random() < 0.5)
    if op == "append":
        hi = _log_int(rng, 1, 16384)
        tokens = rng.choice(["one", "all"])
        return dict(op=op, S=_log_int(rng, 1, 64), Hq=hkv * group, Hkv=hkv, d=d, page=page, dtype=dtype,
                    lo=_log_int(rng, 1, hi), hi=hi, tokens=tokens, with_q=tokens == "one" or rng.random() < 0.5,
                    demand=tokens == "all" and rng.random() < 0.7, axes=axes, adjacent=adjacent)
    if op == "decode":
        hi = _log_int(rng, 1, 131072)
        return dict(op=op, S=_log_int(rng, 1, 64), Hq=hkv * group, Hkv=hkv, d=d, page=page, dtype=dtype,
                    lo=_log_int(rng, 1, hi), hi=hi, idle=rng.random() < 0.3)
    hi = _log_int(rng, 1, 2000)
    return dict(op=op, S=_log_int(rng, 2, 64), Hq=hkv * group, Hkv=hkv, d=d, page=page, dtype=dtype,
                prefix=page * max(1, _log_int(rng, 64, 131072) // page), lo=_log_int(rng, 1, hi), hi=hi)


def _room(case):
    """Bytes that the plain form holds for a case, roughly: drawn cases stay far below the card."""
    if case["op"] in ("rope", "append"):
        return 0.0
    S, L = case["S"], case["hi"] + case.get("prefix", 0)
    keys = S * case["hi"] + case.get("prefix", 0)
    return 8.0 * keys * case["Hkv"] * case["d"] + 24.0 * S * case["Hq"] * L


def draw(rng):
    while True:
        case = _draw_once(rng)
        if work(case)["bytes"] <= MOST_BYTES and work(case)["flops"] <= 1.0e11 and _room(case) <= 2.5e10:
            return case


def _lens(case):
    """Lengths of the case's sequences (before they are shuffled): spread evenly over their logarithm."""
    S, lo, hi = case["S"], case["lo"], case["hi"]
    lens = [int(round(lo * (hi / lo) ** (i / max(1, S - 1)))) if lo < hi else hi for i in range(S)]
    lens[-1] = hi
    if case.get("idle"):
        lens = [0 if i % 8 == 3 else n for i, n in enumerate(lens)]
    return [n + case.get("prefix", 0) for n in lens] if "prefix" in case else lens


def work(case):
    d, e = case["d"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["B"] * case["T"]
        elems = n * (case["Hq"] + case["Hk"]) * d
        return {"bytes": 2 * elems * e + 4 * n * case["axes"], "flops": 3 * elems * case["rot"] // d}
    hq, hkv = case["Hq"], case["Hkv"]
    if case["op"] == "append":
        n = case["S"] if case["tokens"] == "one" else sum(_lens(case))
        per = 2 * (2 * hkv * d * e) + 4 * hq + 4 * case["axes"]
        per += 2 * hq * d * e * case["with_q"] + 4 * hq * case["demand"]
        return {"bytes": n * per, "flops": 3 * n * d * (hkv + hq * case["with_q"])}
    seen = sum(_lens(case))                                          # (sequence, key) pairs
    held = seen - (case["S"] - 1) * case["prefix"] if "prefix" in case else seen
    return {"bytes": 2 * held * hkv * d * e + 8 * seen * hq + 2 * case["S"] * hq * d * e, "flops": 4 * seen * hq * d}


# ---------------------------------------------------------------------------------------------------------- the inputs
def _randn(g, *shape, std=1.0, dtype=torch.float32):
    """Normal values, rounded once to `dtype`."""
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _rotary(case, g, n_tok):
    """Frequencies, each pair's axis and the tokens' positions [axes, tokens] of a case."""
    pairs, axes = case.get("rot", case["d"]) // 2, case["axes"]
    inv_freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(DEV)
    if case.get("interleaved"):
        pair_axis = [j % axes for j in range(pairs)]
    else:
        pair_axis = [min(axes - 1, j * axes // max(1, pairs)) for j in range(pairs)]
    i = torch.arange(n_tok, device=DEV, dtype=torch.int64)
    start = int(torch.randint(0, 4000, (1,), generator=g, device=DEV))
    # one axis: text.  Two: the rows and columns of an image.  Three: frames of 24 x 32 patches.
    cols = {1: [i + start], 2: [i // 32 + start, i % 32], 3: [i // 768 + start, i // 32 % 24, i % 32]}[axes]
    return inv_freq, pair_axis, torch.stack(cols).to(torch.int32).contiguous()


def _pools(case, g, lens, hold=None):
    """A paged cache for sequences of these lengths: pages in random order, entries past a sequence's end -1."""
    S, page, d = case["S"], case["page"], case["d"]
    prefix_pages = case.get("prefix", 0) // page
    need = [-(-n // page) for n in lens]
    width = max(need) + 1
    table = torch.full((S, width), -1, dtype=torch.int32)
    dtable = torch.full((S, width), -1, dtype=torch.int32)
    kv_pages, dem_pages = prefix_pages + sum(n - prefix_pages for n in need) + 2, sum(need) + 2
    order = torch.randperm(kv_pages, generator=g, device=DEV).cpu().to(torch.int32)
    dorder = torch.randperm(dem_pages, generator=g, device=DEV).cpu().to(torch.int32)
    at, dat = prefix_pages, 0
    for s, n in enumerate(need):
        table[s, :prefix_pages] = order[:prefix_pages]
        table[s, prefix_pages:n] = order[at:at + n - prefix_pages]
        dtable[s, :n] = dorder[dat:dat + n]
        at, dat = at + n - prefix_pages, dat + n
    t = TYPES[case["dtype"]]
    k = _randn(g, kv_pages, case["Hkv"], page, d, dtype=t)
    v = _randn(g, kv_pages, case["Hkv"], page, d, dtype=t)
    # about one unit of demand a key, with the heavy tail that earlier queries leave
    u = torch.rand((dem_pages, case["Hq"], page), generator=g, device=DEV).clamp_min_(1e-6)
    demand = u.log_().neg_()
    return dict(k_pages=k, v_pages=v, demand_pages=demand, page_table=table.to(DEV), demand_table=dtable.to(DEV),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                prefix_table=order[:prefix_pages].to(DEV) if prefix_pages else None)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, d = TYPES[case["dtype"]], case["d"]
    st = dict(case=dict(case))
    if case["op"] == "rope":
        B, Hq, Hk, T = (case[x] for x in ("B", "Hq", "Hk", "T"))
        inv_freq, pair_axis, pos = _rotary(case, g, T)
        # the projection's output: queries, keys and values of a token side by side
        rows = torch.empty(B, T, (Hq + 2 * Hk) * d, dtype=t, device=DEV)
        if case["bwd"]:
            st["q"], st["k"] = _randn(g, B, Hq, T, d, dtype=t), _randn(g, B, Hk, T, d, dtype=t)
            rows.zero_()
        else:
            rows[..., :Hq * d] = _randn(g, B, T, Hq * d, std=1.5, dtype=t)
            rows[..., Hq * d:] = _randn(g, B, T, 2 * Hk * d, dtype=t)
        heads = rows.view(B, T, Hq + 2 * Hk, d).transpose(1, 2)
        at = ("dq", "dk") if case["bwd"] else ("q", "k")
        st[at[0]], st[at[1]] = heads[:, :Hq], heads[:, Hq:Hq + Hk]
        st.update(rows=rows, inv_freq=inv_freq, pair_axis=torch.tensor(pair_axis, device=DEV), positions=pos)
        if own:
            from long_context_attention_gb300 import binding
            st["spec"] = binding.rope_spec(inv_freq, pair_axis, case["axes"], case["adjacent"])
        return st
    lens = _lens(case)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=g, device=DEV).tolist()]
    st.update(_pools(case, g, lens))
    if case["op"] == "append":
        Hq, Hkv = case["Hq"], case["Hkv"]
        counts = [min(1, n) if case["tokens"] == "one" else n for n in lens]
        N = sum(counts)
        cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
        cu[1:] = torch.tensor(counts).cumsum(0)
        inv_freq, pair_axis, pos = _rotary(case, g, N)
        rows = _randn(g, N, (Hq + 2 * Hkv) * d, dtype=t).view(N, Hq + 2 * Hkv, d)
        st.update(q=rows[:, :Hq] if case["with_q"] else None, k=rows[:, Hq:Hq + Hkv], v=rows[:, Hq + Hkv:],
                  cu_tokens=cu.to(torch.int32).to(DEV), inv_freq=inv_freq, positions=pos,
                  pair_axis=torch.tensor(pair_axis, device=DEV),
                  demand=torch.rand(Hq, N, generator=g, device=DEV).mul_(2.0).t() if case["demand"] else None)
    else:
        st.update(q=_randn(g, case["S"], case["Hq"], d, std=1.5, dtype=t), max_len=max(lens))
    if own:
        from long_context_attention_gb300 import binding
        st["cache"] = binding.PagedCache(st["k_pages"], st["v_pages"], st["demand_pages"], st["page_table"],
                                         st["demand_table"], st["seq_lens"])
        if case["op"] == "append":
            st["spec"] = binding.rope_spec(st["inv_freq"], pair_axis, case["axes"], case["adjacent"])
            st["workspace"] = binding.dilution_attn_paged_append_workspace(st["cache"])
        else:
            st["workspace"] = binding.dilution_attn_paged_decode_workspace(st["cache"], st["max_len"])
    return st


# ------------------------------------------------------------------------------------------------------ the plain forms
def _rotate(x, pos, st, sign):
    """x [..., tokens, d] rotated by sign * position * frequency; pos [axes, tokens]."""
    n, d = st["inv_freq"].numel(), x.shape[-1]
    angle = pos[st["pair_axis"]].double().t() * st["inv_freq"].double()      # [tokens, pairs]: 64 bits for far positions
    c, s = angle.cos().float(), angle.sin().float() * sign
    f = x.float()
    if st["case"]["adjacent"]:
        a, b = f[..., 0:2 * n:2], f[..., 1:2 * n:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = f[..., :n], f[..., n:2 * n]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, f[..., 2 * n:]], -1).to(x.dtype)


def _run_rope(st):
    case = st["case"]
    if own:
        from long_context_attention_gb300 import binding
        if case["bwd"]:
            binding.dilution_attn_rope_bwd(st["q"], st["k"], st["positions"], st["spec"], st["dq"], st["dk"])
            return st["rows"]
        return binding.dilution_attn_rope(st["q"], st["k"], st["positions"], st["spec"])
    sign = -1.0 if case["bwd"] else 1.0
    q, k = _rotate(st["q"], st["positions"], st, sign), _rotate(st["k"], st["positions"], st, sign)
    if case["bwd"]:
        st["dq"].copy_(q)
        st["dk"].copy_(k)
        return st["rows"]
    return q, k


def _run_append(st):
    case, page = st["case"], st["case"]["page"]
    if own:
        from long_context_attention_gb300 import binding
        q = binding.dilution_attn_paged_append(st["q"], st["k"], st["v"], st["cache"], st["cu_tokens"], rope=st["spec"],
                                               positions=st["positions"], demand=st["demand"], workspace=st["workspace"])
    else:
        cu, N = st["cu_tokens"].long(), st["k"].shape[0]
        tok = torch.arange(N, device=DEV)
        seq = (tok[:, None] >= cu[None, 1:]).sum(1)                          # the sequence of each token
        at = st["seq_lens"].long()[seq] - cu[seq + 1] + tok                  # its place in the cache
        pg, dpg = st["page_table"][seq, at // page].long(), st["demand_table"][seq, at // page].long()
        turn = lambda x: _rotate(x.transpose(0, 1), st["positions"], st, 1.0).transpose(0, 1)
        st["k_pages"][pg, :, at % page] = turn(st["k"])
        st["v_pages"][pg, :, at % page] = st["v"]
        st["demand_pages"][dpg, :, at % page] = st["demand"] if case["demand"] else 0.0
        q = turn(st["q"]).contiguous() if case["with_q"] else None
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"], "demand_pages": st["demand_pages"]}


def _keys(pages, table):
    """The rows of pages [P, H, page, d] behind table [..., n], in order: fp32 [..., H, n * page, d]."""
    x = pages[table.long().clamp_min(0)].float()                             # [..., n, H, page, d]
    return x.transpose(-4, -3).flatten(-3, -2)


def _run_decode(st):
    case, page, P = st["case"], st["case"]["page"], st["case"].get("prefix", 0)
    if own:
        from long_context_attention_gb300 import binding
        out = binding.dilution_attn_paged_decode(st["q"], st["cache"], st["max_len"], prefix_table=st["prefix_table"],
                                                 eps=EPS, workspace=st["workspace"])
        return {"out": out, "demand_pages": st["demand_pages"]}
    S, Hq, Hkv, d = (case[x] for x in ("S", "Hq", "Hkv", "d"))
    n, first = -(-st["max_len"] // page), P // page
    q = st["q"].float().view(S, Hkv, Hq // Hkv, d) / math.sqrt(d)
    mine = st["page_table"][:, first:n]
    x = q @ _keys(st["k_pages"], mine).transpose(-1, -2)                     # [S, Hkv, group, own keys]
    if P:
        rows = q.transpose(0, 1).reshape(Hkv, -1, d)                         # the whole batch against the prefix at once
        shared = rows @ _keys(st["k_pages"], st["prefix_table"]).transpose(-1, -2)
        x = torch.cat([shared.view(Hkv, S, -1, P).transpose(0, 1), x], -1)
    seen = torch.arange(n * page, device=DEV) < st["seq_lens"][:, None]      # [S, keys]
    seen = seen[:, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-3.0e38)
    e = torch.exp(x - m)
    p = e / e.sum(-1, keepdim=True).clamp_min(1e-30)
    dpg = st["demand_table"][:, :n].long().clamp_min(0)
    D = st["demand_pages"][dpg].transpose(1, 2).reshape(S, Hkv, -1, n * page)
    share = torch.where(seen, p / (D + p + EPS), 0.0)
    num = share[..., P:] @ _keys(st["v_pages"], mine)
    if P:
        rows = share[..., :P].transpose(0, 1).reshape(Hkv, -1, P)
        num = num + (rows @ _keys(st["v_pages"], st["prefix_table"])).view(Hkv, S, -1, d).transpose(0, 1)
    out = num / share.sum(-1, keepdim=True).clamp_min(1e-37)
    add = p.reshape(S, Hq, n, page).transpose(1, 2).reshape(-1, Hq, page)    # 0 at every key that is not seen
    st["demand_pages"].index_add_(0, dpg.reshape(-1), add)
    return {"out": out.reshape(S, Hq, d).to(st["q"].dtype), "demand_pages": st["demand_pages"]}


def run(state):
    return {"rope": _run_rope, "append": _run_append}.get(state["case"]["op"], _run_decode)(state)


# ------------------------------------------------------------------------------------- the definition, in 64 bits, apart
def _exact_turn(x, pos, st, back):
    """Complex numbers: each pair times exp(+-i position frequency).  x [tokens, H, d] in 64 bits."""
    inv, axis, n = st["inv_freq"].double(), st["pair_axis"].tolist(), st["inv_freq"].numel()
    out = x.clone()
    for j in range(n):
        a, b = (2 * j, 2 * j + 1) if st["case"]["adjacent"] else (j, j + n)
        w = torch.polar(torch.ones_like(pos[0], dtype=torch.float64), pos[axis[j]].double() * inv[j])
        z = torch.complex(x[..., a], x[..., b]) * (w.conj() if back else w)[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        got = []
        for name in ("q", "k"):
            x = st[name]
            y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
            for b in range(x.shape[0]):
                y[b] = _exact_turn(x[b].transpose(0, 1).double(), st["positions"], st, case["bwd"]).transpose(0, 1)
            got.append(y)
        if not case["bwd"]:
            return tuple(got)
        B, T, Hq, Hk, d = (case[x] for x in ("B", "T", "Hq", "Hk", "d"))
        both = torch.cat([got[0], got[1], torch.zeros(B, Hk, T, d, dtype=torch.float64, device=DEV)], 1)
        return both.transpose(1, 2).reshape(B, T, -1)
    page = case["page"]
    lens, table, dtable = st["seq_lens"].tolist(), st["page_table"].tolist(), st["demand_table"].tolist()
    D = st["demand_pages"].double()
    if case["op"] == "append":
        K, V, cu = st["k_pages"].double(), st["v_pages"].double(), st["cu_tokens"].tolist()
        turned = _exact_turn(st["k"].double(), st["positions"], st, False)
        for s, n in enumerate(lens):
            lo, hi = cu[s], cu[s + 1]
            for pg in range((n - (hi - lo)) // page, -(-n // page)):
                a, b = max(pg * page, n - (hi - lo)), min((pg + 1) * page, n)
                i = lo + a - (n - (hi - lo))
                to = slice(a - pg * page, b - pg * page)
                K[table[s][pg], :, to] = turned[i:i + b - a].transpose(0, 1)
                V[table[s][pg], :, to] = st["v"][i:i + b - a].double().transpose(0, 1)
                D[dtable[s][pg], :, to] = st["demand"][i:i + b - a].double().t() if case["demand"] else 0.0
        q = _exact_turn(st["q"].double(), st["positions"], st, False) if case["with_q"] else None
        return {"q": q, "k_pages": K, "v_pages": V, "demand_pages": D}
    group = case["Hq"] // case["Hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        np_ = -(-n // page)
        idx = torch.tensor(table[s][:np_], device=DEV)
        didx = torch.tensor(dtable[s][:np_], device=DEV)
        for h in range(case["Hkv"]):
            k = st["k_pages"][idx, h].reshape(-1, case["d"])[:n].double()
            v = st["v_pages"][idx, h].reshape(-1, case["d"])[:n].double()
            for r in range(h * group, (h + 1) * group):
                logit = (k * st["q"][s, r].double()).sum(-1) / math.sqrt(case["d"])
                bid = torch.exp(logit - torch.logsumexp(logit, 0))
                rows = D[didx, r]
                held = rows.reshape(-1)[:n]
                part = bid / (held + bid + EPS)
                out[s, r] = (part[:, None] * v).sum(0) / part.sum()
                rows.view(-1)[:n] += bid
                D[didx, r] = rows
    return {"out": out, "demand_pages": D}
