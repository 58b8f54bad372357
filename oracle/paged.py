"""Float64 oracle of the rotary positions and of the paged cache (NumPy, test
infrastructure only).  Written from the formulas; a paged cache is read row by
row through its tables."""
from __future__ import annotations

import numpy as np


def rope_angles(positions, inv_freq, pair_axis):
    """positions int [n_axes, ...], inv_freq [n] -> angles [..., n] (radians)."""
    pos = np.asarray(positions, dtype=np.float64)
    return np.stack([pos[a] * np.float64(f) for f, a in zip(np.asarray(inv_freq, np.float64), pair_axis)], axis=-1) \
        if len(pair_axis) else np.zeros(pos.shape[1:] + (0,))


def rotate(x, angles, adjacent=False, back=False):
    """x [..., d] with angles broadcastable to [..., n]: each pair times exp(+-i angle)."""
    x = np.array(x, dtype=np.float64)
    n = angles.shape[-1]
    if n == 0:
        return x
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    z = (x[..., a] + 1j * x[..., b]) * np.exp((-1j if back else 1j) * angles)
    x[..., a], x[..., b] = z.real, z.imag
    return x


def gather(pages, table, length):
    """Rows 0 .. length-1 behind a table: pages [P, H, page, ...] -> [H, length, ...]."""
    page = pages.shape[2]
    rows = [pages[int(table[t // page]), :, t % page] for t in range(length)]
    return np.stack(rows, axis=1) if rows else np.zeros((pages.shape[1], 0) + pages.shape[3:])


def paged_decode(q, k_pages, v_pages, demand_pages, page_table, demand_table, seq_lens, tau, eps, earlier=False,
                 prefix_table=None):
    """One decode step: returns (out [S, Hq, d], new demand_pages, logits scale data).

    tau: scalar or [S, Hq].  With a prefix_table its pages replace the first
    entries of every page_table row."""
    S, Hq, d = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    tau = np.broadcast_to(np.asarray(tau, np.float64), (S, Hq))
    out, D = np.zeros((S, Hq, d)), np.array(demand_pages, np.float64)
    info = {"spread": np.zeros((S, Hq)), "vmax": np.zeros((S, Hq)), "bids": {}}
    for s in range(S):
        n = int(seq_lens[s])
        if n == 0:
            continue
        table = np.array(page_table[s])
        if prefix_table is not None:
            table[:len(prefix_table)] = prefix_table
        K, V = gather(k_pages, table, n), gather(v_pages, table, n)
        for h in range(Hq):
            k, v, qq = K[h // G], V[h // G], q[s, h]
            x = tau[s, h] * (k @ qq) / np.sqrt(d)
            e = np.exp(x - x.max())
            p = e / e.sum()
            held = np.array([demand_pages[int(demand_table[s][t // page]), h, t % page] for t in range(n)], np.float64)
            share = p / ((held if earlier else held + p) + eps)
            out[s, h] = share @ v / share.sum()
            for t in range(n):
                D[int(demand_table[s][t // page]), h, t % page] = held[t] + p[t]
            info["spread"][s, h] = (np.abs(k) @ np.abs(qq)).max() * tau[s, h] / np.sqrt(d)
            info["vmax"][s, h] = np.abs(v).max()
            info["bids"][s, h] = p
    return out, D, info


def paged_chunk(q, k_pages, v_pages, demand_pages, page_table, demand_table, seq_lens, cu_tokens, tau, eps, earlier=False):
    """Chunks of new tokens: sequence s has the queries cu_tokens[s] .. cu_tokens[s + 1] - 1, its last tokens, one
    decode step after the other.  Returns (out [N, Hq, d], new demand_pages, info); rows of out without a query are 0.

    info: per row and head "spread" (the logits' scale) and "vmax"; per row, head and column "dev" (sum of A |v - out|)
    and "dev2" (the root of sum of A^2 (v - out)^2); per (sequence, head) "bids" (the column sums of the bids)."""
    N, Hq, d = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    tau = np.broadcast_to(np.asarray(tau, np.float64), (len(seq_lens), Hq))
    out, D = np.zeros((N, Hq, d)), np.array(demand_pages, np.float64)
    info = {"spread": np.zeros((N, Hq)), "vmax": np.zeros((N, Hq)), "dev": np.zeros((N, Hq, d)),
            "dev2": np.zeros((N, Hq, d)), "bids": {}}
    for s in range(len(seq_lens)):
        a, b = int(cu_tokens[s]), int(cu_tokens[s + 1])
        if a == b:
            continue
        n = int(seq_lens[s])
        t = np.arange(n)
        pg, dpg, row = np.array(page_table[s])[t // page], np.array(demand_table[s])[t // page], t % page
        for h in range(Hq):
            k, v = k_pages[pg, h // (Hq // Hkv), row], v_pages[pg, h // (Hq // Hkv), row]
            total = D[dpg, h, row]
            first = total.copy()
            for i in range(a, b):
                m = n - (b - a) + (i - a) + 1               # the keys that the query sees
                x = tau[s, h] * (k[:m] @ q[i, h]) / np.sqrt(d)
                e = np.exp(x - x.max())
                p = e / e.sum()
                share = p / ((total[:m] if earlier else total[:m] + p) + eps)
                total[:m] += p
                A = share / share.sum()
                out[i, h] = A @ v[:m]
                info["dev"][i, h] = A @ np.abs(v[:m] - out[i, h])
                info["dev2"][i, h] = np.sqrt((A * A) @ (v[:m] - out[i, h]) ** 2)
                info["spread"][i, h] = (np.abs(k[:m]) @ np.abs(q[i, h])).max() * tau[s, h] / np.sqrt(d)
                info["vmax"][i, h] = np.abs(v[:m]).max()
            D[dpg, h, row] = total
            info["bids"][s, h] = total - first
    return out, D, info


def paged_evict(k_pages, v_pages, demand_pages, page_table, demand_table, seq_lens, keep, max_keep, sinks=0, recent=0,
                dst_page_table=None, dst_demand_table=None):
    """Eviction by accumulated demand; scores are fp32 sums in the heads' order.  Returns copies of the pools after it,
    the new lengths and the places that stayed [S, Hkv, max_keep] (then -1)."""
    K, V, D = np.array(k_pages), np.array(v_pages), np.array(demand_pages)
    Hkv, page, Hq = K.shape[1], K.shape[2], D.shape[1]
    G = Hq // Hkv
    new_lens, kept = np.array(seq_lens), np.full((len(seq_lens), Hkv, max_keep), -1, np.int32)
    dpt = page_table if dst_page_table is None else dst_page_table
    ddt = demand_table if dst_demand_table is None else dst_demand_table
    for s, n in enumerate(seq_lens):
        n = int(n)
        m = new_lens[s] = min(n, int(keep[s]))
        t = np.arange(n)
        pg, dpg, row = np.array(page_table[s])[t // page], np.array(demand_table[s])[t // page], t % page
        to = np.arange(m)
        tpg, tdpg, trow = np.array(dpt[s])[to // page], np.array(ddt[s])[to // page], to % page
        for h in range(Hkv):
            score = np.asarray(demand_pages[dpg, h * G, row], np.float32)
            for g in range(1, G):
                score = (score + np.asarray(demand_pages[dpg, h * G + g, row], np.float32)).astype(np.float32)
            score = np.where(np.isnan(score) | (t < sinks) | (t >= n - recent), np.float32(np.inf), score)
            best = sorted(range(n), key=lambda i: (-score[i], i))[:m]
            stay = np.array(sorted(best), dtype=np.int64)
            kept[s, h, :m] = stay
            K[tpg, h, trow], V[tpg, h, trow] = k_pages[pg[stay], h, row[stay]], v_pages[pg[stay], h, row[stay]]
            for g in range(h * G, (h + 1) * G):
                D[tdpg, g, trow] = demand_pages[dpg[stay], g, row[stay]]
    return K, V, D, new_lens, kept
