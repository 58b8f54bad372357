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
