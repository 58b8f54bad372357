"""GPU parity of the rotary positions and the paged append against the float64
oracle, and the serving path run together.

Tolerances (written before any run): a rotated element is x c - y s in fp32.
The angle is held to 2^-33 turns or better and reaches the sine as an fp32
fraction (half a step of an angle below pi: 2^-24 pi < 2^-22), sine and cosine
are good to 2^-23, the product and sum round three times (3 2^-24): below
2^-21 (|x| + |y|) in all.  A bf16 result adds half a step, 2^-8 |result|.
"""
import numpy as np
import pytest
import torch

import oracle.dilution as od
from long_context_attention_gb300 import binding as b
from long_context_attention_gb300 import rope_inv_freq, rope_pair_axis
from oracle import paged as op
from tests._paged import DEV, TYPES, check_step, make_cache, oracle_step
from tests._parity import host64

pytestmark = pytest.mark.gpu


def close(got, x, angles, adjacent, back=False):
    """got against the oracle's rotation of x (both [..., d]), with the tolerance above."""
    hx = host64(x)
    ref = op.rotate(hx, angles, adjacent, back)
    n = angles.shape[-1]
    mag = np.zeros(hx.shape)
    a, c = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    mag[..., a] = mag[..., c] = np.abs(hx[..., a]) + np.abs(hx[..., c])
    tol = 2.0 ** -21 * mag + (2.0 ** -8 * np.abs(ref) * (mag > 0) if got.dtype == torch.bfloat16 else 0.0)
    g = host64(got)
    assert (np.abs(g - ref) <= tol).all(), float((np.abs(g - ref) - tol).max())


def spec_of(n, axes, adjacent, interleaved=False, base=10000.0):
    inv = rope_inv_freq(2 * n, base).to(DEV)
    pa = rope_pair_axis(n, axes, interleaved)
    return b.rope_spec(inv, pa, axes, adjacent), inv, pa


def positions(axes, B, T, seed=0, span=4096):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-7, span, (axes, B, T), generator=g, dtype=torch.int32).to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hk,T,d,n,axes,adjacent,interleaved", [
    (1, 1, 1, 1, 64, 32, 1, False, False),
    (2, 4, 2, 37, 64, 32, 3, False, False),
    (3, 3, 3, 130, 128, 64, 3, True, True),
    (1, 12, 12, 257, 64, 16, 2, False, True),       # half of each head rotates
    (2, 2, 1, 65, 128, 12, 1, True, False),         # 24 elements rotate
    (2, 2, 1, 65, 128, 11, 4, False, False),        # odd number of pairs: no whole 16-byte pieces
    (1, 5, 0, 40, 64, 7, 2, True, False),           # queries only
    (1, 2, 2, 9, 64, 0, 1, False, False),           # nothing rotates: a copy
    (3, 5, 2, 301, 128, 63, 2, False, True),        # all but two elements, rows of odd halves
    (2, 3, 1, 77, 64, 1, 1, False, False),          # one pair
    (2, 3, 1, 77, 128, 61, 3, True, False),         # adjacent, cut inside a 16-byte piece
])
def test_rope_matches_oracle_both_ways(dtype, B, Hq, Hk, T, d, n, axes, adjacent, interleaved):
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(T)
    q = torch.randn(B, Hq, T, d, generator=g).to(t).to(DEV)
    k = torch.randn(B, Hk, T, d, generator=g).to(t).to(DEV) if Hk else None
    spec, inv, pa = spec_of(n, axes, adjacent, interleaved)
    for pb in {1, B}:
        pos = positions(axes, pb, T, seed=pb)
        ang = op.rope_angles(pos.cpu().numpy(), inv.cpu().numpy(), pa)[:, None]      # [pb, 1, T, n]
        qo, ko = b.dilution_attn_rope(q, k, pos, spec)
        close(qo, q, ang, adjacent)
        dq, dk = b.dilution_attn_rope_bwd(q, k, pos, spec)
        close(dq, q, ang, adjacent, back=True)
        if Hk:
            close(ko, k, ang, adjacent)
            close(dk, k, ang, adjacent, back=True)
        else:
            assert ko is None and dk is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 3])     # 3: rows that are not 16-byte aligned
def test_rope_through_a_fused_projection(dtype, pad):
    # q and k are views of [B, T, (Hq + 2 Hk) d (+ pad)]; the gradients are written back into such a view
    B, Hq, Hk, T, d, t = 2, 4, 2, 50, 64, TYPES[dtype]
    width = (Hq + 2 * Hk) * d + pad
    rows = torch.randn(B, T, width, generator=torch.Generator().manual_seed(3)).to(t).to(DEV)
    heads = rows[..., :width - pad].unflatten(-1, (-1, d)).transpose(1, 2)
    q, k = heads[:, :Hq], heads[:, Hq:Hq + Hk]
    spec, inv, pa = spec_of(32, 3, False)
    pos = positions(3, B, T, seed=4)
    ang = op.rope_angles(pos.cpu().numpy(), inv.cpu().numpy(), pa)[:, None]
    qo, ko = b.dilution_attn_rope(q, k, pos, spec)
    assert qo.is_contiguous() and ko.is_contiguous()
    close(qo, q, ang, False)
    close(ko, k, ang, False)
    grad = torch.full_like(rows, 9.0)
    gh = grad[..., :width - pad].unflatten(-1, (-1, d)).transpose(1, 2)
    b.dilution_attn_rope_bwd(qo, ko, pos, spec, gh[:, :Hq], gh[:, Hq:Hq + Hk])
    close(gh[:, :Hq], qo, ang, False, back=True)
    close(gh[:, Hq:Hq + Hk], ko, ang, False, back=True)
    assert (gh[:, Hq + Hk:] == 9.0).all() and (pad == 0 or (grad[..., -pad:] == 9.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,axes,d", [(32, 3, 64), (11, 1, 64), (61, 4, 128)])
def test_rope_adjacent_pairs_of_unaligned_rows(dtype, n, axes, d):
    # rows of a fused projection that start at any element: pairs move element by element, in both directions
    B, Hq, Hk, T, pad, t = 2, 3, 1, 41, 3, TYPES[dtype]
    width = (Hq + 2 * Hk) * d + pad
    rows = torch.randn(B, T, width, generator=torch.Generator().manual_seed(n)).to(t).to(DEV)
    heads = rows[..., 1:width - pad + 1].unflatten(-1, (-1, d)).transpose(1, 2)
    q, k = heads[:, :Hq], heads[:, Hq:Hq + Hk]
    spec, inv, pa = spec_of(n, axes, True)
    pos = positions(axes, B, T, seed=n)
    ang = op.rope_angles(pos.cpu().numpy(), inv.cpu().numpy(), pa)[:, None]
    qo, ko = b.dilution_attn_rope(q, k, pos, spec)
    close(qo, q, ang, True)
    close(ko, k, ang, True)
    grad = torch.full_like(rows, 9.0)
    gh = grad[..., 1:width - pad + 1].unflatten(-1, (-1, d)).transpose(1, 2)
    b.dilution_attn_rope_bwd(qo, ko, pos, spec, gh[:, :Hq], gh[:, Hq:Hq + Hk])
    close(gh[:, :Hq], qo, ang, True, back=True)
    close(gh[:, Hq:Hq + Hk], ko, ang, True, back=True)
    assert (gh[:, Hq + Hk:] == 9.0).all() and (grad[..., 0] == 9.0).all() and (grad[..., 1 - pad:] == 9.0).all()


def test_rope_in_place_broadcast_and_strided_positions():
    spec, inv, pa = spec_of(64, 1, True)
    x = torch.randn(2, 1, 33, 128, device=DEV)
    pos = positions(1, 1, 33, seed=8)
    ang = op.rope_angles(pos.cpu().numpy(), inv.cpu().numpy(), pa)[:, None]
    kept = x.clone()
    shared = x.expand(2, 4, 33, 128)                    # one head read four times
    qo, _ = b.dilution_attn_rope(shared, None, pos[:, 0], spec)
    close(qo, shared, ang, True)
    b.dilution_attn_rope(x, None, pos, spec, x)         # in place
    close(x, kept, ang, True)


@pytest.mark.parametrize("far", [(1 << 24) - 1, (1 << 30) + 12345, -(1 << 31)])
def test_rope_far_positions(far):
    spec, inv, pa = spec_of(64, 1, False)
    x = torch.randn(1, 2, 4, 128, device=DEV)
    pos = torch.tensor([[far, far + 1, 0, -1]], dtype=torch.int32, device=DEV)
    # the angle's reference in exact integer arithmetic: fp32 frequencies are integers over a power of two
    from fractions import Fraction
    pi2 = Fraction(31415926535897932384626433832795028841971693993751, 5 * 10 ** 48)
    ang = np.array([[float(Fraction(int(p)) * Fraction(float(f)) % pi2) for f in inv.cpu().numpy()]
                    for p in pos[0].tolist()])
    qo, _ = b.dilution_attn_rope(x, None, pos, spec)
    close(qo, x, ang, False)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_high_frequencies_at_far_positions(adjacent):
    # every frequency and position that is taken keeps the angle: references in exact integer arithmetic
    from fractions import Fraction
    inv = torch.tensor([2.0 ** 24 - 1, -(2.0 ** 24 - 1), 2.0 ** 20, 12345678.0, 1234.5, 6.2831855, 1.0, 1e-30], device=DEV)
    pos = torch.tensor([[(1 << 31) - 1, -(1 << 31), 1 << 24, (1 << 30) + 12345, -1, 1]], dtype=torch.int32, device=DEV)
    pi2 = Fraction(31415926535897932384626433832795028841971693993751, 5 * 10 ** 48)
    ang = np.array([[float(Fraction(int(p)) * Fraction(float(f)) % pi2) for f in inv.cpu().numpy()] for p in pos[0].tolist()])
    x = torch.randn(1, 2, 6, 64, generator=torch.Generator().manual_seed(9)).to(DEV)
    spec = b.rope_spec(inv, adjacent=adjacent)
    close(b.dilution_attn_rope(x, None, pos, spec)[0], x, ang, adjacent)
    close(b.dilution_attn_rope_bwd(x, None, pos, spec)[0], x, ang, adjacent, back=True)


def test_rope_gradient_against_differences():
    # the map is linear: a central difference of sum(w rope(x)) is exact up to fp32 rounding
    spec, _, _ = spec_of(32, 2, False)
    g = torch.Generator().manual_seed(11)
    x, w = (torch.randn(1, 2, 5, 64, generator=g).to(DEV) for _ in range(2))
    pos = positions(2, 1, 5, seed=12)
    dx, _ = b.dilution_attn_rope_bwd(w, None, pos, spec)
    for i in range(0, 640, 37):
        e = torch.zeros(640, device=DEV)
        e[i] = 0.5
        e = e.view_as(x)
        up = (b.dilution_attn_rope(x + e, None, pos, spec)[0].double() * w.double()).sum()
        down = (b.dilution_attn_rope(x - e, None, pos, spec)[0].double() * w.double()).sum()
        # two rotated elements differ, each off by 2^-21 (|x| + |y|) < 2^-21 * 10, times |w| < 5, twice
        assert abs(float(up - down) - float(dx.flatten()[i])) <= 2 * 2 * 2.0 ** -21 * 10 * 5


def test_rope_frequencies_that_are_no_numbers():
    inv = torch.tensor([float("nan"), float("inf"), 2.0 ** 24, 1.0], device=DEV)
    x = torch.ones(1, 1, 2, 64, device=DEV)
    pos = torch.tensor([[3, 4]], dtype=torch.int32, device=DEV)
    y, _ = b.dilution_attn_rope(x, None, pos, b.rope_spec(inv))
    bad = [0, 1, 2, 4, 5, 6]
    assert y[..., bad].isnan().all()
    good = [i for i in range(64) if i not in bad]
    assert y[..., good].isfinite().all()
    # the largest frequencies that are taken: 3 (2^24 - 1) radians, in exact arithmetic
    from fractions import Fraction
    pi2 = Fraction(31415926535897932384626433832795028841971693993751, 5 * 10 ** 48)
    inv = torch.tensor([2.0 ** 24 - 1, -(2.0 ** 23), 2.0 ** -40], device=DEV)
    y, _ = b.dilution_attn_rope(x, None, pos, b.rope_spec(inv))
    ang = np.array([[float(Fraction(p) * Fraction(float(f)) % pi2) for f in inv.tolist()] for p in (3, 4)])
    close(y, x, ang, False)


# ------------------------------------------------------------------------------- append
def append_oracle(cache, k, v, cu, spec_pa, pos, demand, adjacent):
    """Expected pools after an append (float64) and where rows were written."""
    inv, pa = spec_pa
    K, V, D = host64(cache.k_pages).copy(), host64(cache.v_pages).copy(), host64(cache.demand_pages).copy()
    hk, hv = host64(k), host64(v)
    tab, dtab, lens, page = cache.page_table.cpu(), cache.demand_table.cpu(), cache.seq_lens.cpu(), cache.page_size
    src = {}
    for s in range(cache.S):
        lo, hi = int(cu[s]), int(cu[s + 1])
        for n in range(lo, hi):
            t = int(lens[s]) - hi + n
            pg, dpg = int(tab[s, t // page]), int(dtab[s, t // page])
            V[pg, :, t % page] = hv[n]
            D[dpg, :, t % page] = 0.0 if demand is None else host64(demand)[n]
            src[pg, t % page] = (n, t)
    ang = {}
    for (pg, r), (n, t) in src.items():
        p = np.full((len(pos) if pos is not None else 8, 1), t) if pos is None else pos[:, n:n + 1].cpu().numpy()
        ang[pg, r] = op.rope_angles(p, inv, pa)
        K[pg, :, r] = op.rotate(hk[n], ang[pg, r], adjacent)
    return K, V, D, src, ang


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,lens,counts,Hq,Hkv,d,page,n,axes,adjacent,pos,dem,withq,pad", [
    (3, [5, 17, 64], [1, 1, 1], 4, 2, 64, 16, 32, 1, False, False, False, True, 0),
    (4, [40, 0, 7, 100], [40, 0, 3, 61], 6, 3, 128, 32, 64, 3, False, True, True, False, 0),
    (2, [33, 90], [33, 20], 2, 2, 64, 16, 16, 2, True, True, True, True, 0),
    (2, [33, 90], [33, 20], 2, 1, 64, 64, 9, 1, False, False, True, True, 1),     # unaligned rows, odd pairs
    (1, [300], [300], 8, 1, 128, 256, 0, 1, False, False, False, True, 0),        # no rotation
    (2, [33, 90], [33, 20], 2, 1, 64, 64, 9, 1, True, False, True, True, 0),      # adjacent, cut inside a piece
    (5, [1, 2, 3, 0, 4], [1, 0, 2, 0, 4], 1, 1, 64, 16, 32, 1, True, False, False, False, 2),
])
def test_append_matches_oracle(dtype, S, lens, counts, Hq, Hkv, d, page, n, axes, adjacent, pos, dem, withq, pad):
    cache, _, _ = make_cache(S, lens, Hq, Hkv, d, page, dtype, seed=sum(lens))
    t, extra = TYPES[dtype], 5                                  # 5 padding tokens behind the last sequence
    N = sum(counts) + extra
    g = torch.Generator().manual_seed(N)
    width = (Hq + 2 * Hkv) * d + pad
    rows = torch.randn(N, width, generator=g).to(t).to(DEV)
    heads = rows[:, :width - pad].unflatten(-1, (-1, d))
    q, k, v = heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:]
    cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    spec, inv, pa = spec_of(n, axes, adjacent) if n else (None, np.zeros(0), [])
    inv = inv.cpu().numpy() if n else inv
    ps = positions(axes, 1, N, seed=N)[:, 0].contiguous() if pos else None
    demand = (torch.rand(Hq, N, generator=g) * 3).to(DEV).t() if dem else None     # strided: [Hq, N] transposed
    K, V, D, src, ang = append_oracle(cache, k, v, cu.tolist(), (inv, pa), ps, demand, adjacent)
    old = cache.k_pages.clone()
    q_out = torch.full((N, Hq, d), 5.0, dtype=t, device=DEV) if withq else None
    ws = b.dilution_attn_paged_append_workspace(cache)
    got = b.dilution_attn_paged_append(q if withq else None, k, v, cache, cu, q_out, rope=spec, positions=ps,
                                       demand=demand, workspace=ws)
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    assert np.array_equal(host64(cache.v_pages), V) and np.array_equal(host64(cache.demand_pages), D)
    touched = torch.zeros(old.shape[0], old.shape[2], dtype=torch.bool, device=DEV)
    for (pg, r), (i, tt) in src.items():
        touched[pg, r] = True
        close(cache.k_pages[pg, :, r], k[i], ang[pg, r], adjacent)
        if withq:
            close(got[i], q[i], ang[pg, r], adjacent)
    same = (cache.k_pages == old) | touched[:, None, :, None]
    assert same.all()
    if withq:
        assert (got[N - extra:] == 5.0).all()                   # rows behind the last sequence stay
    else:
        assert got is None


def test_append_long_runs_of_tokens():
    # blocks of many tokens: prompts of different lengths in the same block, padding at the end, all types of rows
    lens = [5000, 1, 0, 777, 3000]
    cache, _, _ = make_cache(5, lens, 4, 2, 64, 64, "bf16", seed=14)
    N = sum(lens) + 3
    spec, inv, pa = spec_of(32, 3, True)
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(N, 8, 64, generator=g).bfloat16().to(DEV)
    ps = positions(3, 1, N, seed=6)[:, 0].contiguous()
    demand = torch.rand(N, 4, generator=g).to(DEV)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    ws = b.dilution_attn_paged_append_workspace(cache)
    q = b.dilution_attn_paged_append(rows[:, :4], rows[:, 4:6], rows[:, 6:], cache, cu, rope=spec, positions=ps,
                                     demand=demand, workspace=ws)
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    seq = torch.repeat_interleave(torch.arange(5), torch.tensor(lens)).to(DEV)
    at = torch.arange(N - 3, device=DEV) - cu.long()[seq]
    pg, dpg = cache.page_table[seq, at // 64].long(), cache.demand_table[seq, at // 64].long()
    ang = op.rope_angles(ps.cpu().numpy(), inv.cpu().numpy(), pa)[:N - 3, None]
    close(q[:N - 3], rows[:N - 3, :4], ang, True)
    close(cache.k_pages[pg, :, at % 64], rows[:N - 3, 4:6], ang, True)
    assert torch.equal(cache.v_pages[pg, :, at % 64], rows[:N - 3, 6:])
    assert torch.equal(cache.demand_pages[dpg, :, at % 64], demand[:N - 3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [32, 11])     # 11: pairs that no 16-byte pieces hold
def test_append_turns_queries_in_place(dtype, n):
    cache, _, _ = make_cache(3, [9, 40, 70], 4, 2, 64, 16, dtype, seed=17)
    spec, inv, pa = spec_of(n, 1, False)
    rows = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(18)).to(TYPES[dtype]).to(DEV)
    q = rows[:, :4].contiguous()
    cu = torch.arange(4, dtype=torch.int32, device=DEV)
    assert b.dilution_attn_paged_append(q, rows[:, 4:6], rows[:, 6:], cache, cu, q, rope=spec) is q
    close(q, rows[:, :4], op.rope_angles(cache.seq_lens.cpu().numpy()[None] - 1, inv.cpu().numpy(), pa)[:, None], False)


def test_append_queries_between_the_rows_of_the_keys():
    # q_out inside the range of the strided keys and values, over none of their rows
    cache, _, _ = make_cache(3, [9, 40, 70], 2, 2, 64, 16, "bf16", seed=17)
    spec, inv, pa = spec_of(32, 1, False)
    buf = torch.randn(3, 2048, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    k, v = buf[:, :128].unflatten(-1, (2, 64)), buf[:, 1024:1152].unflatten(-1, (2, 64))
    q, q_out = torch.randn(3, 2, 64, device=DEV).bfloat16(), buf[1, 512:896].view(3, 2, 64)
    kept = buf.clone()
    cu = torch.arange(4, dtype=torch.int32, device=DEV)
    ang = op.rope_angles(cache.seq_lens.cpu().numpy()[None] - 1, inv.cpu().numpy(), pa)[:, None]
    assert b.dilution_attn_paged_append(q, k, v, cache, cu, q_out, rope=spec) is q_out
    close(q_out, q, ang, False)
    at = (cache.seq_lens - 1).long()
    pg = cache.page_table[torch.arange(3, device=DEV), at // 16].long()
    close(cache.k_pages[pg, :, at % 16], k, ang, False)
    assert torch.equal(cache.v_pages[pg, :, at % 16], v)
    kept[1, 512:896] = buf[1, 512:896]
    assert torch.equal(buf, kept)
    with pytest.raises(b.DilutionAttnError):                  # over the second token's keys
        b.dilution_attn_paged_append(q, k, v, cache, cu, buf[1, 64:448].view(3, 2, 64), rope=spec)


def test_append_many_sequences():
    # more sequences than the search holds in shared memory, one token each
    S = 1500
    cache, _, _ = make_cache(S, [1 + i % 3 for i in range(S)], 1, 1, 64, 16, "bf16", seed=2)
    k = torch.randn(S, 1, 64, device=DEV).bfloat16()
    v = torch.randn(S, 1, 64, device=DEV).bfloat16()
    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    b.dilution_attn_paged_append(None, k, v, cache, cu)
    pg = cache.page_table[:, 0].long()
    at = (cache.seq_lens - 1).long()
    assert torch.equal(cache.k_pages[pg, :, at], k) and torch.equal(cache.v_pages[pg, :, at], v)
    assert not cache.demand_pages[cache.demand_table[:, 0].long(), :, at].any()


def test_append_reports_bad_device_data_and_skips_the_token():
    def after(change, cu=(0, 2, 4)):
        cache, _, _ = make_cache(2, [20, 40], 2, 2, 64, 16, "bf16", seed=7)
        change(cache)
        old = [x.clone() for x in (cache.k_pages, cache.v_pages, cache.demand_pages)]
        k = torch.randn(4, 2, 64, device=DEV).bfloat16()
        ws = b.dilution_attn_paged_append_workspace(cache)
        b.dilution_attn_paged_append(None, k, k, cache, torch.tensor(cu, dtype=torch.int32, device=DEV), workspace=ws)
        rows = ((cache.v_pages != old[1]).any(-1).any(1)).sum().item()     # (page, row) pairs written
        return b.dilution_attn_get_error(ws), rows

    assert after(lambda c: None) == (b.DA_OK, 4)
    assert after(lambda c: c.seq_lens.__setitem__(0, 1)) == (b.DA_ERR_INVALID, 2)        # fewer than its new tokens
    assert after(lambda c: c.seq_lens.__setitem__(0, 1000)) == (b.DA_ERR_INVALID, 2)     # beyond the table
    assert after(lambda c: c.page_table.__setitem__((1, 2), 999)) == (b.DA_ERR_INVALID, 2)
    assert after(lambda c: c.demand_table.__setitem__((1, 2), -1)) == (b.DA_ERR_INVALID, 2)
    assert after(lambda c: None, (0, 2, 9)) == (b.DA_ERR_INVALID, 2)                     # more tokens than given
    assert after(lambda c: None, (0, 2, 2)) == (b.DA_OK, 2)                              # two padding tokens
    assert after(lambda c: None, (1, 3, 4))[0] == b.DA_ERR_INVALID                       # does not start at 0


# --------------------------------------------------------------------- the path, run together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_to_decode_steps(dtype):
    """A prompt goes through the rotation and the framework's prefill, its keys, values and demand into the paged
    cache; two sequences then share it as their prefix and decode three tokens each.  Every step is compared with the
    framework's contiguous decode step on the same tokens."""
    H, d, P, page, steps, t = 3, 64, 96, 32, 3, TYPES[dtype]
    S, T_cap = 2, P + steps
    g = torch.Generator().manual_seed(19)
    spec, inv, pa = spec_of(32, 1, False)
    rows = torch.randn(1, P, 3 * H * d, generator=g).to(t).to(DEV)
    heads = rows.unflatten(-1, (-1, d)).transpose(1, 2)
    pos = torch.arange(P, dtype=torch.int32, device=DEV)[None]
    q, k = b.dilution_attn_rope(heads[:, :H], heads[:, H:2 * H], pos, spec)
    v = heads[:, 2 * H:].contiguous()
    demand = torch.empty(1, H, P, device=DEV)
    b.dilution_attn_fwd(q, k, v, demand_out=demand)
    # the paged cache: 3 shared pages, one own page a sequence; 4 demand pages each
    kp = torch.zeros(6, H, page, d, dtype=t, device=DEV)
    vp = torch.zeros_like(kp)
    dp = torch.zeros(9, H, page, device=DEV)
    table = torch.tensor([[4, 0, 2, 1], [4, 0, 2, 5]], dtype=torch.int32, device=DEV)
    dtable = torch.tensor([[8, 1, 3, 0], [2, 7, 5, 4]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([P, 0], dtype=torch.int32, device=DEV)
    cache = b.PagedCache(kp, vp, dp, table, dtable, lens)
    cu = torch.tensor([0, P, P], dtype=torch.int32, device=DEV)
    tok = rows[0].unflatten(-1, (-1, d))
    b.dilution_attn_paged_append(None, tok[:, H:2 * H], tok[:, 2 * H:], cache, cu, rope=spec, positions=pos,
                                 demand=demand[0].t())
    assert torch.equal(kp[table[0, :3].long()].transpose(0, 1).reshape(H, P, d), k[0])     # the same rotation
    dp[dtable[1, :3].long()] = dp[dtable[0, :3].long()]                                    # the second sequence forks
    lens.fill_(P)
    # the contiguous caches of the framework's decode step
    kc = torch.zeros(S, H, T_cap, d, dtype=t, device=DEV)
    vc, dc = torch.zeros_like(kc), torch.zeros(S, H, T_cap, device=DEV)
    kc[:, :, :P], vc[:, :, :P], dc[:, :, :P] = k, v, demand
    cu1 = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    pt = table[0, :3].contiguous()
    ws = b.dilution_attn_paged_decode_workspace(cache, T_cap)
    for i in range(steps):
        new = torch.randn(S, 3 * H, d, generator=g).to(t).to(DEV)
        lens += 1
        qn = b.dilution_attn_paged_append(new[:, :H], new[:, H:2 * H], new[:, 2 * H:], cache, cu1, rope=spec,
                                          workspace=ws)
        before = dp.clone()
        ref = oracle_step(cache, qn, prefix_table=pt)
        out = b.dilution_attn_paged_decode(qn, cache, T_cap, prefix_table=pt, workspace=ws)
        assert b.dilution_attn_get_error(ws) == b.DA_OK
        check_step(cache, qn, before, out, ref)
        # the contiguous step takes the rotated token
        p1 = torch.full((1, 1), P + i, dtype=torch.int32, device=DEV)
        qr, kr = b.dilution_attn_rope(new[:, :H, None], new[:, H:2 * H, None], p1, spec)
        assert torch.equal(qr[:, :, 0], qn)
        same = b.dilution_attn_decode_step(qn, kr[:, :, 0].contiguous(), new[:, 2 * H:].contiguous(), kc, vc, dc, P + i)
        # both are within the tolerance of tests/_paged.py of the same value; bf16 outputs each round once
        vmax = float(vc.abs().max())
        tol = 2 * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -16) * vmax
        assert (out.double() - same.double()).abs().max() <= tol
        got = dp[dtable.long()].transpose(1, 2).reshape(S, H, -1)[..., :T_cap]
        assert torch.allclose(got, dc, rtol=1e-4, atol=1e-5)


def test_captured_append_and_decode_step():
    """Append and decode captured as one graph and replayed: lengths grow on the device between replays."""
    S, H, d, page = 3, 2, 64, 16
    cache, _, _ = make_cache(S, [48, 64, 33], H, H, d, page, "bf16", seed=3, extra_width=1)
    cache.seq_lens.copy_(torch.tensor([40, 60, 28], dtype=torch.int32))
    spec, inv, pa = spec_of(32, 1, True)
    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    new = torch.randn(S, 3 * H, d, device=DEV).bfloat16()
    ws = b.dilution_attn_paged_decode_workspace(cache, 64)
    qn, out = torch.empty(S, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(S, H, d, dtype=torch.bfloat16, device=DEV)

    def step():
        b.dilution_attn_paged_append(new[:, :H], new[:, H:2 * H], new[:, 2 * H:], cache, cu, qn, rope=spec, workspace=ws)
        b.dilution_attn_paged_decode(qn, cache, 64, out, workspace=ws)

    saved = [x.clone() for x in (cache.k_pages, cache.v_pages, cache.demand_pages)]
    step()
    torch.cuda.synchronize()
    for x, y in zip((cache.k_pages, cache.v_pages, cache.demand_pages), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        cache.seq_lens += 1
        new.copy_(torch.randn(S, 3 * H, d, device=DEV))
        # what the step should see: the same append on a copy, then the oracle
        copy = b.PagedCache(cache.k_pages.clone(), cache.v_pages.clone(), cache.demand_pages.clone(), cache.page_table,
                            cache.demand_table, cache.seq_lens)
        qc = b.dilution_attn_paged_append(new[:, :H], new[:, H:2 * H], new[:, 2 * H:], copy, cu, rope=spec)
        ref = oracle_step(copy, qc)
        before = copy.demand_pages.clone()
        graph.replay()
        assert b.dilution_attn_get_error(ws) == b.DA_OK
        assert torch.equal(qn, qc) and torch.equal(cache.k_pages, copy.k_pages)
        check_step(cache, qn, before, out, ref)


@pytest.mark.parametrize("cap", [200, 2600])      # one kernel, and the kernels for long caches
def test_fork_and_join_around_the_calls(cap):
    """Lengths, queries and new keys made by other kernels just before each call, on a
    forked stream and on the call's own, run eagerly and as a captured graph."""
    S, H, d, page = 5, 4, 64, 32
    cache, _, _ = make_cache(S, [100, 31, 64, 1, 150], H, 2, d, page, "bf16", seed=23)
    start = torch.tensor([90, 20, 50, 0, 140], dtype=torch.int32, device=DEV)
    spec, inv, pa = spec_of(32, 1, False)
    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    src = torch.randn(S, H + 4, d, device=DEV).bfloat16()
    new = torch.zeros_like(src)
    ws = b.dilution_attn_paged_decode_workspace(cache, cap)
    ws2 = b.dilution_attn_paged_append_workspace(cache)
    qn, out = torch.empty(2, S, H, d, dtype=torch.bfloat16, device=DEV).unbind(0)
    pools = [x.clone() for x in (cache.k_pages, cache.v_pages, cache.demand_pages)]
    work, work2 = torch.zeros(2, 1 << 22, device=DEV).unbind(0)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        work.add_(1.0)                                   # something long before the writes below
        cache.seq_lens.add_(1)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            work.mul_(0.5)
            new.copy_(src)
            new.mul_(2.0)
            b.dilution_attn_paged_append(new[:, :H], new[:, H:H + 2], new[:, H + 2:], cache, cu, qn, rope=spec, workspace=ws2)
        work2.sub_(1.0)
        main.wait_stream(side)
        b.dilution_attn_paged_decode(qn, cache, cap, out, workspace=ws)

    def reset():
        for x, y in zip((cache.k_pages, cache.v_pages, cache.demand_pages), pools):
            x.copy_(y)
        cache.seq_lens.copy_(start)

    def expect(steps):
        """The same steps one at a time, each against the oracle."""
        reset()
        outs = []
        for _ in range(steps):
            cache.seq_lens.add_(1)
            two = src * 2
            torch.cuda.synchronize()
            q = b.dilution_attn_paged_append(two[:, :H], two[:, H:H + 2], two[:, H + 2:], cache, cu, rope=spec)
            torch.cuda.synchronize()
            before, ref = cache.demand_pages.clone(), oracle_step(cache, q)
            torch.cuda.synchronize()
            o = b.dilution_attn_paged_decode(q, cache, cap)
            torch.cuda.synchronize()
            check_step(cache, q, before, o, ref)
            outs.append(o)
        return outs[-1], cache.demand_pages.clone()

    want, demand = expect(8)
    reset()
    for _ in range(8):
        step()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(cache.demand_pages, demand)
    reset()
    capture = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=capture):
        step()
    reset()
    out.zero_()
    for _ in range(8):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(cache.demand_pages, demand)
    assert b.dilution_attn_get_error(ws) == b.DA_OK and b.dilution_attn_get_error(ws2) == b.DA_OK
