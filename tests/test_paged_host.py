"""CPU checks of the rotary and paged entry points: refusals before any CUDA
call, the oracle's own pins and the host helpers."""
import ctypes
import math

import numpy as np
import pytest

import oracle.dilution as od
from long_context_attention_gb300 import binding as b
from long_context_attention_gb300 import rope_inv_freq, rope_pair_axis
from oracle import paged as op

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    return b.load()


def spec(n=32, axes=1, adjacent=0, inv=FAKE, pair_axis=()):
    pa = list(pair_axis) or [0] * n
    return b._CRopeSpec(inv, n, axes, adjacent, (ctypes.c_uint8 * 64)(*pa[:64]))


def test_rope_refusals(lib):
    def call(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, pos=FAKE, pb=1, sp=None, B=1, Hq=2, Hk=2, T=8, d=64, dtype=1, qs=None,
             qos=None, fn="dilution_attn_rope"):
        s = spec() if sp is None else sp
        arr = lambda x: None if x is None else (ctypes.c_int64 * 3)(*x)
        return getattr(lib, fn)(q, arr(qs), k, None, qo, arr(qos), ko, None, pos, pb, ctypes.byref(s), B, Hq, Hk, T, d,
                                dtype, None)
    for fn in ("dilution_attn_rope", "dilution_attn_rope_bwd"):
        assert call(fn=fn, q=None) == b.DA_ERR_INVALID
        assert call(fn=fn, qo=None) == b.DA_ERR_INVALID
        assert call(fn=fn, k=None) == b.DA_ERR_INVALID
        assert call(fn=fn, pos=None) == b.DA_ERR_INVALID
        assert call(fn=fn, q=FAKE + 1) == b.DA_ERR_INVALID                 # not aligned to an element
        assert call(fn=fn, q=FAKE + 2, dtype=0) == b.DA_ERR_INVALID
        assert call(fn=fn, dtype=2) == b.DA_ERR_INVALID
        assert call(fn=fn, d=96) == b.DA_ERR_UNSUPPORTED
        assert call(fn=fn, T=-1) == b.DA_ERR_INVALID
        assert call(fn=fn, T=(1 << 24) + 1) == b.DA_ERR_UNSUPPORTED
        assert call(fn=fn, pb=2) == b.DA_ERR_INVALID                       # neither 1 nor B
        assert call(fn=fn, sp=spec(n=33)) == b.DA_ERR_INVALID              # 66 elements of 64
        assert call(fn=fn, sp=spec(axes=0)) == b.DA_ERR_INVALID
        assert call(fn=fn, sp=spec(axes=5)) == b.DA_ERR_INVALID
        assert call(fn=fn, sp=spec(adjacent=2)) == b.DA_ERR_INVALID
        assert call(fn=fn, sp=spec(inv=None)) == b.DA_ERR_INVALID
        assert call(fn=fn, sp=spec(axes=2, pair_axis=[0, 2] + [0] * 30)) == b.DA_ERR_INVALID
        assert call(fn=fn, qs=(-64, 64, 64)) == b.DA_ERR_INVALID
        # outputs that address an element twice
        assert call(fn=fn, qos=(1024, 0, 64)) == b.DA_ERR_INVALID
        assert call(fn=fn, qos=(1024, 64, 64)) == b.DA_ERR_INVALID
        assert call(fn=fn, qos=(1024, 512, 32)) == b.DA_ERR_INVALID
        assert call(fn=fn, qos=(1024, 100, 64)) == b.DA_ERR_INVALID
        # empty problems do nothing, whatever the pointers
        assert call(fn=fn, q=None, T=0) == b.DA_OK
        assert call(fn=fn, q=None, B=0, pb=0) == b.DA_OK


def cache(S=2, Hq=4, Hkv=2, d=64, page_size=16, num_pages=8, num_demand_pages=8, max_pages=4, dtype=1, **ptr):
    p = dict(k_pages=FAKE, v_pages=FAKE, demand_pages=FAKE, page_table=FAKE, demand_table=FAKE, seq_lens=FAKE)
    p.update(ptr)
    return b._CPagedCache(*p.values(), S, Hq, Hkv, d, page_size, num_pages, num_demand_pages, max_pages, dtype)


BAD_CACHES = [(dict(S=-1), b.DA_ERR_INVALID), (dict(Hq=5), b.DA_ERR_INVALID), (dict(Hkv=0), b.DA_ERR_INVALID),
              (dict(d=32), b.DA_ERR_UNSUPPORTED), (dict(page_size=24), b.DA_ERR_UNSUPPORTED),
              (dict(page_size=8), b.DA_ERR_UNSUPPORTED), (dict(page_size=512), b.DA_ERR_UNSUPPORTED),
              (dict(page_size=0), b.DA_ERR_INVALID), (dict(num_pages=-1), b.DA_ERR_INVALID),
              (dict(max_pages=-1), b.DA_ERR_INVALID), (dict(dtype=3), b.DA_ERR_INVALID),
              (dict(k_pages=None), b.DA_ERR_INVALID), (dict(v_pages=FAKE + 8), b.DA_ERR_INVALID),
              (dict(demand_pages=FAKE + 4), b.DA_ERR_INVALID), (dict(page_table=None), b.DA_ERR_INVALID),
              (dict(demand_table=FAKE + 2), b.DA_ERR_INVALID), (dict(seq_lens=None), b.DA_ERR_INVALID),
              (dict(max_pages=1 << 21), b.DA_ERR_UNSUPPORTED)]


def test_append_refusals(lib):
    def call(c=None, q=FAKE, k=FAKE, v=FAKE, qo=FAKE, cu=FAKE, N=4, sp=None, ws=FAKE, wsb=256, ks=None, dem=None):
        c = cache() if c is None else c
        arr = None if ks is None else (ctypes.c_int64 * 2)(*ks)
        return lib.dilution_attn_paged_append(q, None, k, arr, v, None, dem, None, qo, cu, N, ctypes.byref(c),
                                              None if sp is None else ctypes.byref(sp), None, ws, wsb, None)
    for kw, want in BAD_CACHES:
        assert call(cache(**kw)) == want, kw
    assert lib.dilution_attn_paged_append(None, None, FAKE, None, FAKE, None, None, None, None, FAKE, 4, None, None,
                                          None, FAKE, 256, None) == b.DA_ERR_INVALID
    assert call(k=None) == b.DA_ERR_INVALID
    assert call(v=None) == b.DA_ERR_INVALID
    assert call(cu=None) == b.DA_ERR_INVALID
    assert call(q=None) == b.DA_ERR_INVALID            # q_out without q
    assert call(qo=None) == b.DA_ERR_INVALID           # q without q_out
    assert call(N=-1) == b.DA_ERR_INVALID
    assert call(ks=(-1, 64)) == b.DA_ERR_INVALID
    assert call(dem=FAKE + 2) == b.DA_ERR_INVALID
    assert call(sp=spec(n=40)) == b.DA_ERR_INVALID
    assert call(ws=None) == b.DA_ERR_WORKSPACE
    assert call(wsb=255) == b.DA_ERR_WORKSPACE
    assert call(ws=FAKE + 16) == b.DA_ERR_INVALID
    assert call(N=0, k=None) == b.DA_OK
    assert call(cache(S=0), k=None) == b.DA_OK


def test_decode_refusals(lib):
    def call(c=None, q=FAKE, out=FAKE, pt=None, npp=0, max_len=64, tau=1.0, tau_bh=None, eps=1e-6, flags=0, ws=FAKE,
             wsb=1 << 30):
        c = cache() if c is None else c
        return lib.dilution_attn_paged_decode(q, ctypes.byref(c), pt, npp, max_len, out, tau, tau_bh, eps, flags, ws,
                                              wsb, None)
    for kw, want in BAD_CACHES:
        assert call(cache(**kw)) == want, kw
    assert call(q=None) == b.DA_ERR_INVALID
    assert call(out=FAKE + 8) == b.DA_ERR_INVALID
    assert call(max_len=65) == b.DA_ERR_INVALID        # longer than the tables
    assert call(max_len=-1) == b.DA_ERR_INVALID
    assert call(npp=1) == b.DA_ERR_INVALID             # a prefix without its table
    assert call(pt=FAKE, npp=5) == b.DA_ERR_INVALID    # longer than max_len
    assert call(pt=FAKE + 2, npp=1) == b.DA_ERR_INVALID
    assert call(tau=-1.0) == b.DA_ERR_INVALID
    assert call(tau=float("nan")) == b.DA_ERR_INVALID
    assert call(eps=0.0) == b.DA_ERR_INVALID
    assert call(eps=1e-20) == b.DA_ERR_UNSUPPORTED     # bf16
    assert call(flags=b.DA_FLAG_KEEP_FOR_BACKWARD) == b.DA_ERR_INVALID
    assert call(tau_bh=FAKE + 2) == b.DA_ERR_INVALID
    assert call(ws=None) == b.DA_ERR_WORKSPACE
    assert call(wsb=300) == b.DA_ERR_WORKSPACE
    assert call(ws=FAKE + 16) == b.DA_ERR_INVALID
    assert call(cache(S=0), q=None) == b.DA_OK


def test_decode_with_a_status_block_refuses_bad_ones(lib):
    def call(status, ws=FAKE, wsb=1 << 30, max_len=64):
        return lib.dilution_attn_paged_decode_ex(FAKE, ctypes.byref(cache()), None, 0, max_len, FAKE, 1.0, None, 1e-6, 0,
                                                 ws, wsb, status, None)
    assert call(None) == b.DA_ERR_INVALID
    assert call(FAKE + 16) == b.DA_ERR_INVALID
    assert call(FAKE, ws=None) == b.DA_ERR_WORKSPACE
    assert call(FAKE, wsb=300) == b.DA_ERR_WORKSPACE
    assert call(FAKE, max_len=65) == b.DA_ERR_INVALID


def test_stall_hook_refusals(lib):
    def call(kernel=0, block=0, limit=2_000_000, c=None, ws=FAKE):
        c = cache() if c is None else c
        return lib.dilution_attn_debug_paged_decode_stall(FAKE, ctypes.byref(c), None, 0, 64, FAKE, 1.0, 1e-6, ws, 1 << 30,
                                                          None, kernel, block, limit)
    for bad in (dict(kernel=-1), dict(kernel=4), dict(block=-1), dict(limit=999), dict(limit=1_000_000_001),
                dict(c=cache(Hq=5))):
        assert call(**bad) == b.DA_ERR_INVALID, bad
    assert call(ws=None) == b.DA_ERR_WORKSPACE


def test_outputs_that_lie_over_inputs_are_refused(lib):
    """Rows written by one block that another still has to read: an output at an input's address with other strides,
    or at another operand's address."""
    def rope(q=FAKE, k=FAKE << 4, qo=FAKE << 5, ko=FAKE << 6, qs=None, ks=None, qos=None):
        arr = lambda x: None if x is None else (ctypes.c_int64 * 3)(*x)
        return lib.dilution_attn_rope(q, arr(qs), k, arr(ks), qo, arr(qos), ko, None, FAKE, 1, ctypes.byref(spec()), 2,
                                      2, 2, 8, 64, 1, None)
    fused = (8 * 256, 64, 256)                                # [B, T, 4 heads of 64]
    assert rope(qo=FAKE, qs=fused) == b.DA_ERR_INVALID        # a projection's queries, turned into its first half
    assert rope(qo=FAKE, qos=fused) == b.DA_ERR_INVALID
    assert rope(ko=FAKE << 4, ks=fused) == b.DA_ERR_INVALID
    assert rope(qo=FAKE, qs=(1024, 0, 64)) == b.DA_ERR_INVALID   # a head read twice, written in place
    assert rope(ko=FAKE << 5) == b.DA_ERR_INVALID             # both outputs in one place
    assert rope(qo=FAKE << 4) == b.DA_ERR_INVALID             # the queries over the keys
    assert rope(ko=FAKE) == b.DA_ERR_INVALID

    def append(q=FAKE, k=FAKE << 4, v=FAKE << 5, qo=FAKE, qs=None, ks=None, dem=None):
        arr = lambda x: None if x is None else (ctypes.c_int64 * 2)(*x)
        c = cache()
        return lib.dilution_attn_paged_append(q, arr(qs), k, arr(ks), v, None, dem, None, qo, FAKE, 4, ctypes.byref(c),
                                              None, None, FAKE, 256, None)
    assert append(qs=(8 * 64, 64)) == b.DA_ERR_INVALID                  # the first heads of a projection of 8
    assert append(qs=(4 * 64, 128)) == b.DA_ERR_INVALID
    assert append(qs=(0, 64)) == b.DA_ERR_INVALID
    assert append(qo=FAKE << 4) == b.DA_ERR_INVALID
    assert append(qo=FAKE << 5) == b.DA_ERR_INVALID
    row, n = 8 * 64 * 2, 4 * 4 * 64 * 2                                 # bytes of a projection's row and of q_out
    at = FAKE << 4
    assert append(qo=at + row, ks=(8 * 64, 64)) == b.DA_ERR_INVALID     # over the second token's keys
    assert append(qo=at + 3 * row + 2 * 128 - 16, ks=(8 * 64, 64)) == b.DA_ERR_INVALID   # the end of the last one
    assert append(qo=at - n + 16) == b.DA_ERR_INVALID                   # the beginning of the first
    assert append(q=FAKE, qo=FAKE + 1024) == b.DA_ERR_INVALID           # one token further on
    assert append(dem=FAKE << 6, qo=(FAKE << 6) + 32) == b.DA_ERR_INVALID


def test_workspace_sizes_grow(lib):
    size = b.dilution_attn_paged_decode_workspace_size
    assert size(4, 8, 2, 64, 1000, 0, 16, 1) > 256
    assert size(4, 8, 2, 96, 1000, 0, 16, 1) == 0
    assert size(4, 8, 2, 64, 1000, 63, 16, 1) == 0     # the prefix is longer than max_len
    assert size(8, 8, 2, 64, 1000, 0, 16, 1) >= size(4, 8, 2, 64, 1000, 0, 16, 1)
    assert b.dilution_attn_paged_append_workspace_size() == 256


def test_binding_refuses_what_is_not_on_the_gpu():
    import torch
    with pytest.raises(ValueError):
        b.rope_spec(torch.ones(8))
    with pytest.raises(ValueError):
        b.PagedCache(*[torch.zeros(1)] * 6)
    with pytest.raises(TypeError):
        b.dilution_attn_paged_decode(torch.zeros(1, 1, 64), None, 4)


def test_host_helpers():
    f = rope_inv_freq(64, 10000.0)
    assert f.shape == (32,) and float(f[0]) == 1.0
    assert math.isclose(float(f[31]), 10000.0 ** (-31 / 32), rel_tol=1e-6)
    assert rope_pair_axis(6, 3) == [0, 0, 1, 1, 2, 2]
    assert rope_pair_axis(7, 3, interleaved=True) == [0, 1, 2, 0, 1, 2, 0]
    assert rope_pair_axis(4, 1) == [0] * 4
    assert rope_pair_axis(6, (1, 2, 3)) == [0, 1, 1, 2, 2, 2]
    with pytest.raises(ValueError):
        rope_pair_axis(6, (1, 2))


# ------------------------------------------------------------------------- the oracle's pins
def test_oracle_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 8))
    ang = op.rope_angles(np.arange(5)[None], [1.0, 0.25, 0.0], [0, 0, 0])
    for adjacent in (False, True):
        y = op.rotate(x, ang, adjacent)
        assert np.allclose(op.rotate(y, ang, adjacent, back=True), x)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[:, 6:], x[:, 6:])
        # scores depend on the distance of positions alone
        z = rng.standard_normal(8)
        a1 = op.rope_angles(np.array([[7], ]), [1.0, 0.25, 0.5], [0, 0, 0])[0]
        a2 = op.rope_angles(np.array([[3], ]), [1.0, 0.25, 0.5], [0, 0, 0])[0]
        a4 = op.rope_angles(np.array([[4], ]), [1.0, 0.25, 0.5], [0, 0, 0])[0]
        assert np.isclose(op.rotate(z, a1, adjacent)[:6] @ op.rotate(x[0], a2, adjacent)[:6],
                          op.rotate(z, a4, adjacent)[:6] @ x[0][:6])
    y = op.rotate(np.array([1.0, 0.0, 2.0, 5.0]), np.array([math.pi / 2]))
    assert np.allclose(y, [0.0, 1.0, 2.0, 5.0])


@pytest.mark.parametrize("earlier", [False, True])
def test_oracle_paged_step_is_the_contiguous_step(earlier):
    """Scattered over pages, a step is the oracle's contiguous decode step (the
    last key's demand starts at 0)."""
    rng = np.random.default_rng(3)
    n, d, page, H = 21, 8, 4, 2
    k, v = rng.standard_normal((2, H, n, d))
    dem = rng.random((H, n))
    dem[:, -1] = 0.0
    q = rng.standard_normal((1, H, d))
    pages = [5, 2, 7, 0, 3, 6]
    kp, vp, dp = np.full((8, H, page, d), np.nan), np.full((8, H, page, d), np.nan), np.full((8, H, page), np.nan)
    for t in range(n):
        kp[pages[t // page], :, t % page] = k[:, t]
        vp[pages[t // page], :, t % page] = v[:, t]
        dp[pages[t // page], :, t % page] = dem[:, t]
    out, D, _ = op.paged_decode(q, kp, vp, dp, [pages], [pages], [n], 1.2, 1e-4, earlier)
    out2, _, _ = op.paged_decode(q, kp, vp, dp, [[-1, -1] + pages[2:]], [pages], [n], 1.2, 1e-4, earlier, pages[:2])
    assert np.array_equal(out, out2)
    for h in range(H):
        x = 1.2 * (k[h] @ q[0, h]) / math.sqrt(d)
        p = np.exp(x) / np.exp(x).sum()
        share = p / ((dem[h] if earlier else dem[h] + p) + 1e-4)
        assert np.allclose(out[0, h], share @ v[h] / share.sum())
        got = np.array([D[pages[t // page], h, t % page] for t in range(n)])
        assert np.allclose(got, dem[h] + p)
        if not earlier:
            ref = od.dilution_decode_step_head(q[0, h], k[h, -1], v[h, -1], k[h, :], v[h, :], dem[h], n - 1, 1.2, 1e-4)
            assert np.allclose(out[0, h], ref[0]) and np.allclose(got, ref[1])
