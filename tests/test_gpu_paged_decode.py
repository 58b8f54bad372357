"""GPU parity of dilution_attn_paged_decode against the float64 oracle: ragged
lengths, page sizes, shared heads, shared prefixes, options, masked rows full
of NaN, bad tables, graphs and streams."""
import numpy as np
import pytest
import torch

from long_context_attention_gb300 import binding as b
from tests._paged import DEV, LONG, both_sizes, check_step, make_cache, oracle_step, step_and_check
from tests._parity import host64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,lens,Hq,Hkv,d,page", [
    (1, [1], 1, 1, 64, 16),
    (1, [500], 12, 12, 64, 16),
    (3, [1, 0, 129], 4, 2, 64, 16),
    (4, [127, 128, 129, 257], 6, 2, 128, 32),
    (5, [16, 17, 1000, 64, 63], 8, 1, 64, 64),
    (2, [700, 3], 16, 1, 128, 128),
    (2, [300, 2], 34, 2, 64, 32),          # 17 query heads a key head: more than one 16-row tile
    (2, [2049, 1025], 3, 3, 128, 256),
    (9, [0, 0, 5, 0, 1, 33, 0, 400, 0], 2, 2, 64, 16),
])
def test_ragged_decode_matches_oracle(dtype, S, lens, Hq, Hkv, d, page):
    cache, q, _ = make_cache(S, lens, Hq, Hkv, d, page, dtype, seed=sum(lens) + Hq)
    both_sizes(cache, q, max(lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 8, 12])
def test_long_runs_of_tiles(G, d, dtype):
    # every CTA takes many tiles in a row, across sequences: 2 CTAs on 152 SMs share 2 x 40000 keys of 4 heads
    cache, q, _ = make_cache(3, [40000, 20001, 30], 4 * G, 4, d, 64, dtype, seed=90 + G)
    before = cache.demand_pages.clone()
    out = b.dilution_attn_paged_decode(q, cache, 40000)
    # the oracle on one query head of every sequence
    for h in (G - 1, 4 * G - 1):
        one = b.PagedCache(cache.k_pages[:, h // G:h // G + 1].contiguous(), cache.v_pages[:, h // G:h // G + 1].contiguous(),
                           before[:, h:h + 1].contiguous(), cache.page_table, cache.demand_table, cache.seq_lens)
        qh = q[:, h:h + 1].contiguous()
        ref = oracle_step(one, qh)
        old = one.demand_pages.clone()
        one.demand_pages.copy_(cache.demand_pages[:, h:h + 1])
        check_step(one, qh, old, out[:, h:h + 1], ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_all_idle(dtype):
    cache, q, _ = make_cache(3, [0, 0, 0], 4, 2, 64, 16, dtype)
    before = cache.demand_pages.clone()
    out = torch.full_like(q, 7.0)
    for max_len in (0, 16):
        b.dilution_attn_paged_decode(q, cache, max_len, out)
        assert not out.any() and torch.equal(cache.demand_pages, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3.0e38])
def test_rows_past_the_end_are_never_used(dtype, junk):
    cache, q, _ = make_cache(4, [1, 15, 130, 333], 4, 2, 64, 32, dtype, seed=5, junk=junk)
    both_sizes(cache, q, 352)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,own,Hq,Hkv,d,page,prefix", [
    (2, [1, 2], 1, 1, 64, 16, 16),
    (5, [1, 40, 130, 7, 300], 4, 2, 64, 16, 272),
    (17, [1 + 13 * i for i in range(17)], 2, 2, 128, 64, 448),
    (3, [5, 1, 129], 8, 1, 128, 128, 128),
    (40, [1 + i % 5 for i in range(40)], 6, 2, 64, 32, 160),
    (70, [1 + i % 3 for i in range(70)], 4, 1, 64, 16, 144),     # 280 rows of one key head
    (36, [2 + i % 7 for i in range(36)], 8, 2, 128, 16, 400),
    (17, [1 + i for i in range(17)], 1, 1, 64, 256, 1024),        # one row past 16; pages of two tiles
    (33, [3] * 33, 4, 2, 128, 32, 32),                            # a prefix shorter than a tile
    (20, [1 + i for i in range(20)], 14, 2, 64, 64, 4096),        # 140 rows in three 64-row segments
])
def test_shared_prefix_matches_oracle(dtype, S, own, Hq, Hkv, d, page, prefix):
    lens = [prefix + n for n in own]
    cache, q, pt = make_cache(S, lens, Hq, Hkv, d, page, dtype, seed=S + prefix, prefix=prefix)
    both_sizes(cache, q, max(lens), prefix_table=pt)


# Prefixes long enough for the kernels that take many rows at once (17 rows of a key
# head and 2^22 (row, key, key head) triples), and one that stays below them.
LONG_PREFIX = [
    (64, 20, 8, 2, 32, 26240),        # 80 rows in two segments of 40, 205 tiles each, cut over all CTAs
    (128, 20, 8, 2, 32, 26240),
    (64, 17, 8, 8, 16, 30848),        # 17 rows: one in the second half
    (128, 11, 12, 4, 64, 32768),      # 33 rows
    (64, 65, 2, 1, 16, 32272),        # 130 rows in three segments; a last tile of 16 keys
    (128, 64, 1, 1, 256, 65792),      # 64 rows; pages of two tiles, the last tile's page half used
    (64, 48, 6, 3, 128, 14592),       # 96 rows in two segments of 48
    (64, 12, 4, 4, 256, 132096),      # 12 rows: 16-row segments, keys that do not stay in L2
]


@pytest.mark.parametrize("d,S,Hq,Hkv,page,prefix", LONG_PREFIX)
def test_long_prefix_with_idle_slots(d, S, Hq, Hkv, page, prefix):
    lens = [0 if i % 7 == 2 else prefix + i % 40 for i in range(S)]
    cache, q, pt = make_cache(S, lens, Hq, Hkv, d, page, "bf16", seed=97 + d + S, prefix=prefix)
    before = cache.demand_pages.clone()
    for flags in (0, b.DA_FLAG_EARLIER_DEMAND_ONLY):
        cache.demand_pages.copy_(before)
        out = b.dilution_attn_paged_decode(q, cache, max(lens), prefix_table=pt, flags=flags, eps=1e-4)
        for h, rows in ((Hq - 1, [0, 1, 2, S - 1]), (0, [S // 2, S // 2 + 1])):   # the oracle on a query head of some
            kv = h // (Hq // Hkv)
            one = b.PagedCache(cache.k_pages[:, kv:kv + 1].contiguous(), cache.v_pages[:, kv:kv + 1].contiguous(),
                               before[:, h:h + 1].contiguous(), cache.page_table[rows].contiguous(),
                               cache.demand_table[rows].contiguous(), cache.seq_lens[rows].contiguous())
            ref = oracle_step(one, q[rows, h:h + 1], eps=1e-4, earlier=bool(flags))
            mine = torch.zeros(one.demand_pages.shape[0], dtype=torch.bool, device=DEV)
            mine[one.demand_table[one.demand_table >= 0].long()] = True
            old = one.demand_pages.clone()
            one.demand_pages[mine] = cache.demand_pages[mine, h:h + 1]
            check_step(one, q[rows, h:h + 1], old, out[rows, h:h + 1], ref)


@pytest.mark.parametrize("d,S,Hq,Hkv,page,prefix", LONG_PREFIX[:3])
def test_long_prefix_reports_bad_pages_and_repeats_its_bits(d, S, Hq, Hkv, page, prefix):
    lens = [prefix + 1 + i for i in range(S)]
    cache, q, pt = make_cache(S, lens, Hq, Hkv, d, page, "bf16", seed=3, prefix=prefix)
    ws = b.dilution_attn_paged_decode_workspace(cache, max(lens), 1)     # the size knows no length of the prefix
    before = cache.demand_pages.clone()

    def run(table=pt):
        cache.demand_pages.copy_(before)
        out = b.dilution_attn_paged_decode(q, cache, max(lens), prefix_table=table, workspace=ws)
        return out, cache.demand_pages.clone(), b.dilution_attn_get_error(ws)

    good, demand, status = run()
    assert status == b.DA_OK
    again, demand2, _ = run()
    assert torch.equal(good, again) and torch.equal(demand, demand2)
    for bad in (-1, -7, cache.k_pages.shape[0], 1 << 30):
        table = pt.clone()
        table[table.numel() // 2] = bad
        assert run(table)[2] == b.DA_ERR_INVALID
    for bad in (-1, cache.demand_pages.shape[0], 1 << 30):               # sequence 4 alone suffers
        keep = cache.demand_table[4, 3].item()
        cache.demand_table[4, 3] = bad
        out, new, status = run()
        cache.demand_table[4, 3] = keep
        others = [i for i in range(S) if i != 4]
        assert status == b.DA_ERR_INVALID and torch.equal(out[others], good[others])
        theirs = cache.demand_table[others].flatten().unique().long()
        theirs = theirs[theirs >= 0]
        assert torch.equal(new[theirs], demand[theirs])
        assert torch.equal(new[keep], before[keep])                      # the page that lost its place
    assert torch.equal(run()[0], good)


# Prefixes that end inside a tile of the kernels that take many rows at once.
@pytest.mark.parametrize("flags", [0, b.DA_FLAG_EARLIER_DEMAND_ONLY])
@pytest.mark.parametrize("page,prefix", [(16, 26256), (32, 26272), (64, 26304)])
@pytest.mark.parametrize("d", [64, 128])
def test_long_prefix_whose_logits_lie_far_below_zero(d, page, prefix, flags):
    # a strong common component of the keys, which the queries oppose: every logit is near -150.  A softmax does not
    # depend on the offset, so the bids are ordinary; 2^(0 - lse2) of a place without a key is not.
    S, Hq, Hkv = 20, 8, 2
    lens = [prefix + 1 + i for i in range(S)]
    cache, q, pt = make_cache(S, lens, Hq, Hkv, d, page, "bf16", seed=d + page, prefix=prefix)
    g = torch.Generator(device=DEV).manual_seed(prefix)
    u = torch.randint(0, 2, (d,), generator=g, device=DEV) * 2.0 - 1.0
    cache.k_pages.copy_(4.0 * u + 0.3 * torch.randn(cache.k_pages.shape, generator=g, device=DEV))
    q.copy_(-150.0 / (4.0 * d ** 0.5) * u * (1.0 + 0.05 * torch.rand(q.shape, generator=g, device=DEV)))
    before = cache.demand_pages.clone()
    ws = b.dilution_attn_paged_decode_workspace(cache, max(lens), prefix // page)
    out = b.dilution_attn_paged_decode(q, cache, max(lens), prefix_table=pt, workspace=ws, flags=flags, eps=1e-4)
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    assert out.isfinite().all() and cache.demand_pages.isfinite().all()
    for h, rows in ((0, [0, 7]), (Hq - 1, [S - 1])):
        kv = h // (Hq // Hkv)
        one = b.PagedCache(cache.k_pages[:, kv:kv + 1].contiguous(), cache.v_pages[:, kv:kv + 1].contiguous(),
                           before[:, h:h + 1].contiguous(), cache.page_table[rows].contiguous(),
                           cache.demand_table[rows].contiguous(), cache.seq_lens[rows].contiguous())
        ref = oracle_step(one, q[rows, h:h + 1], eps=1e-4, earlier=bool(flags))
        mine = torch.zeros(one.demand_pages.shape[0], dtype=torch.bool, device=DEV)
        mine[one.demand_table[one.demand_table >= 0].long()] = True
        old = one.demand_pages.clone()
        one.demand_pages[mine] = cache.demand_pages[mine, h:h + 1]
        check_step(one, q[rows, h:h + 1], old, out[rows, h:h + 1], ref)


@pytest.mark.parametrize("d,S,Hq,Hkv,page,prefix", [(64, 9, 4, 2, 64, 8192), (128, 3, 12, 2, 16, 6160), (64, 20, 1, 1, 256, 12288)])
def test_long_prefix_in_fp32(d, S, Hq, Hkv, page, prefix):
    # 18 to 20 rows of a key head: a segment of 16 and one of the rest
    lens = [0 if i == 1 else prefix + 3 * i for i in range(S)]
    cache, q, pt = make_cache(S, lens, Hq, Hkv, d, page, "f32", seed=prefix, prefix=prefix)
    step_and_check(cache, q, max(lens), prefix_table=pt)


@pytest.mark.parametrize("d,S,Hq,Hkv,page,prefix", LONG_PREFIX[:4])
def test_captured_step_behind_a_long_prefix(d, S, Hq, Hkv, page, prefix):
    # the kernels for many rows in a graph, replayed over lengths that change on the device: the bits of eager calls
    cache, q, pt = make_cache(S, [prefix + 40] * S, Hq, Hkv, d, page, "bf16", seed=S, prefix=prefix)
    ws = b.dilution_attn_paged_decode_workspace(cache, prefix + 40)
    before, out = cache.demand_pages.clone(), torch.empty_like(q)
    b.dilution_attn_paged_decode(q, cache, prefix + 40, out, prefix_table=pt, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.dilution_attn_paged_decode(q, cache, prefix + 40, out, prefix_table=pt, workspace=ws)
    for step in range(3):
        cache.seq_lens.copy_(torch.tensor([0 if (i + step) % 9 == 4 else prefix + (7 * i + step) % 40 for i in range(S)],
                                          dtype=torch.int32))
        cache.demand_pages.copy_(before)
        want = b.dilution_attn_paged_decode(q, cache, prefix + 40, prefix_table=pt)
        demand = cache.demand_pages.clone()
        cache.demand_pages.copy_(before)
        out.fill_(9.0)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(cache.demand_pages, demand)
        assert b.dilution_attn_get_error(ws) == b.DA_OK and b.dilution_attn_get_error(cache.status) == b.DA_OK


def test_more_sequences_than_one_part():
    lens = [64 + i % 3 for i in range(900)]
    cache, q, pt = make_cache(900, lens, 1, 1, 64, 16, "bf16", seed=98, prefix=64)
    tau = torch.linspace(0.5, 1.5, 900, device=DEV)
    step_and_check(cache, q, 66, tau_bh=tau)
    step_and_check(cache, q, 66, tau_bh=tau, prefix_table=pt)


def test_parts_that_take_their_prefix_differently():
    # 900 sequences go as 704 and 196: 704 rows x 8192 keys to the kernels for many rows, the rest to the streaming ones
    S, prefix = 900, 8192
    lens = [0 if i % 50 == 0 else prefix + i % 70 for i in range(S)]
    cache, q, pt = make_cache(S, lens, 1, 1, 64, 64, "bf16", seed=7, prefix=prefix, extra_width=1)
    before = cache.demand_pages.clone()
    out = b.dilution_attn_paged_decode(q, cache, max(lens), prefix_table=pt)
    assert b.dilution_attn_get_error(cache.status) == b.DA_OK
    rows = [0, 1, 333, 703, 704, 750, 899]
    one = b.PagedCache(cache.k_pages, cache.v_pages, before.clone(), cache.page_table[rows].contiguous(),
                       cache.demand_table[rows].contiguous(), cache.seq_lens[rows].contiguous())
    ref = oracle_step(one, q[rows])
    mine = one.demand_table[one.demand_table >= 0].long()
    one.demand_pages[mine] = cache.demand_pages[mine]
    check_step(one, q[rows], before, out[rows], ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,Hq,Hkv,d,page,prefix", [(5, 4, 2, 64, 16, 272), (3, 4, 4, 128, 64, 2048)])
def test_max_len_is_the_prefix(S, Hq, Hkv, d, page, prefix, dtype):
    lens = [0 if i == 3 else prefix for i in range(S)]
    cache, q, pt = make_cache(S, lens, Hq, Hkv, d, page, dtype, seed=3, prefix=prefix)
    step_and_check(cache, q, prefix, prefix_table=pt)


@pytest.mark.parametrize("dtype,S,Hq,page,prefix,lens", [
    ("bf16", 3, 4, 64, 0, [700, 300, 1]), ("bf16", 3, 4, 64, 0, [7000, 3000, 1]), ("f32", 3, 4, 64, 0, [700, 300, 1]),
    ("bf16", 20, 8, 64, 26304, [26304 + i for i in range(20)])])
def test_demand_pool_past_32_bit_offsets(dtype, S, Hq, page, prefix, lens):
    # the same pages at the end of a pool of more than 2^31 floats: the same bits, of an append and of a step
    small, q, pt = make_cache(S, lens, Hq, 2, 64, page, dtype, seed=9, prefix=prefix)
    n = small.demand_pages.shape[0]
    skip = (1 << 31) // (Hq * page) + 3
    pool = torch.empty(skip + n, Hq, page, device=DEV)
    pool[skip:] = small.demand_pages
    table = torch.where(small.demand_table >= 0, small.demand_table + skip, small.demand_table)
    big = b.PagedCache(small.k_pages, small.v_pages, pool, small.page_table, table, small.seq_lens)
    k, demand = torch.randn(S, 2, 64, device=DEV).to(q.dtype), torch.rand(S, Hq, device=DEV)
    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    outs = []
    for c in (big, small):
        b.dilution_attn_paged_append(None, k, k, c, cu, demand=demand)
        outs.append(b.dilution_attn_paged_decode(q, c, max(lens), prefix_table=pt))
        assert b.dilution_attn_get_error(c.status) == b.DA_OK
    assert torch.equal(*outs) and torch.equal(pool[skip:], small.demand_pages)


def test_threads_with_their_own_streams():
    """Four host threads append and decode at once, each on its own stream and cache: the bits of one after another."""
    import threading
    cases = [(5, [300, 7, 130, 1, 900], 4, 2, 64, 32, "bf16", 0, 900), (4, [5000, 1, 0, 3000], 8, 2, 128, 64, "bf16", 0, 5000),
             (3, [70, 2600, 500], 4, 4, 64, 16, "f32", 0, 2600), (20, [26272 + i for i in range(20)], 8, 2, 64, 32, "bf16", 26272, 26291)]
    made, want, got = [], [], [None] * len(cases)
    for i, (S, lens, Hq, Hkv, d, page, dtype, prefix, cap) in enumerate(cases):
        cache, q, pt = make_cache(S, lens, Hq, Hkv, d, page, dtype, seed=200 + i, prefix=prefix)
        k = torch.randn(S, Hkv, d, device=DEV).to(q.dtype)
        cu = torch.tensor([0] + list(np.cumsum([min(n, 1) for n in lens])), dtype=torch.int32, device=DEV)
        made.append((cache, q, pt, k, cu, cap, b.dilution_attn_paged_decode_workspace(cache, cap), torch.cuda.Stream()))

    def steps(i, stream):
        cache, q, pt, k, cu, cap, ws, _ = made[i]
        b.dilution_attn_paged_append(None, k, k, cache, cu, workspace=ws, stream=stream)
        for _ in range(5):
            out = b.dilution_attn_paged_decode(q, cache, cap, prefix_table=pt, workspace=ws, stream=stream)
        return out

    before = [m[0].demand_pages.clone() for m in made]
    torch.cuda.synchronize()
    for i in range(len(cases)):
        want.append((steps(i, None).clone(), made[i][0].demand_pages.clone()))
        made[i][0].demand_pages.copy_(before[i])
    torch.cuda.synchronize()
    gate = threading.Barrier(len(cases))

    def work(i):
        gate.wait()
        got[i] = steps(i, made[i][7])
        made[i][7].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, (out, demand) in enumerate(want):
        assert b.dilution_attn_get_error(made[i][6]) == b.DA_OK
        assert torch.equal(got[i], out) and torch.equal(made[i][0].demand_pages, demand), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_prefix_with_idle_slots_and_nothing_of_their_own(dtype):
    # idle slots among the sequences, and sequences that end with the prefix
    lens = [0, 160, 165, 0, 160, 300, 0]
    cache, q, pt = make_cache(7, lens, 4, 2, 64, 32, dtype, seed=9, prefix=160, junk=float("nan"))
    both_sizes(cache, q, 300, prefix_table=pt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_equals_the_same_pages_in_the_tables(dtype):
    lens = [512 + n for n in (3, 70, 200, 1)]
    cache, q, pt = make_cache(4, lens, 4, 2, 64, 64, dtype, seed=21, prefix=512)
    old = cache.demand_pages.clone()
    a = step_and_check(cache, q, 800, prefix_table=pt)
    da = cache.demand_pages.clone()
    cache.demand_pages.copy_(old)
    step_and_check(cache, q, 800)
    # two roundings of bids that differ by the order of their sums (see tests/_paged.py)
    assert torch.allclose(da, cache.demand_pages, rtol=1e-5, atol=1e-6)
    assert a.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_options(dtype):
    lens = [40, 0, 300]
    for flags, tau, per_head, prefix in ((b.DA_FLAG_EARLIER_DEMAND_ONLY, 1.3, False, 0), (0, 1.0, True, 0),
                                         (0, 0.0, False, 0), (b.DA_FLAG_EARLIER_DEMAND_ONLY, 1.0, True, 32),
                                         (0, 2.0, False, 32)):
        cache, q, pt = make_cache(3, lens, 4, 2, 64, 16, dtype, seed=31, prefix=prefix)
        tau_bh = torch.linspace(0.0, 2.0, 12, device=DEV) if per_head else None
        both_sizes(cache, q, 300, tau=tau, tau_bh=tau_bh, flags=flags, eps=1e-3, prefix_table=pt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sharp_logits(dtype):
    # one key takes nearly the whole bid of its row; another row is uniform
    cache, q, _ = make_cache(2, [200, 90], 2, 2, 64, 16, dtype, seed=41)
    q[0, 0] = cache.k_pages[int(cache.page_table[0, 3]), 0, 5] * 4
    q[1, 1] = 0
    both_sizes(cache, q, 200)


def test_max_len_beyond_every_sequence_and_repeats():
    cache, q, pt = make_cache(3, [70, 200, 64], 4, 2, 64, 32, "bf16", seed=51, prefix=64, extra_width=300)
    b.dilution_attn_paged_decode(q, cache, 200)         # whatever ran before
    old = cache.demand_pages.clone()
    outs = []
    for max_len, table in ((200, None), (9000, None), (200, pt), (200, pt), (9000, pt)):
        cache.demand_pages.copy_(old)
        outs.append((step_and_check(cache, q, max_len, prefix_table=table), cache.demand_pages.clone()))
    for _ in range(3):                                  # equal bits from equal calls, on every path
        for max_len, table in ((200, None), (200, pt), (9000, None), (9000, pt)):
            got = []
            for _ in range(2):
                cache.demand_pages.copy_(old)
                got.append((b.dilution_attn_paged_decode(q, cache, max_len, prefix_table=table),
                            cache.demand_pages.clone()))
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype,max_len", [("bf16", 224), ("bf16", LONG), ("f32", 224)])
@pytest.mark.parametrize("S", [3, 12])          # 12: 24 rows a key head at the prefix
def test_bad_device_data_is_reported(dtype, max_len, S):
    lens = [70, 200] + [64] * (S - 2)
    good, q, pt = make_cache(S, lens, 4, 2, 64, 32, dtype, seed=61, prefix=64)
    ws = b.dilution_attn_paged_decode_workspace(good, max_len)

    def after(change, prefix=None):
        cache, qq, _ = make_cache(S, lens, 4, 2, 64, 32, dtype, seed=61, prefix=64)
        change(cache)
        p = None if prefix is None else prefix.clone()
        b.dilution_attn_paged_decode(qq, cache, max_len, prefix_table=p, workspace=ws)
        first = b.dilution_attn_get_error(ws)
        assert b.dilution_attn_get_error(ws) == b.DA_OK      # read once
        return first

    assert after(lambda c: None) == b.DA_OK
    assert after(lambda c: c.seq_lens.__setitem__(1, max_len + 1)) == b.DA_ERR_INVALID
    assert after(lambda c: c.seq_lens.__setitem__(1, -1)) == b.DA_ERR_INVALID
    assert after(lambda c: c.seq_lens.__setitem__(1, 63), pt) == b.DA_ERR_INVALID     # shorter than the prefix
    assert after(lambda c: c.page_table.__setitem__((1, 3), -5)) == b.DA_ERR_INVALID
    assert after(lambda c: c.page_table.__setitem__((1, 3), 10 ** 6)) == b.DA_ERR_INVALID
    assert after(lambda c: c.demand_table.__setitem__((0, 0), 10 ** 6)) == b.DA_ERR_INVALID
    assert after(lambda c: c.page_table.__setitem__((1, 0), -5), pt) == b.DA_OK       # not read behind a prefix
    bad = pt.clone()
    bad[1] = 10 ** 6
    assert after(lambda c: None, bad) == b.DA_ERR_INVALID
    # the other sequences of a call with one bad length are right
    cache, qq, _ = make_cache(S, lens, 4, 2, 64, 32, dtype, seed=61)
    cache.seq_lens[1] = 0
    ref = oracle_step(cache, qq)
    cache.seq_lens[1] = max_len + 5
    out = b.dilution_attn_paged_decode(qq, cache, max_len, workspace=ws)
    assert b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID
    keep = [0] + list(range(2, S))
    assert np.abs(host64(out)[keep] - ref[0][keep]).max() <= 2e-2


@pytest.mark.parametrize("max_len,dtype", [(224, "bf16"), (LONG, "bf16"), (224, "f32")])
def test_errors_of_calls_without_a_workspace_stay_readable(max_len, dtype):
    lens = [70, 200, 64]
    cache, q, pt = make_cache(3, lens, 4, 2, 64, 32, dtype, seed=61, prefix=64)
    before = cache.demand_pages.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    good = b.dilution_attn_paged_decode(q, cache, max_len, prefix_table=pt)
    assert b.dilution_attn_get_error(cache.status) == b.DA_OK

    def step(**kw):
        cache.demand_pages.copy_(before)
        torch.cuda.synchronize()
        return b.dilution_attn_paged_decode(q, cache, max_len, **kw)

    cache.seq_lens[1] = max_len + 1
    step()
    assert b.dilution_attn_get_error(cache.status) == b.DA_ERR_INVALID
    assert b.dilution_attn_get_error(cache.status) == b.DA_OK          # read once
    step(stream=side)
    assert torch.equal(step(prefix_table=pt)[[0, 2]], good[[0, 2]])    # an error waits until it is read
    torch.cuda.synchronize()
    assert b.dilution_attn_get_error(cache.status, side) == b.DA_ERR_INVALID
    cache.seq_lens[1] = 200
    page = cache.page_table[1, 3].item()
    cache.page_table[1, 3] = 10 ** 6
    step()
    assert b.dilution_attn_get_error(cache.status) == b.DA_ERR_INVALID
    k = torch.zeros(3, 2, 64, dtype=q.dtype, device=DEV)
    cache.demand_table[0, 2] = -1
    b.dilution_attn_paged_append(None, k, k, cache, torch.arange(4, dtype=torch.int32, device=DEV))
    assert b.dilution_attn_get_error(cache.status) == b.DA_ERR_INVALID
    # a call with a workspace records in that
    ws = b.dilution_attn_paged_decode_workspace(cache, max_len)
    step(workspace=ws)
    assert b.dilution_attn_get_error(cache.status) == b.DA_OK and b.dilution_attn_get_error(ws) == b.DA_ERR_INVALID
    # a captured step without one
    cache.page_table[1, 3] = page
    cache.demand_table[0, 2] = 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.dilution_attn_paged_decode(q, cache, max_len)
    cache.page_table[1, 3] = -3
    graph.replay()
    assert b.dilution_attn_get_error(cache.status) == b.DA_ERR_INVALID and out.shape == q.shape


@pytest.mark.parametrize("max_len,dtype", [(264, "bf16"), (LONG, "bf16"), (264, "f32")])
def test_graph_replay_with_growing_sequences(max_len, dtype):
    # one captured step replays over lengths and tables that change on the device
    cache, q, pt = make_cache(3, [64 + 100, 64 + 200, 64 + 30], 4, 2, 64, 32, dtype, seed=71, prefix=64)
    cache.seq_lens.copy_(torch.tensor([70, 64, 65], dtype=torch.int32))
    ws = b.dilution_attn_paged_decode_workspace(cache, max_len)
    out = torch.empty_like(q)
    old = cache.demand_pages.clone()
    b.dilution_attn_paged_decode(q, cache, max_len, out, prefix_table=pt, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.dilution_attn_paged_decode(q, cache, max_len, out, prefix_table=pt, workspace=ws)
    cache.demand_pages.copy_(old)
    for lens in ([70, 64, 65], [100, 0, 94], [164, 264, 94]):
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        before = cache.demand_pages.clone()
        ref = oracle_step(cache, q, prefix_table=pt)
        g.replay()
        assert b.dilution_attn_get_error(ws) == b.DA_OK
        check_step(cache, q, before, out, ref)


@pytest.mark.parametrize("max_len", [900, LONG])
def test_two_streams_with_their_own_workspaces(max_len):
    made = [make_cache(4, [900, 1, 333, 64], 4, 4, 64, 32, "bf16", seed=80 + i) for i in range(2)]
    refs = [oracle_step(c, q) for c, q, _ in made]
    before = [c.demand_pages.clone() for c, _, _ in made]
    wss = [b.dilution_attn_paged_decode_workspace(c, max_len) for c, _, _ in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _, q, _ in made]
    for (c, q, _), ws, st, out in zip(made, wss, streams, outs):
        b.dilution_attn_paged_decode(q, c, max_len, out, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for (c, q, _), o, r, old in zip(made, outs, refs, before):
        check_step(c, q, old, o, r)


@pytest.mark.parametrize("max_len", [300, LONG])
def test_call_on_another_stream_without_buffers(max_len):
    # out and workspace are the call's own: allocated and zeroed on its stream, not the busy current one
    cache, q, _ = make_cache(3, [300, 7, 130], 4, 2, 64, 32, "bf16", seed=66)
    ref = oracle_step(cache, q)
    before = cache.demand_pages.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.zeros(1 << 28, device=DEV)
    for _ in range(20):
        busy.add_(1.0)                                   # the current stream is behind
    out = b.dilution_attn_paged_decode(q, cache, max_len, stream=side)
    junk = [torch.full((1 << 20,), 7.0, device=DEV) for _ in range(8)]   # memory handed out meanwhile
    side.synchronize()
    check_step(cache, q, before, out, ref)
    torch.cuda.synchronize()
    assert len(junk) == 8


def test_error_of_a_call_beside_a_busy_stream():
    # a cache made while the current stream is behind: its status block is zero for a call on another stream already
    made, q, _ = make_cache(3, [300, 7, 130], 4, 2, 64, 32, "bf16", seed=66)
    tensors = [getattr(made, n) for n in ("k_pages", "v_pages", "demand_pages", "page_table", "demand_table", "seq_lens")]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.dilution_attn_paged_decode(q, made, 300, stream=side)   # memory for the call below: no allocation stops the device
    made.page_table[0, 1] = 10 ** 6
    junk = [torch.full((256,), 0x55, dtype=torch.uint8, device=DEV) for _ in range(64)]
    busy = torch.zeros(1 << 28, device=DEV)
    torch.cuda.synchronize()
    del junk                                             # what the next small block may hold
    for _ in range(50):
        busy.add_(1.0)
    cache = b.PagedCache(*tensors)
    b.dilution_attn_paged_decode(q, cache, 300, stream=side)
    side.synchronize()
    assert b.dilution_attn_get_error(cache.status, side) == b.DA_ERR_INVALID
    torch.cuda.synchronize()
    assert b.dilution_attn_get_error(cache.status) == b.DA_OK


def test_error_of_a_call_whose_cache_is_gone():
    # the call still runs when its cache is dropped: its error does not land in a later cache's status block
    made, q, _ = make_cache(3, [300, 7, 130], 4, 2, 64, 32, "bf16", seed=66)
    tensors = [getattr(made, n) for n in ("k_pages", "v_pages", "demand_pages", "page_table", "demand_table", "seq_lens")]
    k, cu = torch.zeros(3, 2, 64, dtype=q.dtype, device=DEV), torch.arange(4, dtype=torch.int32, device=DEV)
    made.page_table[0, :] = 10 ** 6
    busy = torch.zeros(1 << 28, device=DEV)
    warm = [b.PagedCache(*tensors) for _ in range(64)]            # memory for what follows: no allocation stops the device
    b.dilution_attn_paged_decode(q, made, 300)
    torch.cuda.synchronize()
    del warm
    for call in ("append", "decode"):
        for _ in range(50):
            busy.add_(1.0)
        cache = b.PagedCache(*tensors)
        if call == "append":
            b.dilution_attn_paged_append(None, k, k, cache, cu)
        else:
            b.dilution_attn_paged_decode(q, cache, 300)
        del cache
        later = [b.PagedCache(*tensors) for _ in range(64)]       # the streams of the blocks repeat after 32
        torch.cuda.synchronize()
        assert not any(c.status.any() for c in later)
    # a graph outlives the cache object whose tensors it reads
    cache = b.PagedCache(*tensors)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.dilution_attn_paged_append(None, k, k, cache, cu)
        b.dilution_attn_paged_decode(q, cache, 300)
    del cache, later
    later = [b.PagedCache(*tensors) for _ in range(64)]
    graph.replay()
    torch.cuda.synchronize()
    assert not any(c.status.any() for c in later)


def test_pool_past_32_bit_offsets():
    # pools of more than 2^32 bytes and 2^31 elements: the sequence's pages lie at the end
    page, d, Hkv = 256, 128, 4
    n = (1 << 31) // (Hkv * page * d) + 40
    k = torch.empty(n, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    lens = [700, 300]
    ids = torch.tensor([[n - 1, n - 5, n - 3], [n - 9, n - 7, -1]], dtype=torch.int32)
    g = torch.Generator(device=DEV).manual_seed(5)
    for i in ids.flatten().tolist():
        if i >= 0:
            k[i] = torch.randn(Hkv, page, d, generator=g, device=DEV)
            v[i] = torch.randn(Hkv, page, d, generator=g, device=DEV)
    small = {int(i): j for j, i in enumerate(x for x in ids.flatten().tolist() if x >= 0)}
    order = list(small)
    dem = torch.rand(6, Hkv, page, generator=g, device=DEV)
    dt = torch.tensor([[0, 1, 2], [3, 4, -1]], dtype=torch.int32, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cache = b.PagedCache(k, v, dem, ids.to(DEV), dt, sl)
    local = torch.tensor([[small.get(int(i), -1) for i in row] for row in ids], dtype=torch.int32, device=DEV)
    mirror = b.PagedCache(k[order].contiguous(), v[order].contiguous(), dem.clone(), local, dt, sl)
    q = torch.randn(2, Hkv, d, generator=g, device=DEV).bfloat16()
    for cap in (700, 768):                                # 1024 keys and more: the kernels for long caches, below
        ref = oracle_step(mirror, q)
        before = cache.demand_pages.clone()
        out = b.dilution_attn_paged_decode(q, cache, cap)
        check_step(cache, q, before, out, ref)
        mirror.demand_pages.copy_(cache.demand_pages)
    wide = torch.cat([ids.to(DEV), torch.full((2, 20), -1, dtype=torch.int32, device=DEV)], 1)
    wdt = torch.cat([dt, torch.full((2, 20), -1, dtype=torch.int32, device=DEV)], 1)
    long = b.PagedCache(k, v, cache.demand_pages, wide, wdt, sl)
    ref = oracle_step(mirror, q)
    before = long.demand_pages.clone()
    out = b.dilution_attn_paged_decode(q, long, LONG)
    check_step(long, q, before, out, ref)


# ------------------------------------------------------------------ waits that run out
def run_out(cache, q, pt, max_len, kernel, block):
    """A step in which one block's hand-over is kept: the waits of its kernel give up, the call completes and says so,
    and the next step gives the bits of the step before."""
    ws = b.dilution_attn_paged_decode_workspace(cache, max_len)
    before = cache.demand_pages.clone()
    good = b.dilution_attn_paged_decode(q, cache, max_len, prefix_table=pt, workspace=ws)
    demand = cache.demand_pages.clone()
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    cache.demand_pages.copy_(before)
    st, _ = b.dilution_attn_debug_paged_decode_stall(q, cache, max_len, workspace=ws, prefix_table=pt, stall_kernel=kernel,
                                                     stall_block=block)
    assert st == b.DA_OK                                      # launched; the failure is on the device
    words = b.dilution_attn_debug_last_timeout(ws)            # synchronises: the call completed
    assert words[0] == b.DA_ERR_TIMEOUT and words[2] == block and words[1] > 0
    assert b.dilution_attn_get_error(ws) == b.DA_ERR_TIMEOUT
    ws[:256].zero_()
    cache.demand_pages.copy_(before)
    again = b.dilution_attn_paged_decode(q, cache, max_len, prefix_table=pt, workspace=ws)
    assert b.dilution_attn_get_error(ws) == b.DA_OK
    assert torch.equal(again, good) and torch.equal(cache.demand_pages, demand)
    return words[3]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kernel", [0, 1])                    # logits, shares
@pytest.mark.parametrize("G,d", [(1, 64), (3, 128), (16, 64)])
def test_streaming_waits_that_run_out_are_reported_and_recovered(G, d, kernel, dtype):
    # 2 x 4 key heads x 60000 keys: more than 8 tiles for each of 304 blocks
    cache, q, _ = make_cache(2, [60000, 59000], 4 * G, 4, d, 64, dtype, seed=7)
    thread = run_out(cache, q, None, 60000, kernel, 17)
    assert 0 <= thread < 288


@pytest.mark.parametrize("kernel", [2, 3])
@pytest.mark.parametrize("d,S", [(64, 17), (128, 40)])
def test_prefix_waits_that_run_out_are_reported_and_recovered(d, S, kernel):
    # one key head, one segment: 3856 tiles, 12 or 13 for a block of the first pass, 25 of the second
    prefix = 493568
    cache, q, pt = make_cache(S, [prefix + 1 + i for i in range(S)], 1, 1, d, 256, "bf16", seed=8, prefix=prefix)
    thread = run_out(cache, q, pt, prefix + S, kernel, 17)
    assert 0 <= thread < 640
