"""Eviction on the GPU: which keys stay (ties, NaN, zeros, lengths and budgets
around every edge, long streams) and their rows moving together, exactly as the
plain forms say; a run of select, compact and trim; graphs and refusals."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import long_cache_plain as plain

BF16 = torch.bfloat16
i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()


def run_select(w, lens, sinks, recent, budget, **kw):
    kept = torch.full((len(lens), budget), 12345, dtype=torch.int32, device="cuda")
    keep = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    mva.evict_select(w, i32(lens), sinks, recent, kept, keep, **kw)
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    return kept, keep


def check_select(w, lens, sinks, recent, budget):
    kept, keep = run_select(w.cuda(), lens, sinks, recent, budget)
    for b, S in enumerate(lens):
        want = plain.select(w[b], S, sinks, recent, budget)
        assert int(keep[b]) == len(want) == min(S, budget)
        got = kept[b].tolist()
        assert got == want + [-1] * (budget - len(want)), "stream %d" % b


def mass(gen, *shape):
    return torch.exp(4 * torch.randn(shape, generator=gen))


@pytest.mark.parametrize("Hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("lens,sinks,recent,budget", [
    ([1], 0, 0, 1),
    ([2], 0, 0, 1),
    ([0, 1, 5, 6, 7, 100], 2, 3, 6),
    ([1000, 999, 1001], 4, 64, 1000),             # one key too many
    ([3000, 100, 2047, 2048, 2049], 4, 100, 500),
    ([4096, 4095], 0, 0, 1),
    ([4096, 300], 100, 28, 128),                  # nothing to choose
    ([5000, 4097, 0, 37, 20000], 4, 512, 2048),   # a cluster a stream
    ([65536, 7], 0, 1, 16384),
])
def test_select(lens, sinks, recent, budget, Hkv):
    gen = torch.Generator().manual_seed(budget)
    w = mass(gen, len(lens), Hkv, max(max(lens), 1))
    for b, n in enumerate(lens):
        w[b, :, n:] = float("nan")                # not looked at
    check_select(w, lens, sinks, recent, budget)


@pytest.mark.parametrize("S", [700, 9000])
def test_ties_go_to_the_first(S):
    gen = torch.Generator().manual_seed(S)
    for levels in (1, 2, 5):
        w = torch.randint(0, levels, (2, 2, S), generator=gen).float()
        for budget in (10, S // 2, S - 1):
            check_select(w, [S, S - 3], 3, 5, budget)


@pytest.mark.parametrize("S", [500, 6000])
def test_odd_weights(S):
    gen = torch.Generator().manual_seed(S)
    w = mass(gen, 1, 1, S)
    at = torch.randperm(S, generator=gen)
    w[0, 0, at[:20]] = float("nan")
    w[0, 0, at[20:40]] = float("inf")
    w[0, 0, at[40:60]] = 0.0
    w[0, 0, at[60:80]] = -0.0
    w[0, 0, at[80:100]] = -torch.rand(20, generator=gen)
    w[0, 0, at[100:120]] = 1e-42                  # below fp32's normal range
    w[0, 0, at[120:130]] = -float("inf")
    for budget in (10, 30, 50, S - 125, S - 95, S - 60, S - 45, S - 5):
        check_select(w, [S], 0, 0, budget)


def test_weights_that_differ_in_their_last_bits():
    base = torch.tensor(1.0).view(torch.int32) + torch.randperm(8192, generator=torch.Generator().manual_seed(0)).int()
    w = base.view(torch.float32).view(1, 1, -1).clone()
    for budget in (1, 1000, 4095, 8191):
        check_select(w, [8192], 0, 0, budget)


def test_many_streams_and_streams_beyond_shared_memory():
    gen = torch.Generator().manual_seed(9)
    lens = [int(x) for x in torch.randint(0, 700, (300,), generator=gen)]
    check_select(mass(gen, 300, 2, 700), lens, 2, 10, 100)
    S = 8 * 49152 + 5
    assert mva.evict_workspace_size(2, S) == 8 * S and mva.evict_workspace_size(2, S - 5) == 0
    w = torch.rand((2, 1, S), generator=gen)
    check_select(w, [S, 40], 4, 1000, 3000)
    check_select(w[:, :, :S - 5].contiguous(), [S - 5, 30000], 0, 0, 20000)


def streams(gen, lens, page, shape, dt=BF16):
    table, total = plain.pages(gen, lens, page)
    pools = [torch.randint(0, 256, (total * page, *shape), dtype=torch.uint8, device="cuda") if dt is torch.uint8
             else torch.randn((total * page, *shape), device="cuda").to(dt) for _ in range(2)]
    return table, pools


def compacted(pool, table, page, lens, kept, keep):
    out = pool.cpu().clone()
    for b, n in enumerate(keep):
        rows = plain.rows_of(table[b], page, lens[b])
        out[rows[:n]] = pool.cpu()[rows[kept[b][:n]]]
    return out


def check_compact(gen, lens, budget, page, shape, dt=BF16, Hkv=2, call=None):
    table, pools = streams(gen, lens, page, shape, dt)
    smax = table.shape[1] * page
    keep = [min(n, budget) for n in lens]
    kept = [torch.randperm(n, generator=gen)[:k].sort().values for n, k in zip(lens, keep)]
    kept_t = torch.full((len(lens), budget), -1, dtype=torch.int32)
    for b, k in enumerate(kept):
        kept_t[b, :len(k)] = k
    w = torch.rand((len(lens), Hkv, smax), generator=gen).cuda()
    want = [compacted(p, table, page, lens, kept, keep) for p in pools]
    want_w = w.cpu().clone()
    for b, k in enumerate(kept):
        want_w[b, :, :lens[b]] = 0
        want_w[b, :, :len(k)] = w[b].cpu()[:, k]
    args = (table.cuda(), page, i32(lens), kept_t.cuda(), i32(keep))
    if call is None:
        mva.gqa_cache_compact(*pools, *args, weights=w)
    else:
        call(pools, args, w)
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    for b, n in enumerate(lens):                   # rows behind the kept ones hold nothing in particular
        rows = plain.rows_of(table[b], page, n)[keep[b]:]
        for p, x in zip(pools, want):
            x[rows] = p.cpu()[rows]
    assert all(torch.equal(p.cpu(), x) for p, x in zip(pools, want))
    assert torch.equal(w.cpu(), want_w)


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("lens,budget", [
    ([1], 1), ([2], 1), ([0, 3, 10], 3), ([100, 50, 60], 50),
    ([4000, 0, 2049, 2100], 2048), ([9000], 8999), ([6000, 6000], 17),
])
def test_compact(lens, budget, page):
    gen = torch.Generator().manual_seed(page + budget)
    check_compact(gen, lens, budget, page, (2, 64))


@pytest.mark.parametrize("shape,dt", [((1, 64), torch.float16), ((8, 128), BF16), ((5, 64), BF16), ((112,), torch.uint8),
                                      ((576,), torch.uint8), ((16,), torch.uint8)])
def test_compact_rows_of_all_kinds(shape, dt):
    gen = torch.Generator().manual_seed(shape[0])
    check_compact(gen, [3000, 700], 600, 16, shape, dt, Hkv=3)
    check_compact(gen, [300] * 40, 70, 16, shape, dt, Hkv=1)       # (slices of 64 bytes)


def test_compact_many_streams():
    gen = torch.Generator().manual_seed(4)
    lens = [int(x) for x in torch.randint(0, 200, (500,), generator=gen)]
    check_compact(gen, lens, 60, 16, (2, 128))


def test_compact_of_the_latent_cache():
    gen = torch.Generator().manual_seed(6)
    def call(pools, args, w):
        mva.cache_compact(pools[0], *args, weights=w)
        mva.cache_compact(pools[1], *args)
    check_compact(gen, [700, 64, 3000], 512, 64, (576,), call=call)


def test_bad_entries_are_reported_and_touch_nothing():
    gen = torch.Generator().manual_seed(1)
    table, pools = streams(gen, [50, 60], 16, (2, 64))
    before = [p.clone() for p in pools]
    call = lambda t=table, lens=(50, 60), kept=((0, 2, 3), (0, 1, 2)), keep=(3, 3): mva.gqa_cache_compact(
        *pools, t.cuda(), 16, i32(lens), i32(kept), i32(keep))
    for kw, want in ((dict(lens=(70, 60), keep=(3, 0)), -8), (dict(lens=(-1, 60), keep=(0, 0)), -8), (dict(keep=(4, 0)), -12),
                     (dict(keep=(-1, 0)), -12), (dict(kept=((0, 50, 1 << 30), (0, 0, 1))), -12),
                     (dict(lens=(2, 60), kept=((0, 1, 2), (0, 1, 2)), keep=(3, 3)), -12)):
        call(**kw)
        assert mva.last_device_error() == want, kw
    t = table.clone()
    t[0, 0] = 1 << 20
    call(t=t)
    assert mva.last_device_error() == -10
    assert all(torch.equal(p, x) for p, x in zip(pools, before))
    kept, keep = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), i32([5, 5])
    mva.evict_select(torch.ones((2, 1, 64), device="cuda"), i32([65, -2]), 0, 0, kept, keep)
    assert mva.last_device_error() == -8
    assert keep.tolist() == [0, 0] and (kept == -1).all()


def test_select_compact_trim_in_a_graph():
    # As a serving loop runs them: pages go back, and what is left is what was chosen.
    gen = torch.Generator().manual_seed(3)
    page, budget = 16, 256
    lens = [700, 100, 256, 1000]
    table, pools = streams(gen, lens, page, (2, 64))
    w = mass(gen, 4, 2, table.shape[1] * page).cuda()
    free = torch.full((200,), -1, dtype=torch.int32, device="cuda")
    count, lens_t, table_t = i32([0]), i32(lens), table.clamp_min(0).cuda()
    kept, keep = torch.empty((4, budget), dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")

    def step():
        mva.evict_select(w, lens_t, 4, 32, kept, keep)
        mva.gqa_cache_compact(*pools, table_t, page, lens_t, kept, keep, weights=w)
        mva.blocks_trim(lens_t, keep, table_t, page, free, count)

    state = [x.clone() for x in (*pools, w, lens_t, table_t, free, count)]
    step()
    torch.cuda.synchronize()
    after = [x.clone() for x in (*pools, w, lens_t, table_t, free, count)]
    want = [plain.select(state[2][b].cpu(), n, 4, 32, budget) for b, n in enumerate(lens)]
    for b, n in enumerate(lens):
        rows = plain.rows_of(table[b], page, n)
        assert kept[b].tolist()[:len(want[b])] == want[b]
        assert torch.equal(pools[0].cpu()[rows[:len(want[b])]], state[0].cpu()[rows[want[b]]])
        assert torch.equal(w[b].cpu()[:, :len(want[b])], state[2][b].cpu()[:, want[b]])
    assert lens_t.tolist() == [min(n, budget) for n in lens]
    assert int(count) == sum(-(-n // page) + -min(n, budget) // page for n in lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for x, y in zip((*pools, w, lens_t, table_t, free, count), state):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*pools, w, lens_t, table_t, free, count), after))
    assert mva.last_device_error() == 0


def test_refusals():
    w, lens = torch.ones((2, 2, 100), device="cuda"), i32([50, 60])
    kept, keep = torch.zeros((2, 10), dtype=torch.int32, device="cuda"), i32([0, 0])
    for sinks, recent in ((-1, 0), (0, -1), (6, 5), (1 << 30, 1 << 30)):
        with pytest.raises(mva.MLAError) as e:
            mva.evict_select(w, lens, sinks, recent, kept, keep)
        assert e.value.status == -2
    for args in ((w.double(), lens, 1, 1, kept, keep), (w[:, :, ::2], lens, 1, 1, kept, keep), (w, lens[:1], 1, 1, kept, keep),
                 (w, lens, 1, 1, kept.long(), keep), (w, lens, 1, 1, kept, keep[:1])):
        with pytest.raises(ValueError):
            mva.evict_select(*args)
    big = torch.ones((1, 1, 8 * 49152 + 1), device="cuda")
    with pytest.raises(mva.MLAError) as e:
        mva.evict_select(big, lens[:1], 0, 0, kept[:1], keep[:1], workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4
    table, pools = streams(torch.Generator().manual_seed(0), [50, 60], 16, (2, 64))
    good = (*pools, table.cuda(), 16, lens, kept, keep)
    for i, bad in ((1, pools[1][:, :1]), (2, table.cuda().long()), (4, lens.long()), (5, kept[:1]), (6, keep[:1])):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            mva.gqa_cache_compact(*args)
    with pytest.raises(ValueError):
        mva.gqa_cache_compact(*good, weights=w)


def test_compact_in_pools_beyond_2_to_the_32_bytes():
    page, rows = 64, 2_300_000
    pools = [torch.zeros((rows // page * page, 8, 128), dtype=BF16, device="cuda") for _ in range(2)]
    lens, budget = [3000], 700
    table = torch.tensor([[rows // page - 1 - j if j % 2 else j for j in range(47)]], dtype=torch.int32)
    at = plain.rows_of(table[0], page, 3000).cuda()
    for p in pools:
        p[at] = torch.randn((3000, 8, 128), device="cuda").to(BF16)
    kept = torch.randperm(3000, generator=torch.Generator().manual_seed(0))[:budget].sort().values
    want = [p[at[kept.cuda()]].clone() for p in pools]
    mva.gqa_cache_compact(*pools, table.cuda(), page, i32(lens), kept.int()[None].cuda(), i32([budget]))
    assert mva.last_device_error() == 0
    assert all(torch.equal(p[at[:budget]], w) for p, w in zip(pools, want))


def test_compact_and_select_of_more_streams_than_a_grid_is_high():
    B, page = 66000, 2
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    pool = torch.arange(4 * B, dtype=torch.int64, device="cuda")[:, None].repeat(1, 2).view(torch.uint8)
    lens = torch.full((B,), 4, dtype=torch.int32, device="cuda")
    w = torch.rand((B, 1, 4), device="cuda")
    kept, keep = torch.empty((B, 3), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    mva.evict_select(w, lens, 0, 0, kept, keep)
    want = w[:, 0].argsort(dim=1, descending=True)[:, :3].sort(dim=1).values
    assert torch.equal(kept.long(), want) and (keep == 3).all()
    second = pool.clone()
    mva.gqa_cache_compact(pool, second, table, page, lens, kept, keep)
    assert mva.last_device_error() == 0
    rows = (torch.arange(B, device="cuda")[:, None] * 4 + want)
    for p in (pool, second):
        assert torch.equal(p.view(torch.int64)[:, 0].view(B, 4)[:, :3], rows)


def streams_for(blocks):
    """How many streams of more than 4,096 keys make select take this many blocks a stream (as many as the device
    holds at once, two an SM, up to eight)."""
    most = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    return {8: 3, 4: most // 8 + 1, 2: most // 4 + 1, 1: most // 2 + 1}[blocks]


@pytest.mark.parametrize("blocks", [8, 4, 2, 1])
@pytest.mark.parametrize("sinks,recent,budget", [
    (0, 0, 700),
    (4, 512, 3000),
    (1200, 800, 2000),                            # nothing to choose: all of it first and last keys
    (0, 2000, 2000),
    (2500, 3100, 5700),                           # whole blocks hold first or last keys only
    (5900, 0, 5901),
    (0, 5900, 5999),
])
def test_select_with_every_number_of_blocks(blocks, sinks, recent, budget):
    gen = torch.Generator().manual_seed(blocks + budget)
    B, S = streams_for(blocks), 6000
    lens = [S, S - 1, budget, budget + 1, 0, 4097] + [37] * B
    lens = lens[:B] if B > 6 else lens[:2] + [budget + 1]
    check_select(mass(gen, B, 2, S), lens, sinks, recent, budget)
    check_select(torch.randint(0, 3, (B, 1, S), generator=gen).float(), lens, sinks, recent, budget)
    check_select(torch.ones((B, 1, S)), lens, sinks, recent, budget)


@pytest.mark.parametrize("blocks", [4, 2, 1])
def test_select_with_long_runs_of_a_block(blocks):
    gen = torch.Generator().manual_seed(blocks)
    B, S = streams_for(blocks), 49000
    check_select(mass(gen, B, 1, S), [S, 5, 30001, 0] + [100] * (B - 4), 4, 1000, 9000)


def test_select_and_compact_on_another_stream_and_in_a_graph_of_it():
    gen = torch.Generator().manual_seed(8)
    page, budget, lens = 16, 2500, [6000, 100, 5000]
    table, pools = streams(gen, lens, page, (2, 64))
    table, smax = table.clamp_min(0).cuda(), table.shape[1] * page
    w, lens_t = mass(gen, 3, 2, smax).cuda(), i32(lens)
    state = [x.clone() for x in (*pools, w)]
    kept, keep = torch.empty((3, budget), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def both(stream):
        mva.evict_select(w, lens_t, 4, 64, kept, keep, stream=stream)
        mva.gqa_cache_compact(*pools, table, page, lens_t, kept, keep, weights=w, stream=stream)

    def check():
        torch.cuda.synchronize()
        assert mva.last_device_error() == 0
        for b, n in enumerate(lens):
            want = plain.select(state[2][b].cpu(), n, 4, 64, budget)
            assert int(keep[b]) == len(want) and kept[b, :len(want)].tolist() == want and (kept[b, len(want):] == -1).all()
            rows = plain.rows_of(table[b], page, n)
            for p, old in zip(pools, state):
                assert torch.equal(p.cpu()[rows[:len(want)]], old.cpu()[rows[want]])
            assert torch.equal(w[b, :, :len(want)].cpu(), state[2][b].cpu()[:, want]) and not w[b, :, len(want):n].any()

    torch.cuda.synchronize()
    both(side)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both(side)
    for x, y in zip((*pools, w), state):
        x.copy_(y)
    kept.fill_(-9)
    graph.replay()
    check()
