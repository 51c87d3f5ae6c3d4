"""Grouped-head verify attention on the GPU against its plain 64-bit form:
types, head layouts, lengths around tile edges, masks that leave nothing,
strided caches, pages of every kind, streams, graphs and refusals."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import gqa_plain as plain

BF16, FP16 = torch.bfloat16, torch.float16


def trees(gen, B, q, kind):
    if kind == "chain":
        return torch.ones(q, q).tril().bool().expand(B, q, q).clone()
    if kind == "any":          # any pattern, rows that see nothing among them
        return torch.rand((B, q, q), generator=gen) < 0.4
    seen = torch.zeros((B, q, q), dtype=torch.bool)
    for b in range(B):
        for i in range(q):
            if i:
                seen[b, i] = seen[b, int(torch.randint(0, i, (1,), generator=gen))]
            seen[b, i, i] = True
    return seen


def normal(gen, shape, dt):
    return torch.randn(shape, generator=gen).to(dt).cuda()


def case(B, q, H, Hkv, D, lens, dt, smax=None, tree="random", seed=0):
    gen = torch.Generator().manual_seed(seed + 17 * q + D)
    smax = smax or max(max(lens), 1)
    c = dict(q=normal(gen, (B, q, H, D), dt), k=normal(gen, (B, smax, Hkv, D), dt), v=normal(gen, (B, smax, Hkv, D), dt),
             lens=lens, seen=trees(gen, B, q, tree), scale=1 / math.sqrt(D), gen=gen)
    for b, n in enumerate(lens):           # rows past a stream's end hold anything
        c["k"][b, n:] = float("nan")
        c["v"][b, n:] = float("nan")
    c["lens_t"] = torch.tensor(lens, dtype=torch.int32).cuda()
    c["mask"] = plain.mask_words(c["seen"]).cuda()
    return c


def run(c, **kw):
    out, lse = mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"], **kw)
    torch.cuda.synchronize()
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    return out, lse


def verify(c, out, lse):
    plain.check(out, lse, c["q"], lambda b: c["k"][b], lambda b: c["v"][b], c["lens"], c["seen"], c["scale"])


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,q,H,Hkv,lens", [
    (1, 1, 1, 1, [1]),                         # one head, one key
    (1, 1, 8, 1, [64]),                        # exactly one tile
    (1, 9, 64, 8, [265]),
    (2, 5, 6, 2, [63, 130]),                   # three heads a key head, ragged
    (3, 16, 8, 1, [16, 0, 700]),               # no prefix; an unused stream; 128 rows exactly
    (1, 33, 16, 4, [2000]),                    # 132 rows: two row tiles, two mask words
    (2, 64, 7, 1, [100, 1000]),                # 448 rows: two row groups, the second one full
    (2, 37, 28, 4, [37, 515]),                 # 259 rows: a second group of three rows
    (5, 2, 4, 4, [2, 65, 128, 129, 191]),      # a key head per head, lengths around tile edges
])
def test_matches_plain(B, q, H, Hkv, lens, D, dt):
    c = case(B, q, H, Hkv, D, lens, dt)
    verify(c, *run(c))


@pytest.mark.parametrize("B,q,H,Hkv,D,lens,dt", [
    (1, 9, 40, 5, 64, [700], BF16),             # heads that no team divides evenly
    (2, 3, 21, 3, 128, [600, 1290], FP16),      # seven heads a key head, three key heads
    (1, 64, 40, 1, 64, [900], BF16),            # 2,560 rows: twenty row groups, two sets of them
    (1, 64, 64, 2, 128, [1000], FP16),          # sixteen row groups
    (3, 33, 24, 8, 64, [33, 2100, 800], BF16),  # heads side by side, 99 rows
    (1, 1, 128, 128, 128, [1500], BF16),        # a key head a head, many of them
    (60, 2, 16, 2, 128, list(range(2, 1202, 20)), BF16),   # many units, cut and whole
])
def test_heads_and_row_groups(B, q, H, Hkv, D, lens, dt):
    c = case(B, q, H, Hkv, D, lens, dt)
    verify(c, *run(c))


@pytest.mark.parametrize("G,Hkv,D,lens,smax,dt", [
    (34, 1, 128, [900], 900, BF16),                        # 17 row groups: nine and eight
    (38, 2, 64, [64, 2500, 700], 2500, FP16),              # 19 groups of two key heads
    (34, 2, 128, [1300, 80, 3000, 0, 511], 3000, BF16),    # more units than CTAs
    (68, 1, 64, [640, 5000], 5000, BF16),                  # 34 groups: three sets of twelve, two missing
    (70, 3, 64, [900, 64, 1700], 1700, FP16),              # 35 groups, three key heads
    (34, 2, 64, [300, 512, 64, 100], 512, BF16),           # units that are not cut
])
def test_row_groups_that_a_set_lacks(G, Hkv, D, lens, smax, dt):
    # Row groups that sets of CTAs do not divide evenly: in the last set some have none.
    c = case(len(lens), 64, G * Hkv, Hkv, D, lens, dt, smax=smax)
    a = run(c)
    verify(c, *a)
    b = run(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("smax", [448, 512, 513, 600])
def test_short_caches_whole_and_cut(smax):
    # Up to 512 keys units are not cut, and there is no merge.
    for lens in ([smax, 9, 0], [70, smax - 1, 64]):
        c = case(3, 9, 16, 4, 128, lens, BF16, smax=smax)
        verify(c, *run(c))


def test_many_segments_of_one_tile():
    # Single tiles one after the other: each is a segment of its own, with one
    # softmax group idle; masked rows among them.
    gen = torch.Generator().manual_seed(8)
    lens = [int(x) for x in torch.randint(5, 70, (700,), generator=gen)]
    for tree in ("random", "any"):
        c = case(700, 5, 8, 1, 128, lens, BF16, smax=70, tree=tree)
        a = run(c)
        verify(c, *a)
        for _ in range(3):
            b = run(c)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D,page", [(64, 0), (128, 0), (128, 16), (64, 5)])
def test_products_see_what_both_their_barriers_guard(D, page):
    # Tiles, weights and results pass between warps all the time: the same bits every time.
    gen = torch.Generator().manual_seed(D + page)
    lens = [int(x) for x in torch.randint(5, 400, (300,), generator=gen)] + [9000]
    c = case(301, 5, 16, 2, D, lens, BF16)
    call = run if not page else lambda c, p=paged(c, page): run_paged(c, page, *p)
    a = call(c)
    verify(c, *a)
    for _ in range(50):
        b = call(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("tree", ["chain", "any"])
@pytest.mark.parametrize("q,G,n", [(9, 8, 9), (9, 8, 70), (40, 2, 41), (64, 4, 64), (64, 4, 129)])
def test_masks(q, G, n, tree):
    c = case(2, q, 2 * G, 2, 128, [n, q], BF16, tree=tree)
    verify(c, *run(c))


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q,used,n,page", [
    (9, 5, 300, 0),            # the padding drafts end inside a tile
    (9, 0, 9, 0),              # nothing but padding
    (64, 33, 160, 0),          # drafts over two tiles, two mask words
    (40, 12, 104, 16),         # pages that end inside a tile
    (40, 20, 1000, 5),         # gathered rows, in several parts
    (33, 32, 128, 0),          # one padding draft, the last key of a whole tile
])
def test_drafts_that_none_sees_hold_anything(q, used, n, page, what):
    # A batch padded to one q_len: the drafts behind `used` see the prefix alone, and none sees them.
    for D, dt in ((64, BF16), (128, FP16)):
        c = case(2, q, 16, 2, D, [n, n + 64], dt)
        c["seen"][0, used:] = False
        c["seen"][0, :, used:] = False
        c["mask"] = plain.mask_words(c["seen"]).cuda()
        junk = {}
        for name in "kv":
            junk[name] = c[name].clone()
            junk[name][0, n - q + used:n] = what
        if page:
            rows = -(-(n + 64) // page) * page
            pools = []
            for name in "kv":
                pool = torch.zeros((2, rows, 2, D), dtype=dt, device="cuda")
                pool[:, :n + 64] = junk[name]
                pools.append(pool.view(2 * rows, 2, D))
            table = torch.arange(2 * rows // page, dtype=torch.int32, device="cuda").view(2, -1)
            out, lse = mva.gqa_verify_attn_paged(c["q"], *pools, table, page, c["lens_t"], c["mask"], c["scale"])
        else:
            out, lse = mva.gqa_verify_attn(c["q"], junk["k"], junk["v"], c["lens_t"], c["mask"], c["scale"])
        assert mva.last_device_error() == 0
        verify(c, out, lse)


@pytest.mark.parametrize("n,smax", [(100, 128), (400, 600), (5000, 5000)])    # whole units, and cut ones
def test_nan_of_a_row_stays_in_it(n, smax):
    c = case(1, 5, 8, 2, 128, [n], BF16, smax=smax)
    c["q"][0, 2, 3, 7] = float("nan")
    c["k"][0, n - 1] = float("nan")                # a key that the last draft alone sees
    c["seen"][0, :4, 4] = False
    c["seen"][0, 4, 4] = True
    c["mask"] = plain.mask_words(c["seen"]).cuda()
    out, lse = run(c)
    bad = torch.zeros((5, 8), dtype=torch.bool, device="cuda")
    bad[2, 3] = bad[4] = True
    assert torch.equal(torch.isnan(lse[0]), bad)
    assert torch.equal(torch.isnan(out[0]).all(-1), bad) and torch.equal(torch.isnan(out[0]).any(-1), bad)


def test_rows_that_see_nothing():
    c = case(1, 9, 8, 1, 64, [9], FP16)
    c["seen"][0, 3] = False
    c["seen"][0, 8] = False
    c["mask"] = plain.mask_words(c["seen"]).cuda()
    out, lse = run(c)
    verify(c, out, lse)
    assert (out[0, [3, 8]] == 0).all() and torch.isneginf(lse[0, [3, 8]]).all()


def test_mask_bits_past_the_drafts_are_ignored():
    c = case(1, 9, 8, 1, 64, [100], BF16)
    a = run(c)
    c["mask"] = c["mask"] | torch.tensor(-512, dtype=torch.int32, device="cuda")    # bits 9..31
    b = run(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("scale", [0.0, -0.09, 0.5])
def test_scales(scale):
    c = case(1, 9, 8, 2, 64, [300], BF16)
    c["scale"] = scale
    verify(c, *run(c))


def test_scores_that_grow_along_the_keys():
    # The running max moves in nearly every tile: O is rescaled again and again.
    c = case(1, 9, 8, 1, 128, [1500], BF16)
    ramp = torch.linspace(0.1, 6, 1500, device="cuda").to(BF16)
    c["k"][0] = c["q"][0, 0, 0] * ramp[:, None, None]
    verify(c, *run(c))


def test_long_and_many_streams():
    c = case(1, 9, 16, 2, 128, [40003], BF16)
    verify(c, *run(c))
    gen = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(0, 300, (900,), generator=gen)]
    lens = [0 if n < 3 else n for n in lens]
    c = case(900, 3, 4, 2, 64, lens, FP16)
    verify(c, *run(c))


def test_more_streams_than_threads_are_found():
    # Most streams unused, the used ones far apart.
    lens = [0] * 5000
    lens[7], lens[2500], lens[4999] = 70, 500, 1
    c = case(5000, 1, 2, 1, 64, lens, BF16, smax=500)
    out, lse = run(c)
    for b in (7, 2500, 4999, 0, 4998):
        plain.check(out[b:b + 1], lse[b:b + 1], c["q"][b:b + 1], lambda _: c["k"][b], lambda _: c["v"][b],
                    [lens[b]], c["seen"][b:b + 1], c["scale"])
    assert (out[8:2500] == 0).all() and torch.isneginf(lse[8:2500]).all()


def test_strided_views():
    B, q, H, Hkv, D, n = 2, 5, 8, 2, 64, 200
    gen = torch.Generator().manual_seed(5)
    qkv = normal(gen, (B, q, H + 2 * Hkv, D), BF16)               # queries out of a fused projection
    kv = normal(gen, (B, n, 2, Hkv, D), BF16)                     # keys and values row by row
    hnd = normal(gen, (B, Hkv, n, D), BF16).transpose(1, 2)       # heads outside rows
    seen = trees(gen, B, q, "random")
    lens = torch.tensor([n, 77], dtype=torch.int32).cuda()
    mask = plain.mask_words(seen).cuda()
    for k, v in ((kv[:, :, 0], kv[:, :, 1]), (hnd, hnd), (kv[:, :, 1], hnd)):
        out, lse = mva.gqa_verify_attn(qkv[:, :, :H], k, v, lens, mask, 0.125)
        torch.cuda.synchronize()
        assert mva.last_device_error() == 0
        plain.check(out, lse, qkv[:, :, :H], lambda b: k[b], lambda b: v[b], [n, 77], seen, 0.125)


def paged(c, page, seed=1, spare=2):
    """The case's caches as shuffled pages (NaN wherever no stream's key is) and a block table."""
    gen = torch.Generator().manual_seed(seed)
    B, smax, Hkv, D = c["k"].shape
    n = [-(-x // page) for x in c["lens"]]
    pages = sum(n) + spare
    order = torch.randperm(pages, generator=gen)
    table = torch.full((B, max(max(n), 1)), -7, dtype=torch.int32)
    pools = [torch.full((pages * page, Hkv, D), float("nan"), dtype=c["k"].dtype, device="cuda") for _ in range(2)]
    at = 0
    for b in range(B):
        table[b, :n[b]] = order[at:at + n[b]]
        at += n[b]
        t = torch.arange(c["lens"][b])
        rows = (table[b].long()[t // page] * page + t % page).cuda()
        for pool, x in zip(pools, (c["k"], c["v"])):
            pool[rows] = x[b, :c["lens"][b]]
    return pools, table.cuda()


def run_paged(c, page, pools, table, **kw):
    out, lse = mva.gqa_verify_attn_paged(c["q"], pools[0], pools[1], table, page, c["lens_t"], c["mask"], c["scale"], **kw)
    torch.cuda.synchronize()
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    return out, lse


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 32, 64, 100, 192, 256])
@pytest.mark.parametrize("B,q,H,Hkv,D,lens,dt", [
    (3, 9, 16, 2, 128, [9, 300, 1001], BF16),
    (2, 33, 8, 1, 64, [33, 520], FP16),            # 264 rows
])
def test_pages(B, q, H, Hkv, D, lens, dt, page):
    c = case(B, q, H, Hkv, D, lens, dt)
    pools, table = paged(c, page)
    verify(c, *run_paged(c, page, pools, table))


@pytest.mark.parametrize("page", [64, 48, 32, 8, 5])
def test_pages_of_long_runs(page):
    # Runs of about fifty tiles: the pages are looked up in several batches.
    c = case(3, 3, 16, 8, 64, [30000, 7001, 23333], BF16)
    pools, table = paged(c, page)
    verify(c, *run_paged(c, page, pools, table))


def test_pages_equal_the_contiguous_call():
    c = case(2, 9, 16, 2, 128, [640, 333], BF16, smax=640)
    a = run(c)
    for page in (64, 16, 5):
        b = run_paged(c, page, *paged(c, page))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), page


def test_strided_pools():
    c = case(2, 3, 4, 2, 64, [100, 30], BF16)
    for page in (16, 6):
        (k, v), table = paged(c, page)
        both = torch.stack([k, v], 1)              # [rows, 2, Hkv, D]
        verify(c, *run_paged(c, page, (both[:, 0], both[:, 1]), table))


@pytest.mark.parametrize("page", [64, 16, 5])
def test_pages_far_into_a_large_pool(page):
    # Row offsets beyond 2^32 bytes.
    c = case(1, 9, 16, 8, 128, [500], BF16)
    rows = (2 ** 32 // (8 * 128 * 2) + 4096) // page * page
    pools, table = paged(c, page, spare=0)
    used = pools[0].shape[0]
    big = []
    for pool in pools:
        x = torch.empty((rows, 8, 128), dtype=BF16, device="cuda")
        x[rows - used:] = pool
        big.append(x)
    table = torch.where(table >= 0, table + (rows - used) // page, table)
    verify(c, *run_paged(c, page, big, table))


def test_streams_far_into_a_large_cache():
    # The last stream's rows begin beyond 2^32 bytes of a contiguous cache.
    smax = 1_100_000
    c = case(3, 9, 16, 8, 128, [300, 9, 700], BF16)
    big = []
    for x in (c["k"], c["v"]):
        y = torch.empty((3, smax, 8, 128), dtype=BF16, device="cuda")
        y[:, :x.shape[1]] = x
        big.append(y)
    assert 2 * smax * 8 * 128 * 2 > 2 ** 32
    out, lse = mva.gqa_verify_attn(c["q"], big[0], big[1], c["lens_t"], c["mask"], c["scale"])
    torch.cuda.synchronize()
    assert mva.last_device_error() == 0
    verify(c, out, lse)


@pytest.mark.parametrize("page", [64, 16, 5])
def test_bad_page_is_reported(page):
    c = case(2, 9, 8, 1, 64, [300, 300], BF16)
    pools, table = paged(c, page)
    table[1, 2] = pools[0].shape[0] // page        # one past the pool
    out, lse = mva.gqa_verify_attn_paged(c["q"], pools[0], pools[1], table, page, c["lens_t"], c["mask"], c["scale"])
    torch.cuda.synchronize()
    assert mva.last_device_error() == -10
    plain.check(out[:1], lse[:1], c["q"], lambda b: c["k"][b], lambda b: c["v"][b], [300], c["seen"], c["scale"])


def test_bad_length_is_reported():
    c = case(3, 9, 8, 1, 64, [100, 200, 300], BF16)
    for bad in (8, 301, -1):
        lens = torch.tensor([100, bad, 300], dtype=torch.int32).cuda()
        out, lse = mva.gqa_verify_attn(c["q"], c["k"], c["v"], lens, c["mask"], c["scale"])
        torch.cuda.synchronize()
        assert mva.last_device_error() == -8
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
        plain.check(out[::2], lse[::2], c["q"][::2], lambda b: c["k"][2 * b], lambda b: c["v"][2 * b], [100, 300],
                    c["seen"][::2], c["scale"])


def test_results_are_the_same_every_time_and_nothing_else_is_written():
    c = case(3, 9, 16, 2, 128, [1000, 64, 2500], BF16)
    pad = 4096
    ref = None
    for fill in (0, 255):
        ws = torch.full((mva.gqa_workspace_size(3, 9, 16, 2, 128),), fill, dtype=torch.uint8, device="cuda")
        raw = torch.full((3 * 9 * 16 * 128 + 2 * pad,), 7.0, dtype=BF16, device="cuda")
        out = raw[pad:-pad].view(3, 9, 16, 128)
        got = run(c, out=out, workspace=ws)
        assert (raw[:pad] == 7).all() and (raw[-pad:] == 7).all()
        got = (got[0].clone(), got[1].clone())
        if ref is not None:
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        ref = got


def test_other_stream():
    c = case(2, 9, 16, 2, 64, [700, 100], BF16)
    ref = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"], stream=side)
    with torch.cuda.stream(side):
        again = mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"])
    torch.cuda.synchronize()
    for x in (got, again):
        assert torch.equal(x[0], ref[0]) and torch.equal(x[1], ref[1])


def test_two_calls_at_once():
    # Each with a workspace of its own, on two streams.
    a, b = case(2, 9, 16, 2, 128, [3000, 100], BF16), case(1, 33, 16, 4, 64, [2500], FP16)
    ref = [run(c) for c in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        got.append((mva.gqa_verify_attn(a["q"], a["k"], a["v"], a["lens_t"], a["mask"], a["scale"]),
                    mva.gqa_verify_attn(b["q"], b["k"], b["v"], b["lens_t"], b["mask"], b["scale"], stream=side)))
    torch.cuda.synchronize()
    assert mva.last_device_error() == 0
    for pair in got:
        for (out, lse), (o, l) in zip(pair, ref):
            assert torch.equal(out, o) and torch.equal(lse, l)


def test_captured_call_follows_new_lengths():
    c = case(2, 9, 16, 2, 128, [900, 1300], BF16, smax=1300)
    c["k"].nan_to_num_(0.5)
    c["v"].nan_to_num_(0.5)
    ws = torch.empty(mva.gqa_workspace_size(2, 9, 16, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = run(c, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"], out=out, lse=lse, workspace=ws)
    for lens in ([1300, 9], [0, 640], [65, 1299]):
        c["lens"] = lens
        c["lens_t"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert mva.last_device_error() == 0
        verify(c, out, lse)


def test_two_graphs_share_a_workspace_in_order():
    a, b = case(1, 9, 16, 2, 128, [900], BF16), case(1, 9, 16, 2, 128, [1700], BF16, seed=9)
    ws = torch.empty(mva.gqa_workspace_size(1, 9, 16, 2, 128), dtype=torch.uint8, device="cuda")
    res, graphs = [run(a, workspace=ws), run(b, workspace=ws)], []
    for c, (out, lse) in zip((a, b), res):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"], out=out, lse=lse, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g, (out, lse) in zip(graphs, res):
            out.fill_(float("nan"))
            g.replay()
    torch.cuda.synchronize()
    verify(a, *res[0])
    verify(b, *res[1])


def test_inputs_rewritten_between_calls():
    # Dependent launches keep the stream's order.
    c = case(1, 9, 16, 2, 64, [300], BF16)
    first = [x.clone() for x in run(c)]
    q0 = c["q"].clone()
    outs = []
    for k in range(6):
        c["q"].copy_(q0 if k % 2 == 0 else -q0)
        outs.append(mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"]))
    torch.cuda.synchronize()
    for k in range(0, 6, 2):
        assert torch.equal(outs[k][0], first[0]) and torch.equal(outs[k][1], first[1])
        assert torch.equal(outs[k + 1][0], outs[1][0])


@pytest.mark.parametrize("page", [0, 16, 5])
def test_wait_that_runs_out_is_reported(page):
    c = case(1, 9, 16, 2, 128, [2000], BF16)
    ref = run(c)
    pools, table = paged(c, page) if page else (None, None)
    with mva.forced(stall=True):
        if page:
            mva.gqa_verify_attn_paged(c["q"], pools[0], pools[1], table, page, c["lens_t"], c["mask"], c["scale"])
        else:
            mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"])
        assert mva.last_device_error() == -7
    got = run(c)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_refusals():
    c = case(1, 9, 16, 2, 64, [100], BF16)
    a = dict(q=c["q"], k=c["k"], v=c["v"], seq_lens=c["lens_t"], tree_mask=c["mask"], scale=0.1)

    def refused(error, **kw):
        with pytest.raises(error):
            mva.gqa_verify_attn(**{**a, **kw})

    refused(ValueError, q=c["q"].half())
    refused(ValueError, q=c["q"].float(), k=c["k"].float(), v=c["v"].float())
    refused(ValueError, seq_lens=c["lens_t"].long())
    refused(ValueError, tree_mask=c["mask"].expand(1, 9, 2))
    refused(ValueError, v=c["v"][:, :50])
    refused(ValueError, q=c["q"].transpose(2, 3).contiguous().transpose(2, 3))
    refused(ValueError, k=c["k"].cpu())
    refused(ValueError, out=torch.empty((1, 9, 16, 64), device="cuda"))
    refused(mva.MLAError, scale=float("inf"))
    refused(mva.MLAError, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    refused(mva.MLAError, q=c["q"][:, :, :15].contiguous())                      # 15 heads over 2
    refused(mva.MLAError, k=c["k"][..., :32].contiguous(), v=c["v"][..., :32].contiguous(),
            q=c["q"][..., :32].contiguous())                                     # a head of 32
    odd = torch.empty(c["k"].numel() + 4, dtype=BF16, device="cuda")[4:].view(c["k"].shape)
    refused(mva.MLAError, k=odd)                                                 # 8-byte aligned only
    torch.cuda.synchronize()
    assert mva.last_device_error() == 0
    out, lse = mva.gqa_verify_attn(c["q"][:0], c["k"][:0], c["v"][:0], c["lens_t"][:0], c["mask"][:0], 0.1)
    assert out.shape == (0, 9, 16, 64) and lse.shape == (0, 9, 16)
