"""Grouped-head attention with a sliding window and first tokens on the GPU
against its plain 64-bit form: windows and sinks around tile edges, trees deeper
than the window, rows without a key, keys in the gap that hold anything, pages
of every kind that were given away, graphs and refusals."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import gqa_plain
import long_cache_plain as plain
from test_gqa_attn import trees

BF16, FP16 = torch.bfloat16, torch.float16
JUNK = float("nan")


def unused(n, q, window, sinks):
    """Rows that the call may not use."""
    return slice(min(sinks, max(n - q - window, 0)), max(n - q - window, 0))


def case(q, H, Hkv, D, lens, window, sinks, dt=BF16, tree="random", smax=None, seed=0):
    gen = torch.Generator().manual_seed(seed + 31 * q + D + window)
    B, smax = len(lens), smax or max(max(lens), 1)
    rand = lambda *s: torch.randn(s, generator=gen).to(dt).cuda()
    c = dict(q=rand(B, q, H, D), k=rand(B, smax, Hkv, D), v=rand(B, smax, Hkv, D), lens=lens, window=window, sinks=sinks,
             seen=trees(gen, B, q, tree), scale=1 / math.sqrt(D), gen=gen)
    for b, n in enumerate(lens):
        for x in (c["k"], c["v"]):
            x[b, n:] = JUNK
            if n:
                x[b, unused(n, q, window, sinks)] = JUNK
    c["lens_t"] = torch.tensor(lens, dtype=torch.int32).cuda()
    c["mask"] = gqa_plain.mask_words(c["seen"]).cuda()
    return c


def run(c, **kw):
    got = mva.gqa_verify_attn_window(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"], c["window"], c["sinks"], **kw)
    torch.cuda.synchronize()
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    return got


def verify(c, got):
    for b, n in enumerate(c["lens"]):
        see = plain.seen_keys(c["seen"][b], n, c["window"], c["sinks"]) if n else torch.zeros((c["q"].shape[1], 0)).bool()
        plain.check(got[0][b], got[1][b], plain.attend(c["q"][b], c["k"][b, :n], c["v"][b, :n], see, c["scale"]), "stream %d" % b)


def paged(c, page, forget=True):
    """The same rows on pages in random order; entries of pages in the gap are -1."""
    q = c["q"].shape[1]
    table, total = plain.pages(c["gen"], c["lens"], page)
    Hkv, D = c["k"].shape[2:]
    pools = [torch.full((total * page, Hkv, D), JUNK, dtype=c["k"].dtype, device="cuda") for _ in range(2)]
    for b, n in enumerate(c["lens"]):
        rows = plain.rows_of(table[b], page, n).cuda()
        pools[0][rows], pools[1][rows] = c["k"][b, :n], c["v"][b, :n]
        if forget and n:
            gap = unused(n, q, c["window"], c["sinks"])
            table[b, -(-gap.start // page):gap.stop // page] = -1
    return pools, table.cuda()


def run_paged(c, page, pools, table, **kw):
    got = mva.gqa_verify_attn_window_paged(c["q"], *pools, table, page, c["lens_t"], c["mask"], c["scale"], c["window"],
                                           c["sinks"], **kw)
    torch.cuda.synchronize()
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    return got


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,H,Hkv,lens,window,sinks", [
    (1, 1, 1, [1], 1, 0),                        # one key
    (1, 8, 1, [1000], 1, 0),                     # nothing but the token itself
    (1, 8, 2, [1000, 64, 65, 130], 64, 4),       # the window is a tile long
    (9, 64, 8, [3000], 256, 4),
    (9, 64, 8, [9000, 12, 300], 1024, 64),       # whole streams within the window among them
    (5, 6, 2, [700, 0, 1300], 63, 65),           # sinks over a tile's edge, an unused stream
    (33, 16, 4, [2000], 300, 1),                 # 132 rows: two row tiles
    (64, 7, 1, [100, 1000], 200, 10),            # 448 rows
    (9, 8, 8, [5000], 4990, 3),                  # a gap of a few keys
    (9, 8, 2, [5000, 200], 100000, 100000),      # a window over everything
])
def test_matches_plain(q, H, Hkv, lens, window, sinks, D, dt):
    c = case(q, H, Hkv, D, lens, window, sinks, dt)
    verify(c, run(c))


@pytest.mark.parametrize("window", [1, 2, 62, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("sinks", [0, 1, 63, 64, 65, 128])
def test_windows_and_sinks_around_tile_edges(window, sinks):
    c = case(3, 8, 2, 128, [3, 64, 67, 128, 131, 192, 195, 260, 500, 803], window, sinks)
    verify(c, run(c))
    verify(c, run_paged(c, 64, *paged(c, 64)))


@pytest.mark.parametrize("tree", ["chain", "random", "any"])
@pytest.mark.parametrize("q,window,sinks", [(40, 7, 2), (64, 1, 0), (64, 33, 70), (33, 32, 600), (17, 16, 0)])
def test_trees_deeper_than_the_window(q, window, sinks, tree):
    # Drafts hide drafts, sinks reach into the drafts, rows that see none of them.
    c = case(q, 8, 2, 64, [q, q + 1, q + 63, 600], window, sinks, tree=tree)
    verify(c, run(c))


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 64, 100, 128])
def test_pages_in_the_gap_may_have_been_given_away(page):
    for D, dt in ((64, FP16), (128, BF16)):
        c = case(5, 16, 2, D, [1500, 5, 700, 64, 0, 4000], 333, 10, dt)
        pools, table = paged(c, page)
        verify(c, run_paged(c, page, pools, table))


def test_a_page_that_is_needed_is_reported():
    c = case(5, 16, 2, 64, [1500], 333, 10)
    for page in (5, 16, 64):
        for key in (0, 1500 - 5 - 333, 1499):
            pools, table = paged(c, page)
            table[0, key // page] = 1 << 20
            mva.gqa_verify_attn_window_paged(c["q"], *pools, table, page, c["lens_t"], c["mask"], c["scale"], 333, 10)
            assert mva.last_device_error() == -10


def test_a_window_over_everything_gives_what_the_call_without_gives():
    c = case(9, 32, 4, 128, [900, 5000, 64], 1 << 30, 0)
    a = run(c)
    b = mva.gqa_verify_attn(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_streams():
    gen = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(5, 3000, (200,), generator=gen)]
    c = case(5, 8, 2, 64, lens, 200, 4)
    a = run(c)
    verify(c, a)
    pools, table = paged(c, 16)
    b = run_paged(c, 16, pools, table)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_strided_views_and_another_stream():
    c = case(9, 16, 2, 128, [3000, 700], 500, 4)
    fused = torch.randn((2, 3000, 8, 128), device="cuda").to(BF16)
    fused[:, :, 2:4], fused[:, :, 5:7] = c["k"], c["v"]
    want = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mva.gqa_verify_attn_window(c["q"], fused[:, :, 2:4], fused[:, :, 5:7], c["lens_t"], c["mask"], c["scale"], 500, 4,
                                     stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_and_replayed_with_other_lengths():
    c = case(1, 16, 2, 128, [5000, 300, 4000], 1024, 4)
    run(c)
    into = dict(out=torch.empty_like(c["q"]), lse=torch.empty(3, 1, 16, device="cuda"),
                workspace=torch.empty(mva.gqa_workspace_size(3, 1, 16, 2, 128), dtype=torch.uint8, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mva.gqa_verify_attn_window(c["q"], c["k"], c["v"], c["lens_t"], c["mask"], c["scale"], 1024, 4, **into)
    for lens in ([5000, 300, 4000], [1100, 0, 2000]):
        c["lens"] = lens
        c["k"].normal_(), c["v"].normal_()
        c["lens_t"].copy_(torch.tensor(lens))
        graph.replay()
        torch.cuda.synchronize()
        verify(c, (into["out"], into["lse"]))


def test_refusals():
    c = case(2, 4, 2, 64, [100], 50, 4)
    call = lambda **kw: mva.gqa_verify_attn_window(*[kw.get(n, c[n]) for n in ("q", "k", "v", "lens_t", "mask", "scale")],
                                                   kw.get("window", 50), kw.get("sinks", 4))
    for bad in (dict(window=0), dict(window=-3), dict(sinks=-1)):
        with pytest.raises(mva.MLAError) as e:
            call(**bad)
        assert e.value.status == -2
    for bad in (dict(v=c["v"][:, :50]), dict(q=c["q"].float()), dict(lens_t=c["lens_t"].long()), dict(mask=c["mask"][:, :1])):
        with pytest.raises(ValueError):
            call(**bad)
    mva.gqa_verify_attn_window(c["q"], c["k"], c["v"], torch.tensor([101], dtype=torch.int32).cuda(), c["mask"], 0.1, 50)
    assert mva.last_device_error() == -8
