"""Grouped-head attention over a cache held in 4 bits, on the GPU against its
plain 64-bit form over the values that the rows stand for: types, head layouts,
lengths around tile edges, masks, steps and rows of q of every size, pages of
every kind, steps of a loop (append, attend, keep), graphs and refusals."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import gqa_plain
import long_cache_plain as plain
from test_gqa_attn import trees

BF16, FP16 = torch.bfloat16, torch.float16


def case(q, H, Hkv, D, lens, page, dt=BF16, tree="random", seed=0, spread=0.0, k_scale=0.125, v_scale=0.5, scale=None, room=0):
    """Pools of random codes and steps, so that every value is exact; rows that no stream has hold NaN.
    room: keys that the table has room for, at least (by which the kernel for few rows is chosen)."""
    gen = torch.Generator().manual_seed(seed + 19 * q + D + page)
    B = len(lens)
    table, total = plain.pages(gen, lens, page)
    if table.shape[1] * page < room:
        table = torch.cat([table, torch.full((B, -(-room // page) - table.shape[1]), -1, dtype=torch.int32)], 1)
    n = mva.gqa_fp4_row_bytes(Hkv, D)
    codes = Hkv * D // 2
    pools = []
    for _ in range(2):
        p = torch.randint(0, 256, (total * page, n), dtype=torch.uint8, generator=gen)
        step = torch.exp(spread * torch.randn((total * page, Hkv * D // 16), generator=gen)) * 0.6
        p[:, codes:codes + Hkv * D // 16] = step.clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pools.append(p)
    used = torch.cat([plain.rows_of(table[b], page, x) for b, x in enumerate(lens)]) if sum(lens) else torch.zeros(0).long()
    junk = torch.ones(total * page, dtype=torch.bool)
    junk[used] = False
    for p in pools:
        p[junk] = 255
    c = dict(q=torch.randn((B, q, H, D), generator=gen).to(dt).cuda(), pools=[p.cuda() for p in pools], cpu=pools, lens=lens,
             page=page, table=table, Hkv=Hkv, seen=trees(gen, B, q, tree), k_scale=k_scale, v_scale=v_scale,
             scale=scale if scale is not None else 0.5 / math.sqrt(D) / k_scale)
    c["lens_t"] = torch.tensor(lens, dtype=torch.int32).cuda()
    c["mask"] = gqa_plain.mask_words(c["seen"]).cuda()
    c["table_t"] = table.clamp_min(0).cuda()
    return c


def run(c, **kw):
    got = mva.gqa_verify_attn_fp4_paged(kw.pop("q", c["q"]), *c["pools"], c["Hkv"], c["table_t"], c["page"], c["lens_t"], c["mask"],
                                        c["scale"], c["k_scale"], c["v_scale"], **kw)
    torch.cuda.synchronize()
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    return got


def verify(c, got):
    D = c["q"].shape[-1]
    for b, n in enumerate(c["lens"]):
        rows = plain.rows_of(c["table"][b], c["page"], n)
        k, v = (plain.unpack_fp4(p[rows], c["Hkv"], D, f).cuda() for p, f in zip(c["cpu"], (c["k_scale"], c["v_scale"])))
        see = plain.seen_keys(c["seen"][b], n) if n else torch.zeros((c["q"].shape[1], 0)).bool()
        # (the weights are fp16 here, whatever q's type)
        plain.check(got[0][b], got[1][b], plain.attend(c["q"][b], k, v, see, c["scale"], weight_u=2.0 ** -11), "stream %d" % b)


@pytest.mark.parametrize("room", [0, 270000])
@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,H,Hkv,lens", [
    (1, 1, 1, [1]),
    (1, 8, 1, [64]),
    (1, 64, 8, [1000, 1, 130]),
    (1, 16, 8, [300, 65]),                     # two rows a key head
    (1, 14, 2, [700]),
    (2, 8, 1, [129, 2]),                       # 16 rows
    (3, 8, 1, [500]),                          # 24 rows
    (4, 16, 2, [500, 66, 4]),                  # 32 rows
    (4, 64, 8, [1500, 300]),
    (2, 64, 8, [700, 2, 65]),                  # 16 and 24 rows of eight key heads
    (3, 64, 8, [1500, 300]),
    (3, 48, 16, [700, 3]),                     # two sets of eight heads
    (11, 9, 3, [700]),                         # 33 rows
    (32, 2, 2, [700, 32, 33, 60]),             # 32 drafts of a head: one mask word, all of it
    (32, 8, 8, [100]),
    (9, 64, 8, [265]),
    (2, 21, 3, [600, 63]),                     # an odd number of heads: rows with padding
    (5, 5, 5, [64, 0, 190]),
    (16, 8, 1, [16, 700]),                     # 128 rows exactly
    (33, 16, 4, [2000]),
    (64, 14, 2, [100, 1000]),                  # 448 rows
])
def test_matches_plain(q, H, Hkv, lens, D, dt, room):
    c = case(q, H, Hkv, D, lens, 64, dt, room=room)
    verify(c, run(c))


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 64, 100, 128, 4096])
@pytest.mark.parametrize("q,H,Hkv", [(1, 16, 2), (5, 16, 2), (5, 24, 8)])
def test_pages(q, H, Hkv, page):
    for D, dt in ((64, FP16), (128, BF16)):
        c = case(q, H, Hkv, D, [1500, 5, 700, 64, 0, 4000], page, dt, room=50000)
        verify(c, run(c))


@pytest.mark.parametrize("q,H,Hkv", [(1, 8, 1), (1, 8, 8), (1, 6, 3), (1, 16, 16), (1, 40, 40), (1, 12, 12), (4, 4, 2), (1, 72, 24), (9, 36, 36)])
def test_head_layouts(q, H, Hkv):
    for D in (64, 128):
        c = case(q, H, Hkv, D, [max(q, 3), 200, 1111], 16, room=90000)
        verify(c, run(c))


@pytest.mark.parametrize("tree", ["chain", "any"])
@pytest.mark.parametrize("q,G,lens", [(1, 8, [1, 64, 65]), (2, 4, [2, 66]), (4, 4, [4, 70]), (6, 4, [6, 65]), (8, 4, [9, 70]),
                                      (9, 8, [9, 70]), (40, 2, [41, 130]), (64, 4, [64, 129])])
def test_masks(q, G, lens, tree):
    for Hkv, room in ((2, 0), (2, 1100), (8, 140000)):
        c = case(q, Hkv * G, Hkv, 64, lens, 16, tree=tree, room=room)
        verify(c, run(c))


def test_lengths_around_tile_edges():
    for q, H, Hkv in ((1, 4, 1), (4, 16, 1), (4, 16, 8)):
        c = case(q, H, Hkv, 128, [n for k in (16, 32, 64, 128, 192, 256, 512, 1024) for n in (k - 1, k, k + 1)], 64)
        verify(c, run(c))
        c = case(q, H, Hkv, 64, list(range(q, 100)), 16)
        verify(c, run(c))


@pytest.mark.parametrize("q", [1, 9])
def test_steps_and_queries_of_every_size(q):
    for D, dt in ((64, BF16), (128, FP16), (128, BF16)):
        c = case(q, 8, 2, D, [900, 77], 16, dt, spread=1.5, room=1024)
        verify(c, run(c))
    for size in (1e-30, 1e-6, 1e4, 1e30):                  # bf16 has fp32's range
        c = case(q, 8, 2, 64, [900, 77], 16, BF16, room=1024)
        c["q"] = (c["q"].float() * size).to(BF16)
        c["scale"] /= size
        verify(c, run(c))
    for scale in (0.0, -0.7, 3.0):
        c = case(q, 8, 2, 128, [900, 77], 16, scale=scale, room=1024)
        verify(c, run(c))
    c = case(q, 8, 2, 128, [900, 77], 16, k_scale=2.0 ** -40, v_scale=2.0 ** 30, room=1024)
    verify(c, run(c))


@pytest.mark.parametrize("q", [1, 2, 9])
def test_drafts_that_none_sees_hold_anything(q):
    # Padding drafts' rows: codes with steps of NaN.
    c = case(q, 16, 8 if q == 2 else 2, 128, [300, 64 + q], 16, room=140000)
    c["seen"][0, :, q - 1] = False
    c["mask"] = gqa_plain.mask_words(c["seen"]).cuda()
    for p, x in zip(c["pools"], c["cpu"]):
        x[plain.rows_of(c["table"][0], 16, 300)[299]] = 255
        p.copy_(x)
    verify(c, run(c))


def test_nan_of_a_row_stays_in_it():
    for n in (100, 5000):
        for q in (1, 5):
            c = case(q, 8, 2, 128, [n], 64)
            c["q"][0, 0, 3, 7] = float("nan")
            out, lse = run(c)
            bad = torch.zeros((q, 8), dtype=torch.bool, device="cuda")
            bad[0, 3] = True
            assert torch.equal(torch.isnan(lse[0]), bad)
            assert torch.equal(torch.isnan(out[0]).all(-1), bad) and torch.equal(torch.isnan(out[0]).any(-1), bad)


@pytest.mark.parametrize("q,H,Hkv", [(1, 8, 2), (3, 16, 2), (5, 16, 2), (3, 24, 8), (4, 32, 8)])
def test_many_streams_and_long_ones(q, H, Hkv):
    gen = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(q, 900, (300,), generator=gen)] + [0]
    c = case(q, H, Hkv, 64, lens, 16)
    a = run(c)
    verify(c, a)
    for _ in range(10):
        b = run(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = case(q, H, Hkv, 128, [40000, q, 20000], 64)
    verify(c, run(c))


def test_strided_queries_and_another_stream():
    for q in (1, 9):
        c = case(q, 16, 2, 128, [3000, 700], 16)
        wide = torch.randn((2, q, 32, 128), device="cuda").to(BF16)
        wide[:, :, 4:20] = c["q"]
        want = run(c)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = run(c, q=wide[:, :, 4:20], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_of_wider_pools():
    for q in (1, 9):
        c = case(q, 16, 2, 128, [3000, 700], 16)
        want = run(c)
        wide = torch.full((len(c["cpu"][0]), 2, 160), 255, dtype=torch.uint8, device="cuda")
        wide[:, 0, :144], wide[:, 1, :144] = c["pools"]
        c["pools"] = [wide[:, 0, :144], wide[:, 1, :144]]
        got = run(c)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("q,H", [(1, 16), (9, 16)])
def test_a_loop_of_steps_and_its_graph(q, H):
    # Extend, append, attend, keep, trim, as a serving loop runs them.
    gen = torch.Generator().manual_seed(q)
    Hkv, D, page, B = 2, 64, 16, 3
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    lens = [100, 0, 37]
    pages = 64
    pools = [torch.zeros((pages * page, mva.gqa_fp4_row_bytes(Hkv, D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    seq, table = i32([0] * B), torch.zeros((B, 20), dtype=torch.int32, device="cuda")
    free, count = torch.randperm(pages, generator=gen).int().cuda(), i32([pages])
    history = [[torch.zeros((0, Hkv, D)), torch.zeros((0, Hkv, D))] for _ in range(B)]

    def append(new):
        slots = torch.empty(sum(new), dtype=torch.int32, device="cuda")
        mva.blocks_extend(seq, i32(new), table, page, free, count, pages, slots)
        x = [torch.randn((sum(new), Hkv, D), generator=gen).to(BF16).cuda() for _ in range(2)]
        held = [torch.empty_like(y) for y in x]
        mva.gqa_cache_append_fp4(*pools, *x, slots, 0.25, 0.25, *held)
        at = 0
        for b, n in enumerate(new):
            for i in range(2):
                history[b][i] = torch.cat([history[b][i], held[i][at:at + n].cpu().float()])
            at += n

    append(lens)
    seen = trees(gen, B, q, "random")
    mask = gqa_plain.mask_words(seen).cuda()
    for step in range(4):
        append([q] * B)
        qs = torch.randn((B, q, H, D), generator=gen).to(BF16).cuda()
        out, lse = mva.gqa_verify_attn_fp4_paged(qs, *pools, Hkv, table, page, seq, mask, 0.125, 0.25, 0.25)
        for b in range(B):
            k, v = (x.cuda().double() for x in history[b])
            plain.check(out[b], lse[b], plain.attend(qs[b], k, v, plain.seen_keys(seen[b], len(k)), 0.125, weight_u=2.0 ** -11))
        kept = [min(q, 1 + (step + b) % 4) for b in range(B)]
        path = torch.stack([torch.randperm(q, generator=gen).sort().values for _ in range(B)]).int()
        mva.gqa_cache_keep_fp4(*pools, table, page, seq, path.cuda(), i32(kept))
        for b in range(B):
            for i in range(2):
                n = len(history[b][i]) - q
                history[b][i] = torch.cat([history[b][i][:n], history[b][i][n + path[b, :kept[b]].long()]])
        mva.blocks_trim(seq, i32([len(h[0]) for h in history]), table, page, free, count)
    graph = torch.cuda.CUDAGraph()
    into = dict(out=torch.empty_like(out), lse=torch.empty_like(lse),
                workspace=torch.empty(mva.gqa_fp4_workspace_size(B, q, H, Hkv, D), dtype=torch.uint8, device="cuda"))
    append([q] * B)
    with torch.cuda.graph(graph):
        mva.gqa_verify_attn_fp4_paged(qs, *pools, Hkv, table, page, seq, mask, 0.125, 0.25, 0.25, **into)
    for _ in range(2):
        qs.copy_(torch.randn((B, q, H, D), generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            k, v = (x.cuda().double() for x in history[b])
            plain.check(into["out"][b], into["lse"][b],
                        plain.attend(qs[b], k, v, plain.seen_keys(seen[b], len(k)), 0.125, weight_u=2.0 ** -11))
    assert mva.last_device_error() == 0


@pytest.mark.parametrize("q,page", [(1, 16), (1, 5), (9, 16), (9, 5)])
def test_a_wait_that_runs_out_is_reported(q, page):
    c = case(q, 16, 2, 128, [3000], page)
    with mva.forced(stall=True):
        mva.gqa_verify_attn_fp4_paged(c["q"], *c["pools"], 2, c["table_t"], page, c["lens_t"], c["mask"], 0.1)
        assert mva.last_device_error() == -7
    verify(c, run(c))


@pytest.mark.parametrize("q,H,room", [(1, 8, 0), (1, 8, 4096), (9, 8, 0)])
def test_pages_and_lengths_out_of_range_are_reported(q, H, room):
    c = case(q, H, 2, 64, [500, 40], 16, room=room)
    call = lambda table, lens: mva.gqa_verify_attn_fp4_paged(c["q"], *c["pools"], 2, table, 16, lens, c["mask"], 0.1)
    for at in (0, 31):
        for bad in (-1, 1 << 20):
            t = c["table_t"].clone()
            t[0, at] = bad
            call(t, c["lens_t"])
            assert mva.last_device_error() == -10
    out, lse = call(c["table_t"], torch.tensor([max(513, room + 1), 40], dtype=torch.int32).cuda())
    assert mva.last_device_error() == -8
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


def test_refusals():
    c = case(2, 4, 2, 64, [100], 16)
    good = [c["q"], *c["pools"], 2, c["table_t"], 16, c["lens_t"], c["mask"], 0.1]
    for i, bad in ((0, c["q"].float()), (1, c["pools"][0][:, :48]), (2, c["pools"][1][:5]), (3, 1), (4, c["table_t"].long()),
                   (6, c["lens_t"][:0]), (7, c["mask"][:, :1])):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            mva.gqa_verify_attn_fp4_paged(*args)
    for i, bad, want in ((5, 0, -2), (5, 7, -2), (8, float("nan"), -9)):
        args = list(good)
        args[i] = bad
        with pytest.raises(mva.MLAError) as e:
            mva.gqa_verify_attn_fp4_paged(*args)
        assert e.value.status == want
    for f in (0.0, -1.0, float("inf"), float("nan")):
        for kw in (dict(k_scale=f), dict(v_scale=f)):
            with pytest.raises(mva.MLAError) as e:
                mva.gqa_verify_attn_fp4_paged(*good, **kw)
            assert e.value.status == -9
    with pytest.raises(mva.MLAError) as e:
        mva.gqa_verify_attn_fp4_paged(*good, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4


@pytest.mark.parametrize("q,Hkv", [(1, 8), (3, 8), (9, 8)])
@pytest.mark.parametrize("page", [64, 100])
def test_pools_beyond_2_to_the_32_bytes(q, Hkv, page):
    # Rows appended to, and read from, both ends of pools of 5 GB.
    D, H, n = 128, 8 * Hkv, 9_000_000
    width = mva.gqa_fp4_row_bytes(Hkv, D)
    pages = n // page
    pools = [torch.zeros((pages * page, width), dtype=torch.uint8, device="cuda") for _ in range(2)]
    lens = [300, 2000]
    table = torch.zeros((2, -(-9000 // page)), dtype=torch.int32)
    for b, length in enumerate(lens):
        for j in range(-(-length // page)):
            table[b, j] = pages - 1 - (2 * j + b) if j % 3 else 2 * j + b
    gen = torch.Generator().manual_seed(q)
    x = [torch.randn((sum(lens), Hkv, D), generator=gen).to(BF16).cuda() for _ in range(2)]
    slots = torch.cat([plain.rows_of(table[b], page, m) for b, m in enumerate(lens)]).int().cuda()
    held = [torch.empty_like(y) for y in x]
    mva.gqa_cache_append_fp4(*pools, *x, slots, 0.25, 0.25, *held)
    seen = trees(gen, 2, q, "random")
    qs = torch.randn((2, q, H, D), generator=gen).to(BF16).cuda()
    out, lse = mva.gqa_verify_attn_fp4_paged(qs, *pools, Hkv, table.cuda(), page, torch.tensor(lens, dtype=torch.int32).cuda(),
                                             gqa_plain.mask_words(seen).cuda(), 0.1, 0.25, 0.25)
    assert mva.last_device_error() == 0
    at = 0
    for b, m in enumerate(lens):
        k, v = (y[at:at + m].double() for y in held)
        plain.check(out[b], lse[b], plain.attend(qs[b], k, v, plain.seen_keys(seen[b], m), 0.1, weight_u=2.0 ** -11), "stream %d" % b)
        at += m


@pytest.mark.parametrize("q,H,Hkv,room", [(1, 8, 2, 4096), (1, 8, 2, 0), (1, 8, 8, 4096), (2, 64, 8, 140000), (3, 64, 8, 270000),
                                          (4, 64, 8, 270000), (3, 64, 8, 0), (9, 8, 2, 0)])
def test_scores_far_below_zero(q, H, Hkv, room):
    # Every score is -2^106 or -2^105 (exact in fp32, as are the quotients): the larger ones share the weight.
    for lens, larger in (([max(q, 1), 70, 900], 0), ([70, 130, 900], 40)):
        c = case(q, H, Hkv, 64, lens, 16, BF16, tree="chain", room=room)
        c["scale"], c["k_scale"] = 2.0 ** -4, 0.25
        head, codes = 32, Hkv * 32
        for h in range(Hkv):
            c["cpu"][0][:, h * head] = 0x22                    # 1.0 and 1.0
            c["cpu"][0][:, codes + h * 4] = 0x38               # a step of 1
        for b, n in enumerate(lens):
            if larger:
                c["cpu"][0][plain.rows_of(c["table"][b], 16, n)[larger - 1], [h * head for h in range(Hkv)]] = 0x21   # 0.5
        c["pools"][0].copy_(c["cpu"][0])
        c["q"].zero_()
        c["q"][..., 0] = -2.0 ** 112
        out, lse = run(c)
        for b, n in enumerate(lens):
            rows = plain.rows_of(c["table"][b], 16, n)
            v = plain.unpack_fp4(c["cpu"][1][rows], Hkv, 64, c["v_scale"]).cuda()
            see = plain.seen_keys(c["seen"][b], n)
            if larger:
                see &= (torch.arange(n) == larger - 1)[None]
            even = plain.attend(torch.zeros_like(c["q"][b]), v, v, see, 1.0, weight_u=2.0 ** -11)
            plain.check(out[b], even[1].float(), even, "stream %d" % b)
            want = torch.full_like(lse[b], -2.0 ** (105 if larger else 106)).double()
            assert ((lse[b].double() - want).abs() <= 2.0 ** -22 * want.abs()).all()


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 100])
@pytest.mark.parametrize("q", [1, 2, 3, 4])
def test_up_to_32_rows_whatever_the_table_has_room_for(q, page, D, dt):
    # 7 or 8 heads a key head, 8 key heads: the kernel for few rows and the other one, by streams and room.
    for H, lens, room in ((64, [700], 0), (64, [700], 140000), (56, [300, 64, 1200], 3000), (56, [300, 64, 1200], 50000)):
        c = case(q, H, 8, D, lens, page, dt, room=room)
        verify(c, run(c))
    gen = torch.Generator().manual_seed(q)
    for B in (33, 70):
        c = case(q, 64, 8, D, [int(x) for x in torch.randint(q, 200, (B,), generator=gen)], page, dt)
        verify(c, run(c))


def test_the_workspace_does_for_every_room():
    # Its size is asked for without a table's room.
    for q, H, Hkv in ((1, 64, 8), (2, 64, 8), (3, 64, 8), (4, 64, 8), (5, 64, 8), (1, 40, 5), (1, 24, 3)):
        ws = torch.full((mva.gqa_fp4_workspace_size(3, q, H, Hkv, 128) + 4096,), 7, dtype=torch.uint8, device="cuda")
        for room in (0, 3000, 70000, 270000):
            c = case(q, H, Hkv, 128, [700, 30, 2500], 16, room=room)
            got = run(c, workspace=ws[:-4096])
            verify(c, got)
            assert (ws[-4096:] == 7).all()


@pytest.mark.parametrize("page", [1, 5, 100])
@pytest.mark.parametrize("q,H,Hkv", [(1, 16, 16), (1, 24, 12), (1, 40, 40), (1, 20, 5), (1, 72, 24), (4, 64, 16), (3, 64, 16)])
def test_sets_of_heads_in_pages_that_are_copied_row_by_row(q, H, Hkv, page):
    # More key heads than a CTA takes at once: their steps begin anywhere in 16 bytes of a row.
    for D, dt in ((64, BF16), (128, FP16)):
        c = case(q, H, Hkv, D, [700, max(q, 3), 0, 1111], page, dt, room=90000)
        verify(c, run(c))
