"""Block tables, slot maps, appended and kept cache rows on the GPU against
plain Python, and whole verify steps over caches that only they maintain."""
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import gqa_plain as plain

BF16, FP16 = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Pool:
    """A plain model of the block tables and the free list."""

    def __init__(self, lens, page, max_blocks, spare, seed=0):
        rng = random.Random(seed)
        self.page, self.lens = page, list(lens)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = rng.sample(range(self.pages), self.pages)
        self.table = [[-1] * max_blocks for _ in lens]
        for b, n in enumerate(need):
            self.table[b][:n] = [order.pop() for _ in range(n)]
        self.free = order + [-5] * 0
        self.count = len(self.free)

    def gpu(self, slots):
        self.t = dict(lens=ints(self.lens), table=ints(self.table), free=ints(self.free + [-9] * (self.pages - len(self.free))),
                      count=ints([self.count]), slots=torch.full((slots,), -77, dtype=torch.int32, device="cuda"))
        return self.t

    def extend(self, new):
        slots = []
        for b, n in enumerate(new):
            for pos in range(self.lens[b], self.lens[b] + n):
                blk = pos // self.page
                if pos % self.page == 0:
                    self.table[b][blk] = self.free[self.count - 1]
                    self.count -= 1
                slots.append(self.table[b][blk] * self.page + pos % self.page)
            self.lens[b] += n
        return slots

    def trim(self, keep):
        gone = []
        for b, n in enumerate(keep):
            gone += self.table[b][-(-n // self.page):-(-self.lens[b] // self.page)]
            self.lens[b] = n
        self.free = self.free[:self.count] + gone[::-1]
        self.count += len(gone)

    def same(self):
        t = self.t
        assert t["lens"].tolist() == self.lens
        assert t["count"].tolist() == [self.count]
        assert t["free"].tolist()[:self.count] == self.free[:self.count]
        table = t["table"].tolist()
        for b, n in enumerate(self.lens):
            k = -(-n // self.page)
            assert table[b][:k] == self.table[b][:k], b


def extend(p, new, stream=None):
    t = p.t
    mva.blocks_extend(t["lens"], ints(new), t["table"], p.page, t["free"], t["count"], p.pages, t["slots"], stream=stream)


def trim(p, keep):
    t = p.t
    mva.blocks_trim(t["lens"], ints(keep), t["table"], p.page, t["free"], t["count"])


def ok(expect=0):
    torch.cuda.synchronize()
    assert mva.last_device_error() == expect


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("B,most,old", [(1, 1, 0), (1, 9, 100), (8, 9, 300), (37, 40, 50), (300, 200, 70), (2500, 6, 9)])
def test_extend_and_trim(B, most, old, page):
    rng = random.Random(B + page)
    p = Pool([rng.randint(0, old) for _ in range(B)], page, (old + 3 * most) // page + 2, B * (3 * most // page + 2))
    p.gpu(B * most + 5)
    for step in range(3):
        new = [rng.randint(0, most) for _ in range(B)]
        before = list(p.lens)
        slots = p.extend(new)
        extend(p, new)
        ok()
        p.same()
        assert p.t["slots"].tolist() == slots + [-1] * (B * most + 5 - len(slots))
        assert len(set(slots)) == len(slots)
        keep = [rng.choice([0, n, rng.randint(n, m)]) for n, m in zip(before, p.lens)]
        p.trim(keep)
        trim(p, keep)
        ok()
        p.same()


def test_trim_undoes_extend():
    p = Pool([5, 0, 64, 63], 16, 20, 40)
    t = p.gpu(100)
    old = {k: t[k].clone() for k in ("lens", "free", "count")}
    extend(p, [20, 33, 1, 0])
    trim(p, [5, 0, 64, 63])
    ok()
    for k, x in old.items():
        assert torch.equal(t[k], x), k


def test_many_tokens():
    # Long prompts and single tokens in one batch: several blocks share the tokens.
    new = [70000, 1, 0, 5000, 1] * 3
    p = Pool([0, 500, 3, 17, 64] * 3, 24, 4000, 12000)
    p.gpu(sum(new))
    slots = p.extend(new)
    extend(p, new)
    ok()
    p.same()
    assert p.t["slots"].tolist() == slots
    p.trim([0] * 15)
    trim(p, [0] * 15)
    ok()
    p.same()


def test_largest_batch():
    B = 16384
    p = Pool([1] * B, 4, 3, 2 * B)
    p.gpu(2 * B)
    new = [b % 3 for b in range(B)]
    slots = p.extend(new)
    extend(p, new)
    ok()
    p.same()
    assert p.t["slots"].tolist() == slots + [-1] * (2 * B - len(slots))


@pytest.mark.parametrize("n", [2 ** 31 - 2, 2 ** 31 - 5, 2 ** 31 - 100000])
def test_largest_slot_map(n):
    # Nearly 2^31 entries: the last ones are still counted in range, and nothing beside them is written.
    raw = torch.full((n + 8,), 7, dtype=torch.int32, device="cuda")
    slots = raw[4:4 + n]
    lens, table, free, count = ints([3, 5]), ints([[0, -1], [1, 2]]), ints([3]), ints([1])
    for new, status, want in (([2, 9], -8, []), ([4, 1], 0, [3, 12, 13, 14, 9])):
        slots.fill_(7)
        mva.blocks_extend(lens, ints(new), table, 4, free, count, 4, slots)
        ok(status)
        assert slots[:len(want)].tolist() == want
        for part in slots[len(want):].split(2 ** 28):
            assert (part == -1).all()
        assert (raw[:4] == 7).all() and (raw[4 + n:] == 7).all()


SHARED_MEMORY = """
import sys
sys.path.insert(0, sys.argv[1])
import torch, mla_verify_attention_gb300 as mva
ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
for B in (4010, 4011, 4074, 4075, 4095, 4096):
    lens, table, count = ints(B), ints(B, 3), ints(1) + 2 * B
    free = torch.arange(2 * B, dtype=torch.int32, device="cuda")
    for room in (2 * B, 40000):
        slots = ints(room) + 7
        mva.blocks_extend(lens, ints(B) + 2, table, 4, free, count, 2 * B, slots)
        torch.cuda.synchronize()
        b = torch.arange(B, device="cuda")
        want = (4 * (2 * B - 1 - b)[:, None] + torch.arange(2, device="cuda")).view(-1)
        assert mva.last_device_error() == 0 and (lens == 2).all() and count.item() == B
        assert torch.equal(slots[:2 * B].long(), want) and (slots[2 * B:] == -1).all()
        mva.blocks_trim(lens, ints(B), table, 4, free, count)
        torch.cuda.synchronize()
        assert mva.last_device_error() == 0 and (lens == 0).all() and count.item() == 2 * B
        assert torch.equal(free.long(), torch.arange(2 * B, device="cuda"))
"""


def test_batches_around_the_shared_memory_that_is_not_asked_for():
    # In a process of its own: a larger batch before it would have asked.
    import subprocess
    import sys
    from conftest import ROOT
    r = subprocess.run([sys.executable, "-c", SHARED_MEMORY, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("why,new,status", [
    ("pages", [10, 40, 0], -11), ("negative", [1, -1, 0], -8), ("table", [0, 0, 90], -8), ("slots", [20, 12, 0], -8)])
def test_extend_all_or_nothing(why, new, status):
    p = Pool([3, 4, 9], 4, 24, 9)
    t = p.gpu(31 if why == "slots" else 64)
    if why == "table":
        p.count = 9
    old = {k: x.clone() for k, x in t.items()}
    extend(p, new)
    ok(status)
    for k in ("lens", "table", "free", "count"):
        assert torch.equal(t[k], old[k]), k
    assert (t["slots"] == -1).all()


def test_trim_refuses_growth_and_a_full_list():
    p = Pool([30, 40], 4, 24, 9)
    t = p.gpu(4)
    old = {k: x.clone() for k, x in t.items()}
    trim(p, [31, 0])
    ok(-8)
    small = t["free"][:10].clone()
    mva.blocks_trim(t["lens"], ints([0, 0]), t["table"], 4, small, t["count"])
    ok(-11)
    for k in ("lens", "table", "free", "count"):
        assert torch.equal(t[k], old[k]), k


@pytest.mark.parametrize("room", [1000, 5000, 40000])
def test_many_streams_all_or_nothing(room):
    # One block, a cluster, two grids: every block of a call comes to the same verdict.
    B, page = 200, 4
    p = Pool([b % 9 for b in range(B)], page, 24, 600)
    t = p.gpu(room)
    old = {k: x.clone() for k, x in t.items()}
    few = [1] * B                                  # (24 * page more than the last stream's one token: no room)
    for new, status in (([-1] + few[1:], -8), (few[:-1] + [24 * page], -8), ([20] * B, -11 if room > 20 * B else -8)):
        t["slots"].fill_(7)
        extend(p, new)
        ok(status)
        for k in ("lens", "table", "free", "count"):
            assert torch.equal(t[k], old[k]), k
        assert (t["slots"] == -1).all()
    for keep in ([0] * (B - 1) + [p.lens[-1] + 1], [-1] + [0] * (B - 1)):
        trim(p, keep)
        ok(-8)
        for k in ("lens", "table", "free", "count"):
            assert torch.equal(t[k], old[k]), k


@pytest.mark.parametrize("B", [2, 3, 4, 7, 8, 16, 64, 1500])
@pytest.mark.parametrize("room", [8, 5000, 40000])
def test_more_new_tokens_than_32_bits_count(B, room):
    # 2^30 - 1 new tokens a stream in a block it already has: eight times as many are more than 2^32.
    lens, new = ints([1] * B), ints([2 ** 30 - 1] * B)
    table, free, count = ints([[0]] * B), ints([0]), ints([1])
    slots = torch.full((room,), 7, dtype=torch.int32, device="cuda")
    mva.blocks_extend(lens, new, table, 2 ** 30, free, count, 1, slots)
    ok(-8)
    assert lens.tolist() == [1] * B and count.tolist() == [1] and free.tolist() == [0]
    assert table.tolist() == [[0]] * B and (slots == -1).all()


def test_more_blocks_than_32_bits_count():
    # Four streams of 2^30 blocks each.
    table = torch.empty((4, 2 ** 30), dtype=torch.int32, device="cuda")
    lens, free, count = ints([2 ** 30] * 4), ints(list(range(9))), ints([2])
    mva.blocks_trim(lens, ints([0] * 4), table, 1, free, count)
    ok(-11)
    assert lens.tolist() == [2 ** 30] * 4 and free.tolist() == list(range(9)) and count.tolist() == [2]
    lens, slots = ints([0] * 4), torch.full((100,), 7, dtype=torch.int32, device="cuda")
    mva.blocks_extend(lens, ints([2 ** 30] * 4), table, 1, free, count, 9, slots)
    ok(-8)
    assert lens.tolist() == [0] * 4 and count.tolist() == [2] and (slots == -1).all()


@pytest.mark.parametrize("B,most", [(3000, 4), (700, 100)])
def test_streams_of_a_thread_are_read_before_they_change(B, most):
    # Several streams a thread, which every block of the call reads twice.
    rng = random.Random(B)
    p = Pool([rng.randint(0, 9) for _ in range(B)], 4, (9 + most) // 4 + 2, B * (most // 4 + 2))
    t = p.gpu(B * most)
    start = {k: t[k].clone() for k in ("lens", "free", "count")}
    new = [rng.randint(0, most) for _ in range(B)]
    new_t, keep_t = ints(new), start["lens"].clone()
    slots = p.extend(new)
    for _ in range(30):
        mva.blocks_extend(t["lens"], new_t, t["table"], 4, t["free"], t["count"], p.pages, t["slots"])
        got, lens = t["slots"].clone(), t["lens"].clone()
        mva.blocks_trim(t["lens"], keep_t, t["table"], 4, t["free"], t["count"])
        ok()
        assert got.tolist() == slots + [-1] * (B * most - len(slots)) and lens.tolist() == p.lens
        for k, x in start.items():
            assert torch.equal(t[k], x), k


@pytest.mark.parametrize("B,most,page", [(3000, 20, 4), (1500, 60, 16), (16384, 9, 3)])
def test_streams_of_a_thread_with_many_tokens(B, most, page):
    # Two grids for the extend, each with several streams a thread.
    rng = random.Random(B)
    p = Pool([rng.randint(0, 30) for _ in range(B)], page, (30 + 3 * most) // page + 2, B * (2 * most // page + 2))
    t = p.gpu(B * most + 3)
    for _ in range(2):
        before = list(p.lens)
        new = [rng.randint(0, most) for _ in range(B)]
        slots = p.extend(new)
        extend(p, new)
        ok()
        p.same()
        assert t["slots"].tolist() == slots + [-1] * (B * most + 3 - len(slots))
        keep = [rng.choice([0, n, m, rng.randint(n, m)]) for n, m in zip(before, p.lens)]
        p.trim(keep)
        trim(p, keep)
        ok()
        p.same()
    old = {k: x.clone() for k, x in t.items()}
    extend(p, [0] * (B - 1) + [10 ** 6])
    ok(-8)
    for k in ("lens", "table", "free", "count"):
        assert torch.equal(t[k], old[k]), k
    assert (t["slots"] == -1).all()


def test_bad_page_in_the_table_gives_no_slot():
    p = Pool([5, 5], 16, 4, 4)
    t = p.gpu(6)
    t["table"][1, 0] = p.pages
    extend(p, [3, 3])
    ok(-10)
    s = t["slots"].tolist()
    assert s[3:] == [-1, -1, -1] and min(s[:3]) >= 0


def test_extend_replayed_from_a_graph():
    p = Pool([5, 60, 0], 16, 30, 60)
    t = p.gpu(27)
    new = ints([9, 9, 9])
    call = lambda: mva.blocks_extend(t["lens"], new, t["table"], 16, t["free"], t["count"], p.pages, t["slots"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        slots = p.extend([9, 9, 9])
        g.replay()
        ok()
        p.same()
        assert t["slots"].tolist() == slots


# ---------------------------------------------------------------- rows

@pytest.mark.parametrize("T,rows", [(1, 1), (7, 50), (300, 4000)])
@pytest.mark.parametrize("fused", [False, True])
def test_append_latent(T, rows, fused):
    gen = torch.Generator().manual_seed(T)
    pool = torch.randn((rows, 576), generator=gen).to(BF16).cuda()
    x = torch.randn((T, 600), generator=gen).to(BF16).cuda()
    a, b = (x[:, :512], x[:, 512:576]) if fused else (x[:, :512].contiguous(), x[:, 512:576].contiguous())
    slots = torch.randperm(rows, generator=gen)[:T].to(torch.int32)
    slots[T // 2] = -1 if T > 1 else slots[0]
    want = pool.clone()
    good = slots >= 0
    want[slots[good].long().cuda()] = x[good.cuda(), :576]
    mva.cache_append(pool, a, b, slots.cuda())
    ok()
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("Hkv,D,dt", [(1, 64, FP16), (8, 128, BF16), (3, 128, FP16), (16, 256, BF16)])
def test_append_keys_and_values(Hkv, D, dt):
    gen = torch.Generator().manual_seed(D)
    T, rows = 100, 300
    qkv = torch.randn((T, 4 * Hkv, D), generator=gen).to(dt).cuda()
    k, v = qkv[:, 2 * Hkv:3 * Hkv], qkv[:, 3 * Hkv:]
    both = torch.randn((rows, 2, Hkv, D), generator=gen).to(dt).cuda()      # pools that share their rows
    want = both.clone()
    slots = torch.randperm(rows, generator=gen)[:T].to(torch.int32).cuda()
    want[slots.long(), 0], want[slots.long(), 1] = k, v
    mva.gqa_cache_append(both[:, 0], both[:, 1], k, v, slots)
    ok()
    assert torch.equal(both.view(torch.int16), want.view(torch.int16))


def test_append_reports_a_slot_past_the_pool():
    pool = torch.zeros((10, 576), dtype=BF16, device="cuda")
    x = torch.ones((3, 576), dtype=BF16, device="cuda")
    mva.cache_append(pool, x[:, :512], x[:, 512:], ints([2, 10, 4]))
    ok(-12)
    assert pool[:, 0].tolist() == [0, 0, 1, 0, 1, 0, 0, 0, 0, 0]


def test_append_far_into_a_large_pool():
    rows = 2 ** 32 // 1152 + 1000
    pool = torch.empty((rows, 576), dtype=BF16, device="cuda")
    x = torch.randn((5, 576), device="cuda").to(BF16)
    slots = [rows - 1, 0, rows - 7, 2 ** 31 // 1152 + 1, 2 ** 32 // 1152 + 2]
    mva.cache_append(pool, x[:, :512], x[:, 512:], ints(slots))
    ok()
    assert torch.equal(pool[torch.tensor(slots).cuda()], x)


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("B,q,latent", [(1, 1, True), (4, 9, True), (3, 33, False), (70, 64, False)])
def test_keep(B, q, latent, page):
    rng = random.Random(q + page)
    lens = [q + rng.randint(0, 50) for _ in range(B)]
    p = Pool(lens, page, (q + 50) // page + 2, 3)
    t = p.gpu(1)
    gen = torch.Generator().manual_seed(q)
    rows = p.pages * page
    pools = ([torch.randn((rows, 576), generator=gen).to(BF16).cuda()] if latent else
             [torch.randn((rows, 2, 64), generator=gen).to(FP16).cuda() for _ in range(2)])
    want = [x.cpu().clone() for x in pools]
    keep = [rng.randint(0, q) for _ in range(B)]
    # A tree's paths go up; any other path has to work in place as well.
    path = [sorted(rng.sample(range(q), q)) if b % 3 else [rng.randrange(q) for _ in range(q)] for b in range(B)]
    row = lambda b, i: p.table[b][(lens[b] - q + i) // page] * page + (lens[b] - q + i) % page
    for x, old in zip(want, [w.clone() for w in want]):
        for b in range(B):
            for j in range(keep[b]):
                x[row(b, j)] = old[row(b, path[b][j])]
    path_t = ints(path)
    if latent:
        mva.cache_keep(pools[0], t["table"], page, t["lens"], path_t, ints(keep))
    else:
        mva.gqa_cache_keep(pools[0], pools[1], t["table"], page, t["lens"], path_t, ints(keep))
    ok()
    for x, w in zip(pools, want):
        assert torch.equal(x.cpu().view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("B,q,heads,D", [
    (400, 9, 0, 0),            # latent rows, three columns
    (130, 16, 8, 128),
    (130, 17, 8, 128),
    (130, 40, 8, 128),
    (130, 41, 8, 128),
    (200, 64, 5, 72),          # rows of 45 units
])
def test_keep_of_many_streams(B, q, heads, D):
    # More blocks than fit the device at once, every number of rows a warp.
    page = 16
    gen = torch.Generator().manual_seed(q)
    lens = torch.randint(q, q + 40, (B,), generator=gen)
    blocks = (q + 40) // page + 1
    table = torch.randperm(B * blocks, generator=gen).view(B, blocks)
    path, keep = torch.randint(0, q, (B, q), generator=gen), torch.randint(0, q + 1, (B,), generator=gen)
    rows = B * blocks * page
    row = lambda i: table.gather(1, (lens[:, None] - q + i) // page) * page + (lens[:, None] - q + i) % page
    kept = torch.arange(q)[None, :] < keep[:, None]
    src, dst = row(path)[kept], row(torch.arange(q).expand(B, q))[kept]
    shape = (rows, 576) if heads == 0 else (rows, heads, D)
    pools = [torch.randn(shape, generator=gen).to(BF16) for _ in range(1 if heads == 0 else 2)]
    want = [x.index_copy(0, dst, x[src]) for x in pools]
    got = [x.cuda() for x in pools]
    call = mva.cache_keep if heads == 0 else mva.gqa_cache_keep
    ints32 = lambda x: x.to(torch.int32).cuda()
    call(*got, ints32(table), page, ints32(lens), ints32(path), ints32(keep))
    ok()
    for x, w in zip(got, want):
        assert torch.equal(x.cpu().view(torch.int16), w.view(torch.int16))


def test_keep_leaves_a_wrong_stream_as_it_was():
    page, q = 4, 3
    for what, status in (("path", -12), ("count", -12), ("length", -8), ("page", -10)):
        p = Pool([10, 10], page, 3, 2)
        t = p.gpu(1)
        pool = torch.randn((p.pages * page, 576), device="cuda").to(BF16)
        old = pool.clone()
        path, keep = [[1, 2, 0], [1, 2, 0]], [2, 2]
        if what == "path":
            path[0][1] = 3
        elif what == "count":
            keep[0] = 4
        elif what == "length":
            t["lens"][0] = 2
        else:
            t["table"][0, 1] = p.pages
        mva.cache_keep(pool, t["table"], page, t["lens"], ints(path), ints(keep))
        ok(status)
        row = lambda i: p.table[1][(7 + i) // page] * page + (7 + i) % page
        want = old.clone()
        want[row(0)], want[row(1)] = old[row(1)], old[row(2)]
        assert torch.equal(pool, want), what


def test_refusals():
    p = Pool([10, 10], 4, 3, 2)
    t = p.gpu(8)
    pool = torch.zeros((p.pages * 4, 576), dtype=BF16, device="cuda")
    x = torch.zeros((8, 576), dtype=BF16, device="cuda")
    for bad in (lambda: mva.cache_append(pool, x[:, :512], x[:, 512:], t["slots"].long()),
                lambda: mva.cache_append(pool, x[:, :512], x[:, 500:564].half(), t["slots"]),
                lambda: mva.cache_append(pool, x[:, :511], x[:, 512:], t["slots"]),
                lambda: mva.cache_append(pool, x[:4, :512], x[:, 512:], t["slots"]),
                lambda: mva.cache_append(pool.float(), x[:, :512], x[:, 512:], t["slots"]),
                lambda: mva.cache_append(pool, x.t().contiguous().t()[:, :512], x[:, 512:], t["slots"]),
                lambda: mva.blocks_extend(t["lens"], t["lens"][:1], t["table"], 4, t["free"], t["count"], p.pages, t["slots"]),
                lambda: mva.blocks_extend(t["lens"].cpu(), t["lens"], t["table"], 4, t["free"], t["count"], p.pages, t["slots"]),
                lambda: mva.blocks_trim(t["lens"], t["lens"].float(), t["table"], 4, t["free"], t["count"]),
                lambda: mva.cache_keep(pool, t["table"], 4, t["lens"], ints([0, 1]), ints([1, 1]))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mva.blocks_extend(t["lens"], t["lens"], t["table"], 0, t["free"], t["count"], p.pages, t["slots"]),
                lambda: mva.blocks_extend(t["lens"], t["lens"], t["table"], 4, t["free"], t["count"], 0, t["slots"]),
                lambda: mva.blocks_extend(t["lens"], t["lens"], t["table"], 4, t["free"], t["count"], p.pages, t["slots"][1:]),
                lambda: mva.cache_append(pool, x[:, 4:516], x[:, 512:], t["slots"]),
                lambda: mva.cache_keep(pool, t["table"], 4, t["lens"], torch.zeros((2, 65), dtype=torch.int32, device="cuda"), ints([1, 1]))):
        with pytest.raises(mva.MLAError):
            bad()
    ok()


# ---------------------------------------------------------------- whole steps

def step_trees(rng, B, q):
    parents = [[-1] + [rng.randrange(i) for i in range(1, q)] for _ in range(B)]
    seen = torch.zeros((B, q, q), dtype=torch.bool)
    for b in range(B):
        for i in range(q):
            if i:
                seen[b, i] = seen[b, parents[b][i]]
            seen[b, i, i] = True
    return parents, seen


def accepted(rng, parents, q):
    """A random root-to-node path of each tree."""
    path, keep = [], []
    for par in parents:
        i, way = rng.randrange(q), []
        while i >= 0:
            way.append(i)
            i = par[i]
        way = way[::-1]
        path.append(way + [-1] * (q - len(way)))
        keep.append(len(way))
    return path, keep


@pytest.mark.parametrize("page", [64, 16, 5])
def test_verify_steps_with_keys_and_values(page):
    """Four steps of extend, append, attend, keep, trim; the caches that the
    operators keep equal plain lists of rows at every step."""
    B, q, H, Hkv, D, dt = 3, 9, 8, 2, 64, BF16
    rng, gen = random.Random(page), torch.Generator().manual_seed(page)
    rand = lambda *s: torch.randn(s, generator=gen).to(dt).cuda()
    p = Pool([0] * B, page, 400 // page + 2, 3 * (400 // page + 2))
    t = p.gpu(400)
    pools = [torch.full((p.pages * page, Hkv, D), float("nan"), dtype=dt, device="cuda") for _ in range(2)]
    held = [[torch.empty((0, Hkv, D), dtype=dt, device="cuda") for _ in range(2)] for _ in range(B)]

    def grow(new):
        T = sum(new) + 3                                     # padding tokens behind the batch
        slots = torch.empty(T, dtype=torch.int32, device="cuda")
        mva.blocks_extend(t["lens"], ints(new), t["table"], page, t["free"], t["count"], p.pages, slots)
        k, v = rand(T, Hkv, D), rand(T, Hkv, D)
        mva.gqa_cache_append(pools[0], pools[1], k, v, slots)
        at = 0
        for b, n in enumerate(new):
            held[b] = [torch.cat([x, y[at:at + n]]) for x, y in zip(held[b], (k, v))]
            at += n

    grow([100, 1, 37])                                       # the prompts
    for _ in range(4):
        parents, seen = step_trees(rng, B, q)
        grow([q] * B)
        lens = [x[0].shape[0] for x in held]
        query = rand(B, q, H, D)
        out, lse = mva.gqa_verify_attn_paged(query, pools[0], pools[1], t["table"], page, t["lens"],
                                             plain.mask_words(seen).cuda(), 1 / math.sqrt(D))
        path, keep = accepted(rng, parents, q)
        mva.gqa_cache_keep(pools[0], pools[1], t["table"], page, t["lens"], ints(path), ints(keep))
        mva.blocks_trim(t["lens"], ints([n - q + k for n, k in zip(lens, keep)]), t["table"], page, t["free"], t["count"])
        ok()
        plain.check(out, lse, query, lambda b: held[b][0], lambda b: held[b][1], lens, seen, 1 / math.sqrt(D))
        for b in range(B):
            way = [lens[b] - q + i for i in path[b][:keep[b]]]
            held[b] = [torch.cat([x[:lens[b] - q], x[way]]) for x in held[b]]
        assert t["lens"].tolist() == [x[0].shape[0] for x in held]
    pos = t["lens"].tolist()
    table = t["table"].long()
    for b in range(B):
        at = torch.arange(pos[b], device="cuda")
        rows = table[b][at // page] * page + at % page
        for pool, x in zip(pools, held[b]):
            assert torch.equal(pool[rows], x)
    assert t["count"].item() == p.pages - sum(-(-n // page) for n in pos)


@pytest.mark.parametrize("page", [64, 16])
def test_verify_step_with_the_latent_cache(page):
    """The same around verify_attn_paged, held to its formula in 64 bits."""
    B, q, H = 2, 9, 8
    rng, gen = random.Random(page), torch.Generator().manual_seed(page)
    rand = lambda *s: torch.randn(s, generator=gen).to(BF16).cuda()
    p = Pool([0] * B, page, 512 // page, 2 * (512 // page))
    t = p.gpu(1)
    pool = torch.full((p.pages * page, 576), float("nan"), dtype=BF16, device="cuda")
    held = [torch.empty((0, 576), dtype=BF16, device="cuda") for _ in range(B)]

    def grow(new):
        slots = torch.empty(sum(new), dtype=torch.int32, device="cuda")
        mva.blocks_extend(t["lens"], ints(new), t["table"], page, t["free"], t["count"], p.pages, slots)
        x = rand(sum(new), 576)
        mva.cache_append(pool, x[:, :512], x[:, 512:], slots)
        at = 0
        for b, n in enumerate(new):
            held[b] = torch.cat([held[b], x[at:at + n]])
            at += n

    grow([200, 77])
    for _ in range(3):
        parents, seen = step_trees(rng, B, q)
        grow([q] * B)
        lens = [x.shape[0] for x in held]
        qn, qr = rand(B, q, H, 512), rand(B, q, H, 64)
        mask = plain.mask_words(seen).cuda()
        out, lse = mva.verify_attn_paged(qn, qr, pool, t["table"], page, t["lens"], mask, 192 ** -0.5)
        path, keep = accepted(rng, parents, q)
        mva.cache_keep(pool, t["table"], page, t["lens"], ints(path), ints(keep))
        mva.blocks_trim(t["lens"], ints([n - q + k for n, k in zip(lens, keep)]), t["table"], page, t["free"], t["count"])
        ok()
        for b in range(B):
            kv = held[b].double()
            s = (qn[b].double() @ kv[:, :512].t() + qr[b].double() @ kv[:, 512:].t()) * 192 ** -0.5
            see = torch.ones((q, lens[b]), dtype=torch.bool, device="cuda")
            see[:, lens[b] - q:] = seen[b].cuda()
            s = s.masked_fill(~see[:, None], -math.inf)
            assert ((s.softmax(-1) @ kv[:, :512]) - out[b]).abs().max() <= 2e-3
            assert (s.logsumexp(-1) - lse[b]).abs().max() <= 1e-3
            way = [lens[b] - q + i for i in path[b][:keep[b]]]
            held[b] = torch.cat([held[b][:lens[b] - q], held[b][way]])
        assert t["lens"].tolist() == [x.shape[0] for x in held]
