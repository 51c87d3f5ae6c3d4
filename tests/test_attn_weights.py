"""The attention weight that each key got, on the GPU against its plain 64-bit
form: types, head layouts, row counts over several chunks, lengths around tile
edges, masks, rows left out, pages of every kind, streams, graphs and refusals."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import gqa_plain
import long_cache_plain as plain
from test_gqa_attn import trees

BF16, FP16 = torch.bfloat16, torch.float16


def case(q, H, Hkv, D, lens, dt=BF16, tree="random", smax=None, seed=0, scale=None):
    gen = torch.Generator().manual_seed(seed + 13 * q + D)
    B, smax = len(lens), smax or max(max(lens), 1)
    c = dict(q=torch.randn((B, q, H, D), generator=gen).to(dt).cuda(), k=torch.randn((B, smax, Hkv, D), generator=gen).to(dt).cuda(),
             lens=lens, seen=trees(gen, B, q, tree), scale=1 / math.sqrt(D) if scale is None else scale, gen=gen,
             w=torch.rand((B, Hkv, smax), generator=gen).cuda())
    c["lens_t"] = torch.tensor(lens, dtype=torch.int32).cuda()
    c["mask"] = gqa_plain.mask_words(c["seen"]).cuda()
    c["lse"] = torch.empty((B, q, H), device="cuda")
    for b, n in enumerate(lens):
        c["lse"][b] = plain.attend(c["q"][b], c["k"][b, :n], c["k"][b, :n], plain.seen_keys(c["seen"][b], n) if n else
                                   torch.zeros((q, 0)).bool(), c["scale"])[1].float()
        c["k"][b, n:] = float("nan")
    return c


def verify(c, got):
    B, q, H, D = c["q"].shape
    Hkv = c["k"].shape[2]
    for b, n in enumerate(c["lens"]):
        old = c["w"][b].double()
        assert torch.equal(got[b, :, n:], c["w"][b, :, n:])
        if n == 0:
            continue
        see = plain.seen_keys(c["seen"][b], n).cuda()
        lse = c["lse"][b].double().view(q, Hkv, H // Hkv)
        adds = torch.isfinite(lse)
        qd = torch.where(adds[..., None], c["q"][b].double().view(q, Hkv, H // Hkv, D), 0.0)
        k = torch.where(see.any(0)[:, None, None], c["k"][b, :n].double(), 0.0)
        s = torch.einsum("ihgd,thd->ihgt", qd, k) * c["scale"]
        size = torch.einsum("ihgd,thd->ihgt", qd.abs(), k.abs()) * abs(c["scale"])
        x = torch.where(adds, lse, 0.0)[..., None]
        ok = see[:, None, None] & adds[..., None]
        w = torch.where(ok, (s - x).exp(), 0.0)
        # As for the attention: D products in fp32, scaling, lse in log2 units (2^-24 of it,
        # twice), ex2's 2^-22; then q_len * G sums in fp32, and one with what was there.
        e = (D + 4) * 2.0 ** -24 * size + 2.0 ** -22 + 2.0 ** -23 * (x.abs() + s.abs())
        rows = q * (H // Hkv)
        bound = (w * (e * 1.01 + rows * 2.0 ** -24)).sum((0, 2)) + 2.0 ** -24 * (w.sum((0, 2)) + old[:, :n]) + rows * 2.0 ** -126
        off = (got[b, :, :n].double() - old[:, :n] - w.sum((0, 2))).abs()
        assert (off <= bound).all(), "stream %d: off by %.3g, %.3g times its bound" % (b, off.max(), (off / bound).max())


def run(c, **kw):
    w = c["w"].clone()
    mva.gqa_attn_weights(c["q"], c["k"], c["lens_t"], c["mask"], c["lse"], c["scale"], w, **kw)
    torch.cuda.synchronize()
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    return w


def run_paged(c, page):
    table, total = plain.pages(c["gen"], c["lens"], page)
    B, smax, Hkv, D = c["k"].shape
    pool = torch.full((total * page, Hkv, D), float("nan"), dtype=c["k"].dtype, device="cuda")
    w = torch.full((B, Hkv, table.shape[1] * page), -3.0, device="cuda")
    for b, n in enumerate(c["lens"]):
        pool[plain.rows_of(table[b], page, n).cuda()] = c["k"][b, :n]
        w[b, :, :n] = c["w"][b, :, :n]
    mva.gqa_attn_weights_paged(c["q"], pool, table.cuda(), page, c["lens_t"], c["mask"], c["lse"], c["scale"], w)
    torch.cuda.synchronize()
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    got = c["w"].clone()
    for b, n in enumerate(c["lens"]):
        assert (w[b, :, n:] == -3.0).all()
        got[b, :, :n] = w[b, :, :n]
    return got


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,H,Hkv,lens", [
    (1, 1, 1, [1]),
    (1, 8, 1, [64]),
    (1, 64, 8, [128, 129, 1]),
    (9, 64, 8, [265, 9, 3000]),                # 72 rows
    (5, 6, 2, [63, 0, 130]),
    (16, 8, 1, [16, 700]),                     # 128 rows exactly
    (17, 8, 1, [17, 500]),                     # 136: two chunks
    (33, 16, 4, [2000]),
    (64, 14, 1, [64, 1000]),                   # 896 rows
    (2, 3, 3, [2, 65, 127, 191, 192, 193, 257]),
    (1, 128, 1, [300]),
    (3, 100, 1, [900]),                        # 300 rows, heads that no chunk divides
])
def test_matches_plain(q, H, Hkv, lens, D, dt):
    c = case(q, H, Hkv, D, lens, dt)
    a = run(c)
    verify(c, a)
    b = run(c)
    assert torch.equal(a, b)


@pytest.mark.parametrize("tree", ["chain", "any"])
@pytest.mark.parametrize("q,G,lens", [(9, 8, [9, 70]), (40, 2, [41, 130]), (64, 4, [64, 129]), (64, 1, [127, 64])])
def test_masks(q, G, lens, tree):
    c = case(q, 2 * G, 2, 64, lens, tree=tree)
    verify(c, run(c))


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 64, 100, 128])
def test_pages(page):
    for D, dt in ((64, FP16), (128, BF16)):
        c = case(5, 16, 2, D, [1500, 5, 700, 64, 0, 4000], dt)
        verify(c, run_paged(c, page))


def test_rows_add_up_to_one():
    c = case(9, 32, 4, 128, [3000, 100])
    c["w"].zero_()
    total = run(c)
    for b, n in enumerate(c["lens"]):
        assert torch.allclose(total[b, :, :n].sum(-1), torch.full((4,), 72.0, device="cuda"), rtol=1e-5)


@pytest.mark.parametrize("out", [float("inf"), -float("inf")])
def test_rows_left_out(out):
    # Drafts that were not accepted, and a batch padded to one q_len: whatever their q and their rows of k hold.
    c = case(9, 16, 2, 128, [300, 40])
    c["lse"][0, 4:] = out
    c["lse"][1, 2, 3] = out
    c["q"][0, 4:] = float("nan")
    c["seen"][0, :, 4:] = False
    c["mask"] = gqa_plain.mask_words(c["seen"]).cuda()
    c["k"][0, 295:300] = float("nan")
    verify(c, run(c))


def test_extreme_scores():
    for scale in (0.0, -0.3, 5.0):
        c = case(5, 8, 2, 64, [200, 77], scale=scale)
        verify(c, run(c))


def test_many_streams_and_long_ones():
    gen = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(5, 900, (400,), generator=gen)]
    c = case(5, 8, 2, 64, lens)
    a = run(c)
    verify(c, a)
    for page in (16, 3):
        assert torch.equal(run_paged(c, page), a)
    c = case(1, 16, 2, 128, [40000, 3, 20000])
    verify(c, run(c))


def test_strided_views_and_another_stream():
    c = case(9, 16, 2, 128, [3000, 700])
    fused = torch.randn((2, 3000, 8, 128), device="cuda").to(BF16)
    fused[:, :, 5:7] = c["k"]
    wide = torch.randn((2, 9, 32, 128), device="cuda").to(BF16)
    wide[:, :, 4:20] = c["q"]
    want, got = run(c), c["w"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mva.gqa_attn_weights(wide[:, :, 4:20], fused[:, :, 5:7], c["lens_t"], c["mask"], c["lse"], c["scale"], got, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_steps_behind_each_other_and_in_a_graph():
    # Attend, then add what the keys got, twice; then the same as a graph.
    c = case(4, 16, 2, 128, [1000, 300])
    v = torch.randn_like(c["k"].nan_to_num(0.0))
    out, lse, ws = torch.empty_like(c["q"]), torch.empty_like(c["lse"]), torch.empty(
        mva.gqa_workspace_size(2, 4, 16, 2, 128), dtype=torch.uint8, device="cuda")
    w = torch.zeros_like(c["w"])

    def step():
        mva.gqa_verify_attn(c["q"], c["k"], v, c["lens_t"], c["mask"], c["scale"], out=out, lse=lse, workspace=ws)
        mva.gqa_attn_weights(c["q"], c["k"], c["lens_t"], c["mask"], lse, c["scale"], w)

    step()
    c["w"], c["lse"] = torch.zeros_like(w), lse.clone()
    verify(c, w)
    once = w.clone()
    step()
    c["w"] = once
    verify(c, w)
    twice = w.clone()
    w.copy_(once)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    w.copy_(once)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, twice) and mva.last_device_error() == 0


def test_a_wait_that_runs_out_is_reported():
    c = case(9, 16, 2, 128, [3000])
    with mva.forced(stall=True):
        mva.gqa_attn_weights(c["q"], c["k"], c["lens_t"], c["mask"], c["lse"], c["scale"], c["w"].clone())
        assert mva.last_device_error() == -7
    verify(c, run(c))


def test_refusals():
    c = case(2, 4, 2, 64, [100])
    call = lambda **kw: mva.gqa_attn_weights(*[kw.get(n, c[n]) for n in ("q", "k", "lens_t", "mask", "lse", "scale", "w")])
    for bad in (dict(q=c["q"].float()), dict(k=c["k"].half()), dict(lens_t=c["lens_t"].long()), dict(mask=c["mask"][:, :1]),
                dict(lse=c["lse"].double()), dict(lse=c["lse"][:, :1]), dict(w=c["w"][:, :, :50]), dict(w=c["w"].half())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(mva.MLAError) as e:
        call(scale=float("nan"))
    assert e.value.status == -9
    call(lens_t=torch.tensor([101], dtype=torch.int32).cuda())
    assert mva.last_device_error() == -8
    before = c["w"].clone()
    call(lens_t=torch.tensor([1], dtype=torch.int32).cuda())
    assert mva.last_device_error() == -8 and torch.equal(before, c["w"])
    pool, table = c["k"].view(100, 2, 64), torch.tensor([[7]], dtype=torch.int32).cuda()
    mva.gqa_attn_weights_paged(c["q"], pool, table, 100, c["lens_t"], c["mask"], c["lse"], c["scale"], c["w"])
    assert mva.last_device_error() == -10


@pytest.mark.parametrize("out", [float("inf"), -float("inf")])
@pytest.mark.parametrize("q,H,Hkv,D,dt", [(9, 16, 2, 128, BF16), (2, 2, 1, 64, FP16), (17, 8, 1, 128, FP16), (64, 8, 2, 64, BF16)])
def test_rows_left_out_see_keys_that_are_not_finite(q, H, Hkv, D, dt, out):
    # A batch padded to one q_len: the padding's drafts see themselves and their ancestors, their rows of k hold
    # anything, and their lse leaves them out.  The sums are those over finite rows, bit by bit.
    accepted = max(q // 3, 1)
    c = case(q, H, Hkv, D, [300, q, 64 + q, 1000], dt)
    c["lse"][:, accepted:] = out
    want = run(c)
    for b, n in enumerate(c["lens"]):
        at = n - q + accepted
        assert torch.equal(want[b, :, at:], c["w"][b, :, at:])
        c["k"][b, at:n] = float("nan")
        c["k"][b, n - 1] = float("inf")
    assert torch.equal(run(c), want)


@pytest.mark.parametrize("q,G", [(1, 1), (3, 8), (9, 8), (17, 8)])
def test_keys_of_minus_infinity(q, G):
    # A key whose score is -inf for every row gets nothing, with rows that fill no sixteen and rows left out beside them.
    c = case(q, 2 * G, 2, 64, [300, 65 + q])
    c["q"][..., 0] = c["q"][..., 0].abs() + 0.1
    keys = [0, 17, 64]
    for b, n in enumerate(c["lens"]):
        c["k"][b, keys, :, 0] = -float("inf")
        see = plain.seen_keys(c["seen"][b], n)
        c["lse"][b] = plain.attend(c["q"][b], c["k"][b, :n], c["k"][b, :n], see, c["scale"])[1].float()
    c["lse"][0, q // 2] = float("inf")
    got = run(c)
    assert torch.equal(got[:, :, keys], c["w"][:, :, keys])
    for b, n in enumerate(c["lens"]):                  # the others as without those keys
        c["k"][b, keys] = 0.0
    rest = run(c)
    at = [t for t in range(c["k"].shape[1]) if t not in keys]
    assert torch.isfinite(got[0, :, :300]).all() and torch.equal(got[:, :, at], rest[:, :, at])
