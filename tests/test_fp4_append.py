"""Rows into a cache held in 4 bits, on the GPU: every byte against the plain
form, values halfway between codes, groups of zeros, infinities and NaN, strided
rows, skipped tokens and refusals; the drafts' rows that move together."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import long_cache_plain as plain

BF16, FP16 = torch.bfloat16, torch.float16


def pools(rows, Hkv, D):
    n = mva.gqa_fp4_row_bytes(Hkv, D)
    return [torch.randint(0, 256, (rows, n), dtype=torch.uint8, device="cuda") for _ in range(2)]


def check(k, v, slots, rows=None, k_scale=1.0, v_scale=1.0):
    T, Hkv, D = k.shape
    rows = rows or 2 * T + 3
    got = pools(rows, Hkv, D)
    want = [p.cpu().clone() for p in got]
    held = [torch.full((T, Hkv, D), 77.0, dtype=k.dtype, device="cuda") for _ in range(2)]
    want_held = [h.cpu().clone() for h in held]
    mva.gqa_cache_append_fp4(*got, k, v, slots.cuda(), k_scale, v_scale, *held)
    st = mva.last_device_error()
    assert st == 0, mva.strerror(st)
    used = Hkv * D // 2 + Hkv * D // 16
    ok = slots >= 0
    for p, w, h, wh, x, f in zip(got, want, held, want_held, (k, v), (k_scale, v_scale)):
        packed = plain.pack_fp4(x.cpu(), f)
        w[slots[ok].long(), :used] = packed[ok]
        bad = (p.cpu() != w).nonzero()
        assert len(bad) == 0, "%d bytes, the first %s" % (len(bad), bad[0].tolist())
        wh[ok] = plain.unpack_fp4(packed, Hkv, D, f)[ok].to(x.dtype)
        assert torch.equal(h.cpu().nan_to_num(nan=1e4), wh.nan_to_num(nan=1e4))


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hkv", [(1, 1), (3, 2), (72, 8), (501, 3), (17, 5), (9, 40)])
def test_bytes(T, Hkv, D, dt):
    gen = torch.Generator().manual_seed(T + Hkv)
    k, v = ((torch.randn((T, Hkv, D), generator=gen) * torch.exp(3 * torch.randn((T, Hkv, 1), generator=gen))).to(dt).cuda()
            for _ in range(2))
    slots = torch.randperm(2 * T + 3, generator=gen)[:T].int()
    slots[T // 2::7] = -1
    check(k, v, slots, None, 0.125, 1.0)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("factor", [1.0, 2.0 ** -7, 2.0 ** 10])
def test_values_between_codes_and_steps_between_steps(dt, factor):
    # Each group: its largest value on or beside a border of two steps, the others on
    # and beside every border of two codes.
    steps = plain.e4m3_values()
    groups = []
    for i in range(1, 127):
        for top in (6 * steps[i], 3 * (steps[i] + steps[i - 1])):
            d = steps[i]
            x = [top] + [b * d for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0)]
            groups.append(x)
            groups.append([y * (1 + 2.0 ** -7) for y in x])
            groups.append([y * (1 - 2.0 ** -7) for y in x])
    x = (torch.tensor(groups, dtype=torch.float64) * factor).to(dt)
    x = torch.cat([x, x[:(-len(x)) % 8]]).view(-1, 2, 64).cuda()
    check(x, -x, torch.arange(len(x)).int(), None, factor, factor)


@pytest.mark.parametrize("dt", [BF16, FP16])
def test_odd_values(dt):
    x = torch.randn((24, 1, 64), generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1] = -0.0
    x[2, 0, 5], x[3, 0, 17], x[4, 0, 33] = float("nan"), float("inf"), -float("inf")
    x[5, 0, 3], x[5, 0, 4] = float("inf"), float("nan")
    x[6] = 6e-8                                     # fp16's smallest
    x[7] = torch.finfo(dt).max
    x[8] = torch.finfo(dt).tiny
    x[9, 0, :16] = 2.0 ** -9 * 6 * 0.5              # the smallest step, halved: a tie with none
    x[10, 0, :16] = 2.0 ** -9 * 6 * 0.51
    x[11] = 3000.0                                  # above the largest step's reach
    x[12] = 2688.0 * 1.03
    x = x.to(dt).cuda()
    check(x, x.flip(0), torch.arange(24).int())
    check(x, x.flip(0), torch.arange(24).int(), None, 2.0 ** -30, 2.0 ** 30)


def test_factors_that_are_no_powers_of_two():
    gen = torch.Generator().manual_seed(5)
    for f in (0.1, 3.7, 1e-3):
        x = torch.randn((300, 2, 64), generator=gen).to(BF16).cuda()
        check(x, 5 * x, torch.arange(300).int(), None, f, 2 * f)


def test_rows_cut_out_of_wider_ones_and_another_stream():
    gen = torch.Generator().manual_seed(2)
    fused = torch.randn((40, 12, 128), generator=gen).to(BF16).cuda()
    wide = torch.zeros((90, 2, 1024), dtype=torch.uint8, device="cuda")
    n = mva.gqa_fp4_row_bytes(3, 128)
    slots = torch.randperm(90, generator=gen)[:40].int()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mva.gqa_cache_append_fp4(wide[:, 0, :n], wide[:, 1, :n], fused[:, 4:7], fused[:, 8:11], slots.cuda(), 0.25, 0.5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for i, (x, f) in enumerate(((fused[:, 4:7], 0.25), (fused[:, 8:11], 0.5))):
        want = torch.zeros((90, 1024), dtype=torch.uint8)
        packed = plain.pack_fp4(x.cpu(), f)
        want[slots.long(), :packed.shape[1]] = packed
        assert torch.equal(wide[:, i].cpu(), want)


def test_slots_out_of_range_are_reported():
    x = torch.ones((3, 1, 64), dtype=BF16, device="cuda")
    p = pools(4, 1, 64)
    before = [y.clone() for y in p]
    mva.gqa_cache_append_fp4(*p, x, x, torch.tensor([4, -1, 1 << 30], dtype=torch.int32).cuda())
    assert mva.last_device_error() == -12
    assert all(torch.equal(a, b) for a, b in zip(p, before))


def test_no_tokens():
    x = torch.ones((0, 2, 64), dtype=BF16, device="cuda")
    mva.gqa_cache_append_fp4(*pools(4, 2, 64), x, x, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert mva.last_device_error() == 0


def test_kept_drafts_move_together():
    # Rows of 4 bits move as bytes, padding (of an odd number of heads) and all.
    B, q, page = 3, 9, 16
    lens = [40, 9, 300]
    table, total = plain.pages(torch.Generator().manual_seed(0), lens, page)
    p = pools(total * page, 3, 64)
    want = [x.cpu().clone() for x in p]
    path = torch.stack([torch.randperm(q, generator=torch.Generator().manual_seed(b)).sort().values for b in range(B)]).int()
    path[0, :4] = torch.tensor([0, 2, 5, 8])
    keep = torch.tensor([4, 0, 9], dtype=torch.int32)
    mva.gqa_cache_keep_fp4(*p, table.cuda(), page, torch.tensor(lens, dtype=torch.int32).cuda(), path.cuda(), keep.cuda())
    assert mva.last_device_error() == 0
    for x, w in zip(p, want):
        old = w.clone()
        for b, n in enumerate(lens):
            rows = plain.rows_of(table[b], page, n)
            for j in range(int(keep[b])):
                w[rows[n - q + j]] = old[rows[n - q + int(path[b, j])]]
        assert torch.equal(x.cpu(), w)


def test_refusals():
    p, x, slots = pools(10, 2, 64), torch.ones((3, 2, 64), dtype=BF16, device="cuda"), torch.arange(3).int().cuda()
    call = mva.gqa_cache_append_fp4
    for args in ((p[0][:, :64], p[1][:, :64], x, x, slots), (p[0], p[1], x.float(), x.float(), slots),
                 (p[0].view(torch.int8), p[1], x, x, slots), (p[0], p[1], x, x[:2], slots), (p[0], p[1], x, x, slots[:2]),
                 (p[0], p[1], x, x, slots.long()), (p[0], p[1], x[..., :32], x[..., :32], slots)):
        with pytest.raises(ValueError):
            call(*args)
    with pytest.raises(ValueError):
        call(p[0], p[1], x, x, slots, k_held=x.half())
    for f in (0.0, -1.0, float("nan"), float("inf"), 1e-30, 1e30):
        for kw in (dict(k_scale=f), dict(v_scale=f)):
            with pytest.raises(mva.MLAError) as e:
                call(p[0], p[1], x, x, slots, **kw)
            assert e.value.status == -9


def allowed(x, factor, step_codes, codes):
    """Whether steps and codes are what the definition says of groups x [n,16]: the nearest to quotients in 64 bits,
    either of two neighbours where a quotient is within 2^-22 of the middle between them."""
    f, t = torch.tensor(factor, dtype=torch.float32).double(), 2.0 ** -22
    steps, levels = plain.e4m3_values(), torch.tensor(plain.LEVELS, dtype=torch.float64)
    z = x.double().abs().amax(-1) / (6 * f)
    ok = torch.zeros_like(z, dtype=torch.bool)
    for e in (1 - t, 1.0, 1 + t):
        ok |= plain.nearest_even(z * e, steps) == step_codes
    d = (steps[step_codes] * f)[:, None]
    z = torch.where(d > 0, x.double().abs() / d, 0.0)
    right = torch.zeros_like(z, dtype=torch.bool)
    for e in (1 - t, 1.0, 1 + t):
        right |= plain.nearest_even(z * e, levels) == (codes & 7)
    sign = (codes >> 3 == torch.signbit(x)) | (d == 0) | (x == 0)
    return ok, right & sign


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("factor", [0.1, 3.7, 1 - 2.0 ** -24, 1 + 2.0 ** -23, 1.5 - 2.0 ** -23, 1.0 / 3, 1.0 / 2688, 0.7853981852531433, 2.0 ** -7])
def test_borders_with_any_factor(dt, factor):
    # The values of the type nearest to every border of two steps, and of two codes at every step, and their neighbours.
    f = torch.tensor(factor, dtype=torch.float32).double()
    steps = plain.e4m3_values()[1:]
    least = torch.finfo(dt).tiny
    one = torch.tensor(1, dtype=torch.int16)
    near = lambda y: (y.to(dt).view(torch.int16) + torch.arange(-2, 3, dtype=torch.int16)[:, None] * one).view(dt)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    groups = []
    tops = torch.cat([6 * f * steps, 6 * f * (steps[1:] + steps[:-1]) / 2, 3 * f * steps[:1]])
    for i, top in enumerate(near(tops[tops >= 4 * least]).flatten()):
        g = torch.zeros(16, dtype=dt)
        g[0] = top
        groups.append(g)
    for s in steps:
        d = s * f
        for y in near((borders * d)).view(5, 7):
            g = torch.zeros(16, dtype=dt)
            g[0] = (6 * d).to(dt)
            g[1:8], g[8:15] = y, -y
            groups.append(g)
    x = torch.stack(groups)
    x = x[(x.abs().double() >= least).any(-1) & torch.isfinite(x).all(-1)]
    x = torch.cat([x, x[:(-len(x)) % 8]])
    rows = x.view(-1, 2, 64)
    p = pools(len(rows), 2, 64)
    mva.gqa_cache_append_fp4(*p, rows.cuda(), (-rows).cuda(), torch.arange(len(rows)).int().cuda(), factor, factor)
    assert mva.last_device_error() == 0
    for pool, y in zip(p, (x, -x)):
        got = pool.cpu().long()
        codes = torch.stack([got[:, :64] & 15, got[:, :64] >> 4], -1).view(-1, 16)
        ok, right = allowed(y, factor, got[:, 64:72].reshape(-1), codes)
        assert ok.all(), "step of %s" % y[~ok][0].tolist()
        assert right.all(), "codes of %s" % y[~right.all(-1)][0].tolist()
    check(rows.cuda(), (-rows).cuda(), torch.arange(len(rows)).int(), None, factor, factor)
