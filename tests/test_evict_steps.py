"""Verify steps of a serving loop that keeps the weight of every key, on the GPU: extend,
append, attend, add the weights of the accepted drafts' rows, move the accepted rows and
their sums together, trim; now and then evict.  Rows, lengths and sums are held against a
plain 64-bit model of the same steps."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
import gqa_plain
import long_cache_plain as plain
from test_gqa_attn import trees

BF16 = torch.bfloat16
i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()


def accepted_path(seen, gen):
    """A random draft's ancestors and itself: what a verify step accepts."""
    last = int(torch.randint(0, seen.shape[0], (1,), generator=gen))
    return seen[last].nonzero()[:, 0]


@pytest.mark.parametrize("how", ["keep", "compact"])
@pytest.mark.parametrize("q,H,Hkv,D,page,first", [(5, 8, 2, 64, 16, [60, 1, 130]), (9, 16, 4, 128, 7, [300, 40, 2])])
def test_sums_go_with_their_keys(q, H, Hkv, D, page, first, how):
    gen = torch.Generator().manual_seed(q)
    B, blocks, pages, steps, budget = len(first), -(-600 // page), 4 * -(-600 // page), 6, 100
    smax, scale = blocks * page, D ** -0.5
    k_pool, v_pool = (torch.zeros((pages * page, Hkv, D), dtype=BF16, device="cuda") for _ in range(2))
    seq, table = i32([0] * B), torch.zeros((B, blocks), dtype=torch.int32, device="cuda")
    free, count = torch.randperm(pages, generator=gen).int().cuda(), i32([pages])
    weights = torch.zeros((B, Hkv, smax), device="cuda")
    kept, keep = torch.empty((B, smax), dtype=torch.int32, device="cuda"), i32([0] * B)
    model = [dict(k=torch.zeros((0, Hkv, D), dtype=BF16), v=torch.zeros((0, Hkv, D), dtype=BF16),
                  w=torch.zeros((Hkv, 0), dtype=torch.float64), off=torch.zeros((Hkv, 0), dtype=torch.float64))
             for _ in range(B)]

    def append(new):
        slots = torch.empty(sum(new), dtype=torch.int32, device="cuda")
        mva.blocks_extend(seq, i32(new), table, page, free, count, pages, slots)
        k, v = (torch.randn((sum(new), Hkv, D), generator=gen).to(BF16) for _ in range(2))
        mva.gqa_cache_append(k_pool, v_pool, k.cuda(), v.cuda(), slots)
        at = 0
        for m, n in zip(model, new):
            m["k"], m["v"] = torch.cat([m["k"], k[at:at + n]]), torch.cat([m["v"], v[at:at + n]])
            m["w"], m["off"] = (torch.cat([m[x], torch.zeros((Hkv, n), dtype=torch.float64)], 1) for x in ("w", "off"))
            at += n

    def only(m, at):
        m["k"], m["v"], m["w"], m["off"] = m["k"][at], m["v"][at], m["w"][:, at], m["off"][:, at]

    def check():
        torch.cuda.synchronize()
        assert mva.last_device_error() == 0
        assert seq.tolist() == [len(m["k"]) for m in model]
        for b, m in enumerate(model):
            rows = plain.rows_of(table[b], page, len(m["k"]))
            assert torch.equal(k_pool.cpu()[rows], m["k"]) and torch.equal(v_pool.cpu()[rows], m["v"])
            off = (weights[b, :, :len(rows)].cpu().double() - m["w"]).abs()
            assert (off <= m["off"]).all(), "stream %d: off by %.3g" % (b, off.max())
            assert not weights[b, :, len(rows):].any()          # new tokens begin at 0

    append(first)
    for step in range(steps):
        append([q] * B)
        seen = trees(gen, B, q, "random")
        qs = torch.randn((B, q, H, D), generator=gen).to(BF16).cuda()
        mask = gqa_plain.mask_words(seen).cuda()
        out, lse = mva.gqa_verify_attn_paged(qs, k_pool, v_pool, table, page, seq, mask, scale)
        paths = [accepted_path(seen[b], gen) for b in range(B)]
        taken = torch.zeros((B, q), dtype=torch.bool)
        for b, path in enumerate(paths):
            taken[b, path] = True
        lse[~taken.cuda()] = float("inf")                         # rejected drafts' rows add nothing
        mva.gqa_attn_weights_paged(qs, k_pool, table, page, seq, mask, lse, scale, weights)
        for b, m in enumerate(model):
            n, see = len(m["k"]), plain.seen_keys(seen[b], len(m["k"]))
            want = plain.attend(qs[b].cpu(), m["k"], m["v"], see, scale)
            plain.check(out[b, taken[b].cuda()].cpu(), lse[b, taken[b].cuda()].cpu(), [x[taken[b]] for x in want])
            x = want[1].view(q, Hkv, H // Hkv, 1)
            qd, k = qs[b].cpu().double().view(q, Hkv, H // Hkv, D), m["k"].double()
            s = torch.einsum("ihgd,thd->ihgt", qd, k) * scale
            size = torch.einsum("ihgd,thd->ihgt", qd.abs(), k.abs()) * scale
            w = torch.where((see & taken[b][:, None])[:, None, None], (s - x).exp(), 0.0)
            # As in the tests of one call (test_attn_weights.py), and the error of the lse that it was given.
            e = (D + 4) * 2.0 ** -24 * size + 2.0 ** -22 + 2.0 ** -23 * (x.abs() + s.abs()) + want[3].view_as(x)
            m["w"] += w.sum((0, 2))
            m["off"] += (w * (1.01 * e + q * H * 2.0 ** -24)).sum((0, 2)) + 2.0 ** -23 * m["w"]
        # The accepted rows move, and their sums with them; the sums behind them become 0.
        lens = [len(m["k"]) for m in model]
        for m, path, n in zip(model, paths, lens):
            only(m, torch.cat([torch.arange(n - q), n - q + path]))
        if how == "keep":
            draft = torch.arange(q, device="cuda")
            path = torch.stack([torch.nn.functional.pad(p, (0, q - len(p))) for p in paths]).int().cuda()
            n_kept = i32([len(p) for p in paths])
            mva.gqa_cache_keep(k_pool, v_pool, table, page, seq, path, n_kept)
            prefix = (seq - q)[:, None]
            places = lambda d: (prefix + d)[:, None].expand(B, Hkv, q).long()
            behind = (draft >= n_kept[:, None])[:, None]
            weights.scatter_(2, places(draft), weights.gather(2, places(path)).masked_fill(behind, 0.0))
        else:
            at = torch.arange(smax)
            for b, (path, n) in enumerate(zip(paths, lens)):
                places = torch.cat([torch.arange(n - q), n - q + path])
                kept[b] = torch.where(at < len(places), torch.nn.functional.pad(places, (0, smax - len(places))), -1).int().cuda()
        keep.copy_(i32([len(m["k"]) for m in model]))
        if how == "compact":
            mva.gqa_cache_compact(k_pool, v_pool, table, page, seq, kept, keep, weights=weights)
        mva.blocks_trim(seq, keep, table, page, free, count)
        check()
        if step % 2:
            few = torch.empty((B, budget), dtype=torch.int32, device="cuda")
            mva.evict_select(weights, seq, 2, 10, few, keep)
            for b, m in enumerate(model):
                stay = plain.select(weights[b].cpu(), len(m["k"]), 2, 10, budget)
                assert few[b, :len(stay)].tolist() == stay
                only(m, torch.tensor(stay).long())
            mva.gqa_cache_compact(k_pool, v_pool, table, page, seq, few, keep, weights=weights)
            mva.blocks_trim(seq, keep, table, page, free, count)
            check()
