"""Kernels that start before the grid ahead of them has ended read what it writes.

Every kernel of the library is launched as a programmatic dependent: it may
start while the grid before it runs, and waits for it.  Read-only loads are not
allowed to see what is written meanwhile; ordinary loads behind the wait are."""
import glob
import os
import re

import pytest

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
from mla_verify_attention_gb300 import _build
import gqa_plain as plain

BF16 = torch.bfloat16


def test_no_read_only_loads():
    for path in _build.sources():
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        assert not re.search(r"__ldg\b|\bld\.global(\.\w+)*\.nc\b|__restrict__", code), os.path.basename(path)


class Steps:
    """Steps of a cache on few pages: each trims the streams to other lengths, extends them and writes new rows,
    so that lengths, block table, slots and pool rows differ from step to step.  All inputs are made before."""

    def __init__(self, page, pools, rows, steps=12):
        gen = torch.Generator().manual_seed(page)
        self.B, self.q, self.page, self.pools = 3, 9, page, pools
        self.max_blocks = -(-700 // page)
        self.pages = pools[0].shape[0] // page
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
        self.lens, self.table = i32([0] * self.B), torch.zeros((self.B, self.max_blocks), dtype=torch.int32).cuda()
        self.free = torch.randperm(self.pages, generator=gen).to(torch.int32).cuda()
        self.count = i32([self.pages])
        self.slots = torch.zeros(self.B * 700, dtype=torch.int32).cuda()
        seen = torch.ones(self.q, self.q).tril().bool().expand(self.B, self.q, self.q)
        self.mask = plain.mask_words(seen).cuda()
        at = [0] * self.B
        self.steps = []
        for _ in range(steps):
            keep = [int(x) for x in (torch.rand(self.B, generator=gen) * torch.tensor([n + 1 for n in at]))]
            new = [int(x) for x in torch.randint(self.q, 690, (self.B,), generator=gen)]
            new = [min(n, 690 - k) for n, k in zip(new, keep)]
            at = [k + n for k, n in zip(keep, new)]
            self.steps.append((i32(keep), i32(new), rows(gen, self.B * 700)))

    def move(self, keep, new):
        mva.blocks_trim(self.lens, keep, self.table, self.page, self.free, self.count)
        mva.blocks_extend(self.lens, new, self.table, self.page, self.free, self.count, self.pages, self.slots)

    def run(self, append, attend, sync):
        start = [x.clone() for x in (self.lens, self.table, self.free, self.count, *self.pools)]
        torch.cuda.synchronize()
        got = []
        for keep, new, rows in self.steps:
            for call in (lambda: self.move(keep, new), lambda: append(rows), lambda: got.append(attend(rows))):
                call()
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert mva.last_device_error() == 0
        for x, y in zip((self.lens, self.table, self.free, self.count, *self.pools), start):
            x.copy_(y)
        return got

    def same(self, append, attend):
        """One call at a time, and all of them behind each other."""
        want = self.run(append, attend, True)
        for _ in range(5):
            for a, b in zip(self.run(append, attend, False), want):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [64, 16, 5])
def test_steps_behind_each_other_with_keys_and_values(page):
    Hkv, H, D = 2, 8, 64
    rand = lambda gen, *s: torch.randn(s, generator=gen).to(BF16).cuda()
    pools = [torch.zeros((-(-2100 // page) * page + 4 * page, Hkv, D), dtype=BF16, device="cuda") for _ in range(2)]
    s = Steps(page, pools, lambda gen, n: (rand(gen, n, Hkv, D), rand(gen, n, Hkv, D), rand(gen, 3, 9, H, D)))
    s.same(lambda r: mva.gqa_cache_append(pools[0], pools[1], r[0], r[1], s.slots),
           lambda r: mva.gqa_verify_attn_paged(r[2], pools[0], pools[1], s.table, page, s.lens, s.mask, 0.125))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [64, 16])
def test_steps_behind_each_other_with_the_latent_cache(page):
    H = 8
    rand = lambda gen, *s: torch.randn(s, generator=gen).to(BF16).cuda()
    pool = torch.zeros((-(-2100 // page) * page + 4 * page, 576), dtype=BF16, device="cuda")
    s = Steps(page, [pool], lambda gen, n: (rand(gen, n, 576), rand(gen, 3, 9, H, 512), rand(gen, 3, 9, H, 64)))
    s.same(lambda r: mva.cache_append(pool, r[0][:, :512], r[0][:, 512:], s.slots),
           lambda r: mva.verify_attn_paged(r[1], r[2], pool, s.table, page, s.lens, s.mask, 0.07))
