"""Memory that a call makes for itself: on another stream than the current one
it comes out of that stream's pool.  (Of the current stream's pool it could be
memory that work still queued there uses: the allocator hands a freed block out
again for later work on the same stream.)"""
import contextlib
import struct
import types

import pytest

torch = pytest.importorskip("torch")

import mla_verify_attention_gb300 as mva
from mla_verify_attention_gb300 import _lib, _serving

BF16 = torch.bfloat16
CURRENT, SIDE = 0, 77


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Tensor:
    """Stands in for a CUDA tensor: what the bindings ask of one."""

    def __init__(self, shape, dtype, made_on=None):
        self.shape, self.dtype, self.made_on = torch.Size(shape), dtype, made_on
        self.device, self.is_cuda, self.recorded = "cuda:0", True, []

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def is_floating_point(self):
        return self.dtype.is_floating_point

    def element_size(self):
        return self.dtype.itemsize

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 256

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class Pool:
    """torch's allocator as far as streams go: a block belongs to the stream that is current when it is made."""

    def __init__(self):
        self.now, self.made = [Stream(CURRENT)], []

    def empty(self, shape, dtype=None, device=None):
        t = Tensor([shape] if isinstance(shape, int) else shape, dtype, self.now[-1].cuda_stream)
        self.made.append(t)
        return t

    @contextlib.contextmanager
    def stream(self, s):
        self.now.append(s)
        try:
            yield
        finally:
            self.now.pop()

    def current_stream(self, device=None):
        return self.now[-1]


@pytest.fixture
def pool(monkeypatch):
    p = Pool()
    monkeypatch.setattr(torch, "empty", p.empty)
    monkeypatch.setattr(torch.cuda, "stream", p.stream)
    monkeypatch.setattr(torch.cuda, "current_stream", p.current_stream)
    p.launched = []

    def packed(which, args):
        p.launched.append(struct.unpack("=q", args[-8:])[0])
        return 0

    _serving._bind()
    monkeypatch.setattr(_serving, "_call", packed)
    monkeypatch.setattr(_serving, "_current_device", lambda: 0)
    monkeypatch.setattr(_serving, "_current_stream", lambda dev: p.now[-1].cuda_stream)
    monkeypatch.setattr(_serving, "gqa_workspace_size", lambda *a: 4096)

    class Library:
        @staticmethod
        def mla_verify_attn(*a):
            p.launched.append(a[-1])
            return 0
        mla_verify_attn_paged = mla_verify_attn

    monkeypatch.setattr(_lib, "load_library", Library)
    monkeypatch.setattr(_lib, "workspace_size", lambda *a: 4096)
    monkeypatch.setattr(_lib, "paged_workspace_size", lambda *a: 4096)
    return p


def ints(*shape):
    return Tensor(shape, torch.int32)


def half(*shape):
    return Tensor(shape, BF16)


def grouped(**kw):
    return mva.gqa_verify_attn(half(1, 5, 8, 64), half(1, 90, 2, 64), half(1, 90, 2, 64), ints(1), ints(1, 5, 1), 0.1, **kw)


def grouped_paged(**kw):
    return mva.gqa_verify_attn_paged(half(1, 5, 8, 64), half(96, 2, 64), half(96, 2, 64), ints(1, 6), 16, ints(1),
                                     ints(1, 5, 1), 0.1, **kw)


@pytest.mark.parametrize("call", [grouped, grouped_paged])
def test_grouped_heads_memory_is_the_streams_own(pool, call):
    out, lse = call(stream=Stream(SIDE))
    assert pool.launched == [SIDE] and len(pool.made) == 3
    for t in pool.made:
        assert t.made_on == SIDE
    # The results are the current stream's to read: not handed out again before its work so far is done.
    assert out.recorded == [CURRENT] and lse.recorded == [CURRENT]
    assert pool.current_stream().cuda_stream == CURRENT


@pytest.mark.parametrize("call", [grouped, grouped_paged])
@pytest.mark.parametrize("stream", [None, Stream(CURRENT)])
def test_grouped_heads_memory_on_the_current_stream(pool, call, stream):
    out, lse = call(stream=stream)
    assert pool.launched == [CURRENT] and [t.made_on for t in pool.made] == [CURRENT] * 3
    assert not out.recorded and not lse.recorded


@pytest.mark.parametrize("call", [grouped, grouped_paged])
def test_grouped_heads_memory_of_the_caller(pool, call):
    given = dict(out=half(1, 5, 8, 64), lse=Tensor((1, 5, 8), torch.float32), workspace=Tensor((4096,), torch.uint8))
    out, lse = call(stream=Stream(SIDE), **given)
    assert out is given["out"] and lse is given["lse"] and not pool.made and pool.launched == [SIDE]


def latent(**kw):
    return mva.verify_attn(half(1, 5, 8, 512), half(1, 5, 8, 64), half(1, 90, 576), ints(1), ints(1, 5, 1), 0.1, **kw)


def latent_paged(**kw):
    return mva.verify_attn_paged(half(1, 5, 8, 512), half(1, 5, 8, 64), half(96, 576), ints(1, 6), 16, ints(1),
                                 ints(1, 5, 1), 0.1, **kw)


@pytest.mark.parametrize("call", [latent, latent_paged])
def test_latent_memory_is_the_streams_own(pool, call):
    out, lse = call(stream=Stream(SIDE))
    assert pool.launched == [SIDE] and [t.made_on for t in pool.made] == [SIDE] * 3
    assert out.recorded == [CURRENT] and lse.recorded == [CURRENT]
    assert [t.recorded for t in pool.made[2:]] == [[]]


@pytest.mark.parametrize("call", [latent, latent_paged])
@pytest.mark.parametrize("stream", [None, Stream(CURRENT)])
def test_latent_memory_on_the_current_stream(pool, call, stream):
    out, lse = call(stream=stream)
    assert pool.launched == [CURRENT] and [t.made_on for t in pool.made] == [CURRENT] * 3
    assert not out.recorded and not lse.recorded


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
def test_calls_on_two_streams_share_no_memory(page, monkeypatch):
    """The first call is held back behind other work when the second one, on another stream, makes its memory."""
    gen = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen).to(BF16).cuda()
    B, q, H, Hkv, D, n = 2, 9, 16, 2, 128, 4000
    lens = torch.full((B,), n, dtype=torch.int32).cuda()
    mask = torch.tensor([(2 << i) - 1 for i in range(q)], dtype=torch.int32).view(1, q, 1).expand(B, q, 1).contiguous().cuda()
    k, v = rand(B * n, Hkv, D), rand(B * n, Hkv, D)
    table = torch.arange(B * n // 16, dtype=torch.int32).view(B, -1).cuda()
    queries = [rand(B, q, H, D) for _ in range(2)]

    def call(x, stream=None):
        if page:
            return mva.gqa_verify_attn_paged(x, k, v, table, page, lens, mask, 0.1, stream=stream)
        return mva.gqa_verify_attn(x, k.view(B, n, Hkv, D), v.view(B, n, Hkv, D), lens, mask, 0.1, stream=stream)

    want = [call(x) for x in queries]
    work = torch.randn((8192, 8192), device="cuda")
    side = torch.cuda.Stream()
    used = []
    kept = _serving._call

    def noted(which, args):
        out, lse, ws, ws_bytes, handle = struct.unpack("=5q", args[-40:])
        used.append((ws, ws + ws_bytes))
        return kept(which, args)

    torch.cuda.synchronize()
    monkeypatch.setattr(_serving, "_call", noted)
    for _ in range(4):
        torch.mm(work, work)                       # the current stream's calls wait behind this
    first = call(queries[0])
    second = call(queries[1], stream=side)
    third = call(queries[0])
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert mva.last_device_error() == 0
    for other in (used[0], used[2]):
        assert used[1][1] <= other[0] or other[1] <= used[1][0]
    for got, ref in ((first, want[0]), (second, want[1]), (third, want[0])):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
def test_latent_calls_on_two_streams_share_no_memory(page, monkeypatch):
    gen = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(s, generator=gen).to(BF16).cuda()
    B, q, H, n = 1, 9, 64, 4000
    lens = torch.full((B,), n, dtype=torch.int32).cuda()
    mask = torch.tensor([(2 << i) - 1 for i in range(q)], dtype=torch.int32).view(1, q, 1).cuda()
    kv, table = rand(n, 576), torch.arange(n // 16, dtype=torch.int32).view(B, -1).cuda()
    queries = [(rand(B, q, H, 512), rand(B, q, H, 64)) for _ in range(2)]

    def call(x, stream=None):
        if page:
            return mva.verify_attn_paged(*x, kv, table, page, lens, mask, 0.07, stream=stream)
        return mva.verify_attn(*x, kv.view(B, n, 576), lens, mask, 0.07, stream=stream)

    want = [call(x) for x in queries]
    work = torch.randn((8192, 8192), device="cuda")
    side = torch.cuda.Stream()
    used = []
    empty = torch.empty

    def noted(shape, **kw):
        t = empty(shape, **kw)
        if t.dtype == torch.uint8:
            used.append((t.data_ptr(), t.data_ptr() + t.numel()))
        return t

    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", noted)
    for _ in range(4):
        torch.mm(work, work)                       # the current stream's calls wait behind this
    first = call(queries[0])
    second = call(queries[1], stream=side)
    third = call(queries[0])
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert mva.last_device_error() == 0 and len(used) == 3
    for other in (used[0], used[2]):
        assert used[1][1] <= other[0] or other[1] <= used[1][0]
    for got, ref in ((first, want[0]), (second, want[1]), (third, want[0])):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.gpu
def test_captured_calls_on_two_streams():
    """A capture that forks and joins, with memory that the calls make themselves on either stream."""
    gen = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=gen).to(BF16).cuda()
    B, q, H, Hkv, D, n = 2, 9, 16, 2, 128, 900
    lens = torch.tensor([n, n - 30], dtype=torch.int32).cuda()
    mask = torch.tensor([(2 << i) - 1 for i in range(q)], dtype=torch.int32).view(1, q, 1).expand(B, q, 1).contiguous().cuda()
    k, v, queries = rand(B, n, Hkv, D), rand(B, n, Hkv, D), [rand(B, q, H, D) for _ in range(3)]
    kv, qn, qr = rand(B, n, 576), rand(B, q, 64, 512), rand(B, q, 64, 64)
    grouped = lambda x, **kw: mva.gqa_verify_attn(x, k, v, lens, mask, 0.1, **kw)
    latent = lambda **kw: mva.verify_attn(qn, qr, kv, lens, mask, 0.07, **kw)
    want = [grouped(x) for x in queries] + [latent()]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        first = queries[0] + 0                     # work of another kind before the fork
        side.wait_stream(here)
        on_side = grouped(queries[1], stream=side), latent(stream=side)
        on_main = grouped(first)
        here.wait_stream(side)
        joined = grouped(queries[2])               # behind both streams
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert mva.last_device_error() == 0
    for got, ref in zip((on_main, on_side[0], joined, on_side[1]), want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
