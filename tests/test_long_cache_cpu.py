"""The entry points that keep a long cache small, without a GPU: host-side
argument checks return their codes before the device is touched, the packed
calls return what the calls do, and the bindings refuse what they cannot pass on."""
import struct

import pytest

import mla_verify_attention_gb300 as mva

OK, NULL, SHAPE, ALIGN, WORKSPACE, NO_DEVICE, ARG = 0, -1, -2, -3, -4, -5, -9


@pytest.fixture(scope="module")
def lib():
    return mva.load_library()


def no_device():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a device is present")


def call(f, args, **kw):
    a = dict(args)
    a.update(kw)
    return f(*a.values())


WINDOW = dict(q=16, k=16, v=16, strides=None, lens=16, mask=16, B=1, q_len=9, H=64, Hkv=8, D=128, Smax=320, dtype=0,
              scale=0.1, window=100, sinks=4, out=16, lse=16, ws=256, ws_bytes=1 << 30, stream=None)
WINDOW_PAGED = dict(q=16, k=16, v=16, strides=None, rows=640, table=16, max_blocks=5, page=64, lens=16, mask=16, B=1,
                    q_len=9, H=64, Hkv=8, D=128, dtype=0, scale=0.1, window=100, sinks=4, out=16, lse=16, ws=256,
                    ws_bytes=1 << 30, stream=None)
APPEND = dict(k=16, ks=2048, v=16, vs=2048, Hkv=8, D=128, dtype=0, kf=1.0, vf=0.5, kp=16, kps=576, vp=16, vps=576, rows=100,
              slots=16, T=3, kh=16, khs=2048, vh=16, vhs=2048, stream=None)
FP4 = dict(q=16, strides=None, k=16, ks=576, v=16, vs=576, rows=640, table=16, max_blocks=5, page=64, lens=16, mask=16, B=1,
           q_len=9, H=64, Hkv=8, D=128, dtype=0, scale=0.1, kf=1.0, vf=0.5, out=16, lse=16, ws=256, ws_bytes=1 << 30, stream=None)
WEIGHTS = dict(q=16, k=16, strides=None, lens=16, mask=16, lse=16, B=1, q_len=9, H=64, Hkv=8, D=128, Smax=320, dtype=0,
               scale=0.1, w=16, stream=None)
WEIGHTS_PAGED = dict(q=16, k=16, strides=None, rows=640, table=16, max_blocks=5, page=64, lens=16, mask=16, lse=16, B=1,
                     q_len=9, H=64, Hkv=8, D=128, dtype=0, scale=0.1, w=16, stream=None)
SELECT = dict(w=16, lens=16, B=2, Hkv=2, Smax=500, sinks=4, recent=10, kept=16, budget=50, keep=16, ws=16, ws_bytes=0, stream=None)
COMPACT = dict(pa=16, pas=1024, na=1024, pb=16, pbs=1024, nb=1024, rows=640, w=16, Hkv=2, table=16, max_blocks=5, page=64,
               lens=16, kept=16, budget=50, keep=16, B=2, stream=None)
CALLS = {"mla_gqa_verify_attn_window": (8, WINDOW), "mla_gqa_verify_attn_window_paged": (9, WINDOW_PAGED),
         "mla_gqa_cache_append_fp4": (10, APPEND), "mla_evict_select": (11, SELECT), "mla_cache_compact": (12, COMPACT),
         "mla_gqa_attn_weights": (13, WEIGHTS), "mla_gqa_attn_weights_paged": (14, WEIGHTS_PAGED),
         "mla_gqa_verify_attn_fp4_paged": (15, FP4)}


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(q_len=0), SHAPE), (dict(D=96), SHAPE),
    (dict(H=63), SHAPE), (dict(Smax=0), SHAPE), (dict(dtype=2), ARG), (dict(scale=float("inf")), ARG), (dict(q=0), NULL),
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(lens=0), NULL), (dict(mask=0), NULL), (dict(out=0), NULL), (dict(lse=0), NULL),
    (dict(k=24), ALIGN), (dict(ws=272), ALIGN), (dict(B=0, q=0), OK)])
def test_window_arguments(lib, kw, want):
    assert call(lib.mla_gqa_verify_attn_window, WINDOW, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), SHAPE), (dict(sinks=-2), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=0), SHAPE), (dict(rows=100), SHAPE),
    (dict(max_blocks=1 << 18), SHAPE), (dict(table=0), NULL), (dict(table=6), ALIGN)])
def test_window_paged_arguments(lib, kw, want):
    assert call(lib.mla_gqa_verify_attn_window_paged, WINDOW_PAGED, **kw) == want


def test_fp4_row_bytes():
    for Hkv in (1, 2, 3, 8, 40, 4096):
        for D in (64, 128):
            n = mva.gqa_fp4_row_bytes(Hkv, D)
            assert n % 16 == 0 and 0 <= n - Hkv * (D // 2 + D // 16) < 16
    assert [mva.gqa_fp4_row_bytes(*x) for x in ((0, 64), (-1, 64), (4097, 64), (8, 96))] == [0] * 4


@pytest.mark.parametrize("kw,want", [
    (dict(Hkv=0), SHAPE), (dict(Hkv=4097), SHAPE), (dict(D=32), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE),
    (dict(rows=0), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(kps=560), SHAPE), (dict(vps=0), SHAPE), (dict(ks=-16), SHAPE),
    (dict(khs=1024), SHAPE), (dict(dtype=2), ARG), (dict(kf=0.0), ARG), (dict(kf=-1.0), ARG), (dict(vf=float("nan")), ARG),
    (dict(vf=1e30), ARG), (dict(k=0), NULL), (dict(v=0), NULL), (dict(kp=0), NULL), (dict(vp=0), NULL), (dict(slots=0), NULL),
    (dict(k=8), ALIGN), (dict(kp=8), ALIGN), (dict(kps=584), ALIGN), (dict(ks=2056), ALIGN), (dict(kh=8), ALIGN),
    (dict(khs=2056), ALIGN), (dict(slots=2), ALIGN), (dict(T=0, k=0), OK)])
def test_append_fp4_arguments(lib, kw, want):
    assert call(lib.mla_gqa_cache_append_fp4, APPEND, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(Hkv=5), SHAPE), (dict(D=96), SHAPE), (dict(ks=560), SHAPE), (dict(vs=1 << 33), SHAPE), (dict(page=0), SHAPE),
    (dict(rows=100), SHAPE), (dict(q_len=65), SHAPE), (dict(dtype=3), ARG), (dict(kf=0.0), ARG), (dict(vf=float("inf")), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=1e38, kf=1e10), ARG), (dict(q=0), NULL), (dict(k=0), NULL), (dict(table=0), NULL),
    (dict(lse=0), NULL), (dict(ks=584), ALIGN), (dict(v=24), ALIGN), (dict(ws=16), ALIGN), (dict(B=0, q=0), OK)])
def test_fp4_attention_arguments(lib, kw, want):
    assert call(lib.mla_gqa_verify_attn_fp4_paged, FP4, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q_len=0), SHAPE), (dict(H=63), SHAPE), (dict(D=32), SHAPE), (dict(Smax=1 << 24), SHAPE), (dict(B=-1), SHAPE),
    (dict(dtype=2), ARG), (dict(scale=float("nan")), ARG), (dict(q=0), NULL), (dict(k=0), NULL), (dict(lens=0), NULL),
    (dict(mask=0), NULL), (dict(lse=0), NULL), (dict(w=0), NULL), (dict(k=8), ALIGN), (dict(w=2), ALIGN), (dict(lse=6), ALIGN),
    (dict(B=0, w=0), OK)])
def test_weights_arguments(lib, kw, want):
    assert call(lib.mla_gqa_attn_weights, WEIGHTS, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(page=0), SHAPE), (dict(rows=10), SHAPE), (dict(max_blocks=0), SHAPE), (dict(table=0), NULL), (dict(table=2), ALIGN)])
def test_weights_paged_arguments(lib, kw, want):
    assert call(lib.mla_gqa_attn_weights_paged, WEIGHTS_PAGED, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(B=1 << 20), SHAPE), (dict(Smax=0), SHAPE), (dict(Smax=1 << 24), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(Hkv=65537), SHAPE), (dict(budget=0), SHAPE), (dict(sinks=-1), SHAPE), (dict(recent=-1), SHAPE),
    (dict(sinks=41), SHAPE), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), SHAPE),
    (dict(budget=(1 << 30) + 1), SHAPE), (dict(w=0), NULL), (dict(lens=0), NULL),
    (dict(kept=0), NULL), (dict(keep=0), NULL), (dict(w=2), ALIGN), (dict(kept=6), ALIGN), (dict(B=0, w=0), OK)])
def test_select_arguments(lib, kw, want):
    assert call(lib.mla_evict_select, SELECT, **kw) == want


def test_select_workspace():
    assert mva.evict_workspace_size(3, 393216) == 0 and mva.evict_workspace_size(3, 393217) == 12 * 393217
    assert mva.evict_workspace_size(-1, 400000) == 0 and mva.evict_workspace_size(1, 1 << 24) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(budget=0), SHAPE), (dict(max_blocks=0), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=1 << 28), SHAPE),
    (dict(max_blocks=(1 << 24) + 1, rows=1 << 30), SHAPE), (dict(budget=(1 << 30) + 1), SHAPE), (dict(na=0), SHAPE), (dict(nb=-16), SHAPE), (dict(rows=10), SHAPE), (dict(pas=512), SHAPE), (dict(pbs=512), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(pa=0), NULL), (dict(pb=0), NULL), (dict(table=0), NULL), (dict(lens=0), NULL), (dict(kept=0), NULL),
    (dict(keep=0), NULL), (dict(pa=8), ALIGN), (dict(na=1000), ALIGN), (dict(pbs=1032), ALIGN), (dict(w=2), ALIGN),
    (dict(kept=2), ALIGN), (dict(B=0, pa=0), OK)])
def test_compact_arguments(lib, kw, want):
    assert call(lib.mla_cache_compact, COMPACT, **kw) == want


def test_strides(lib):
    import ctypes
    good = [9 * 64 * 128, 64 * 128, 128, 320 * 1024, 1024, 128, 320 * 1024, 1024, 128]
    arr = lambda x: ctypes.cast((ctypes.c_longlong * 9)(*x), ctypes.c_void_p)
    for name, args, used in (("mla_gqa_verify_attn_window", WINDOW, 9), ("mla_gqa_attn_weights", WEIGHTS, 6),
                             ("mla_gqa_verify_attn_fp4_paged", FP4, 3)):
        for i, bad, want in ((1, 64 * 128 + 4, ALIGN), (2, -128, SHAPE), (4, 0, SHAPE), (5, 1 << 38, SHAPE), (7, 4, SHAPE)):
            if i < used:
                x = list(good)
                x[i] = bad
                assert call(getattr(lib, name), args, strides=arr(x)) == want, (name, i)


def test_packed_calls(lib):
    # The same statuses as the calls themselves, argument by argument.
    no_device()                           # (the addresses are made up)

    def packed(which, args):
        v = [x if x is not None else 0 for x in args.values()]
        return lib.mla_call_packed(which, b"".join(struct.pack("=d" if isinstance(x, float) else "=q", x) for x in v))

    for name, (which, args) in CALLS.items():
        f = getattr(lib, name)
        assert call(f, args) == packed(which, args) == NO_DEVICE, name
        for key, value in args.items():
            if key in ("stream", "strides", "ws_bytes"):
                continue
            for bad in (0, -1, 2, 1 << 20):
                a = dict(args)
                a[key] = float(bad) if isinstance(value, float) else bad
                assert packed(which, a) == call(f, a), (name, key, bad)
    assert packed(11, dict(SELECT, B=(1 << 32) + 2)) == SHAPE       # more than an int holds
    for unknown in (6, 7, 16, -1):
        assert lib.mla_call_packed(unknown, b"\0" * 300) == ARG


def test_without_a_device(lib):
    no_device()
    assert lib.mla_gqa_fp4_workspace_size(1, 9, 64, 8, 128) == 0


def test_bindings_want_cuda_tensors():
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(s)
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)
    for bad in (lambda: mva.gqa_verify_attn_window(h(1, 2, 4, 64), h(1, 9, 2, 64), h(1, 9, 2, 64), i(1), i(1, 2, 1), 0.1, 5,
                                                   workspace=h(1)),
                lambda: mva.gqa_verify_attn_window_paged(h(1, 2, 4, 64), h(9, 2, 64), h(9, 2, 64), i(1, 3), 3, i(1), i(1, 2, 1),
                                                         0.1, 5, 1, workspace=h(1)),
                lambda: mva.gqa_cache_append_fp4(u(9, 80), u(9, 80), h(3, 2, 64), h(3, 2, 64), i(3)),
                lambda: mva.gqa_verify_attn_fp4_paged(h(1, 2, 4, 64), u(9, 80), u(9, 80), 2, i(1, 3), 3, i(1), i(1, 2, 1), 0.1,
                                                      workspace=h(1)),
                lambda: mva.gqa_cache_keep_fp4(u(9, 80), u(9, 80), i(2, 3), 3, i(2), i(2, 4), i(2)),
                lambda: mva.gqa_attn_weights(h(1, 2, 4, 64), h(1, 9, 2, 64), i(1), i(1, 2, 1), f(1, 2, 4), 0.1, f(1, 2, 9)),
                lambda: mva.gqa_attn_weights_paged(h(1, 2, 4, 64), h(9, 2, 64), i(1, 3), 3, i(1), i(1, 2, 1), f(1, 2, 4), 0.1,
                                                   f(1, 2, 9)),
                lambda: mva.evict_select(f(2, 2, 9), i(2), 0, 1, i(2, 4), i(2)),
                lambda: mva.gqa_cache_compact(h(9, 2, 64), h(9, 2, 64), i(2, 3), 3, i(2), i(2, 4), i(2)),
                lambda: mva.gqa_cache_compact(u(9, 80), u(9, 80), i(2, 3), 3, i(2), i(2, 4), i(2), weights=f(2, 2, 9)),
                lambda: mva.cache_compact(h(9, 576), i(2, 3), 3, i(2), i(2, 4), i(2))):
        with pytest.raises(ValueError, match="CUDA"):
            bad()
