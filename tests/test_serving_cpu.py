"""The grouped-head and cache entry points without a GPU: host-side argument
checks return their codes before the device is touched."""
import pytest

import mla_verify_attention_gb300 as mva

OK, NULL, SHAPE, ALIGN, NO_DEVICE, ARG = 0, -1, -2, -3, -5, -9


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


GQA = dict(q=16, k=16, v=16, strides=None, lens=16, mask=16, B=1, q_len=9, H=64, Hkv=8, D=128, Smax=320, dtype=0,
           scale=0.1, out=16, lse=16, ws=256, ws_bytes=1 << 30, stream=None)
PAGED = dict(q=16, k=16, v=16, strides=None, rows=640, table=16, max_blocks=5, page=64, lens=16, mask=16, B=1, q_len=9,
             H=64, Hkv=8, D=128, dtype=0, scale=0.1, out=16, lse=16, ws=256, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q_len=0), SHAPE), (dict(q_len=65), SHAPE), (dict(H=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(H=63), SHAPE),
    (dict(D=96), SHAPE), (dict(B=-1), SHAPE), (dict(B=1 << 20), SHAPE), (dict(B=1 << 16, Smax=1 << 18), SHAPE), (dict(Smax=0), SHAPE),
    (dict(Smax=1 << 24), SHAPE), (dict(dtype=2), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(lens=0), NULL), (dict(mask=0), NULL),
    (dict(out=0), NULL), (dict(lse=0), NULL), (dict(k=24), ALIGN), (dict(out=8), ALIGN), (dict(ws=272), ALIGN),
    (dict(lse=2), ALIGN), (dict(B=0, q=0, k=0), OK)])
def test_gqa_arguments(lib, kw, want):
    assert call(lib.mla_gqa_verify_attn, GQA, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(page=0), SHAPE), (dict(max_blocks=0), SHAPE), (dict(rows=100), SHAPE), (dict(rows=0), SHAPE),
    (dict(max_blocks=1 << 18), SHAPE), (dict(table=0), NULL), (dict(table=6), ALIGN), (dict(H=65), SHAPE)])
def test_gqa_paged_arguments(lib, kw, want):
    assert call(lib.mla_gqa_verify_attn_paged, PAGED, **kw) == want


def test_gqa_strides(lib):
    import ctypes
    good = [9 * 64 * 128, 64 * 128, 128, 320 * 1024, 1024, 128, 320 * 1024, 1024, 128]
    arr = lambda x: ctypes.cast((ctypes.c_longlong * 9)(*x), ctypes.c_void_p)
    for i, bad, want in ((1, 64 * 128 + 4, ALIGN), (4, 0, SHAPE), (5, -128, SHAPE), (7, 1 << 38, SHAPE)):
        x = list(good)
        x[i] = bad
        assert call(lib.mla_gqa_verify_attn, GQA, strides=arr(x)) == want, i
    no_device()
    x = list(good)
    x[0] = x[3] = 3                       # batch strides of one stream are not used
    assert call(lib.mla_gqa_verify_attn, GQA, strides=arr(x)) == NO_DEVICE


EXTEND = dict(lens=16, new=16, table=16, B=2, max_blocks=4, page=16, free=16, cap=8, count=16, pages=8, slots=16,
              tokens=18, stream=None)
TRIM = dict(lens=16, keep=16, table=16, B=2, max_blocks=4, page=16, free=16, cap=8, count=16, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(B=16385), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(max_blocks=1 << 28), SHAPE), (dict(cap=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 28), SHAPE), (dict(lens=0), NULL), (dict(new=0), NULL), (dict(table=0), NULL), (dict(free=0), NULL),
    (dict(count=0), NULL), (dict(slots=0), NULL), (dict(slots=8), ALIGN), (dict(lens=2), ALIGN),
    (dict(B=0, tokens=0), OK)])
def test_extend_arguments(lib, kw, want):
    assert call(lib.mla_blocks_extend, EXTEND, **kw) == want


def test_block_counts_that_sums_cannot_tell_apart(lib):
    # Sums stop at 2^31 - 1, which has to be more than any limit.
    most = 2 ** 31 - 2
    assert call(lib.mla_blocks_extend, EXTEND, tokens=most + 1) == SHAPE
    assert call(lib.mla_blocks_extend, EXTEND, cap=most + 1) == SHAPE
    assert call(lib.mla_blocks_trim, TRIM, cap=most + 1) == SHAPE
    no_device()
    assert call(lib.mla_blocks_extend, EXTEND, tokens=most, cap=most) == NO_DEVICE
    assert call(lib.mla_blocks_trim, TRIM, cap=most) == NO_DEVICE


@pytest.mark.parametrize("kw,want", [
    (dict(B=16385), SHAPE), (dict(page=0), SHAPE), (dict(cap=-1), SHAPE), (dict(keep=0), NULL), (dict(count=0), NULL),
    (dict(table=2), ALIGN), (dict(B=0), OK)])
def test_trim_arguments(lib, kw, want):
    assert call(lib.mla_blocks_trim, TRIM, **kw) == want


APPEND = dict(a=16, sa=1024, na=1024, pa=16, psa=1152, b=16, sb=128, nb=128, pb=1040, psb=1152, rows=100, slots=16, T=3,
              stream=None)
KEEP = dict(pa=16, psa=1152, na=1152, pb=0, psb=0, nb=0, rows=640, table=16, max_blocks=5, page=64, lens=16, path=16,
            keep=16, B=2, q=9, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(na=0), SHAPE), (dict(nb=-16), SHAPE), (dict(rows=0), SHAPE), (dict(rows=1 << 31), SHAPE),
    (dict(psa=512), SHAPE), (dict(sa=-1024), SHAPE), (dict(na=1000), ALIGN), (dict(sa=1000), ALIGN), (dict(psb=1160), ALIGN),
    (dict(pa=8), ALIGN), (dict(a=8), ALIGN), (dict(pa=0), NULL), (dict(a=0), NULL), (dict(b=0), NULL), (dict(pb=0), NULL),
    (dict(slots=0), NULL), (dict(slots=2), ALIGN), (dict(T=0), OK)])
def test_append_arguments(lib, kw, want):
    assert call(lib.mla_cache_append, APPEND, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), SHAPE), (dict(q=65), SHAPE), (dict(B=-1), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(rows=10), SHAPE), (dict(na=1150), ALIGN), (dict(pa=0), NULL), (dict(table=0), NULL), (dict(path=0), NULL),
    (dict(keep=0), NULL), (dict(lens=0), NULL), (dict(path=2), ALIGN), (dict(B=0), OK)])
def test_keep_arguments(lib, kw, want):
    assert call(lib.mla_cache_keep, KEEP, **kw) == want


def test_packed_calls(lib):
    # The same statuses as the calls themselves, argument by argument.
    import struct
    no_device()                           # (the addresses are made up)
    names = dict(enumerate((EXTEND, TRIM, APPEND, KEEP, GQA, PAGED)))
    fns = (lib.mla_blocks_extend, lib.mla_blocks_trim, lib.mla_cache_append, lib.mla_cache_keep,
           lib.mla_gqa_verify_attn, lib.mla_gqa_verify_attn_paged)

    def packed(which, args):
        v = [x if x is not None else 0 for x in args.values()]
        return lib.mla_call_packed(which, b"".join(struct.pack("=d" if isinstance(x, float) else "=q", x) for x in v))

    for which, args in names.items():
        for key, value in args.items():
            if key in ("stream", "strides", "ws_bytes"):
                continue
            for bad in (0, -1, 2, 1 << 20):
                a = dict(args)
                a[key] = float(bad) if isinstance(value, float) else bad
                want = call(fns[which], a)
                if want not in (OK, NO_DEVICE):
                    assert packed(which, a) == want, (which, key, bad)
            if isinstance(value, int) and 0 < value < 4096 and value != 16 and key not in ("pb", "ws"):
                a = dict(args)
                a[key] = 1 << 40
                assert packed(which, a) != OK
    assert packed(1, dict(TRIM, B=(1 << 32) + 2)) == SHAPE          # more than an int holds
    assert packed(4, dict(GQA, scale=float("nan"))) == ARG
    assert lib.mla_call_packed(6, b"\0" * 200) == ARG and lib.mla_call_packed(0, None) == NULL


def test_without_a_device(lib):
    no_device()
    for f, a in ((lib.mla_gqa_verify_attn, GQA), (lib.mla_gqa_verify_attn_paged, PAGED), (lib.mla_blocks_extend, EXTEND),
                 (lib.mla_blocks_trim, TRIM), (lib.mla_cache_append, APPEND), (lib.mla_cache_keep, KEEP)):
        assert call(f, a) == NO_DEVICE
    assert lib.mla_gqa_workspace_size(1, 9, 64, 8, 128) == 0


def test_bindings_want_cuda_tensors():
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for bad in (lambda: mva.gqa_verify_attn(h(1, 2, 4, 64), h(1, 9, 2, 64), h(1, 9, 2, 64), i(1), i(1, 2, 1), 0.1,
                                            workspace=h(1)),
                lambda: mva.blocks_extend(i(2), i(2), i(2, 3), 4, i(5), i(1), 5, i(8)),
                lambda: mva.blocks_trim(i(2), i(2), i(2, 3), 4, i(5), i(1)),
                lambda: mva.cache_append(h(9, 576), h(3, 512), h(3, 64), i(3)),
                lambda: mva.gqa_cache_append(h(9, 2, 64), h(9, 2, 64), h(3, 2, 64), h(3, 2, 64), i(3)),
                lambda: mva.cache_keep(h(9, 576), i(2, 3), 3, i(2), i(2, 4), i(2)),
                lambda: mva.gqa_cache_keep(h(9, 2, 64), h(9, 2, 64), i(2, 3), 3, i(2), i(2, 4), i(2))):
        with pytest.raises(ValueError, match="CUDA"):
            bad()
